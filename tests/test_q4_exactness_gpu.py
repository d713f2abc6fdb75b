"""How many outputs of the 4-bit attention calls are not the correctly rounded ones,
at the lengths the calls are made for.

An output rounds to a neighbour of the right number where the error before the
rounding carries it over the middle between two numbers.  With errors much smaller
than a step that happens to a share of E|error| / step of the outputs, so the share
measures the error before the rounding, which the rounding itself hides.

The yardstick is computed on the same data in 64 bits: attention whose weights
p * scale are rounded once to half precision (11 bits, in place of the fp32 that the
plain form holds).  The kernels hold weights to 22 bits and everything else in
fp32, 2^-20 in relative terms: what they leave must be below a quarter of that
yardstick's share, with five standard deviations of its count as room.  Value
sums that are 2^-15 short, which is what the matrix unit's cut-off products add up
to over 2000 tokens, are put into the reference as well and have to exceed it.
"""
import math

import pytest
import torch

from long_context_emitting_b200 import api, paging
from test_q4_gpu import DEV, SCALE, TYPES, _gen, _i32, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    api.device_status()
    yield
    assert api.device_status() == 0, "a test left a device status behind"


def _store(g, T, Hkv, page):
    pages, table = paging.q4_store([T], Hkv, page, DEV, seed=T)
    strong = 1.0 + 3.0 * (torch.rand(1, Hkv, 1, 128, generator=g, device=DEV) < 0.06)
    for lo in range(0, T, 8192):
        n = min(8192, T - lo)
        k, v = _randn(g, 1, Hkv, n, 128) * strong, _randn(g, 1, Hkv, n, 128)
        api.kv_write_paged_q4(k.to(torch.bfloat16), v.to(torch.bfloat16), pages, table, page, _i32(lo))
    return pages, table


def _values(pages, table, T, h):
    """Codes, scales and minima of K and V of one key head's rows in 64 bits, from the row's definition."""
    rows = pages[table[0].long(), h].reshape(-1, 160)[:T]
    tail = rows[:, 128:].contiguous().view(torch.bfloat16).double().view(-1, 4, 4)
    c = torch.arange(128, device=DEV)
    place = (8 * (4 * ((c >> 3) & 3) + (c >> 5)) + (c & 7),
             8 * (2 * ((c >> 2) & 7) + (c >> 6)) + 4 * ((c >> 5) & 1) + (c & 3))
    out = []
    for i in range(2):
        b = rows[:, 64 * i:64 * i + 64]
        n = ((b[:, place[i] >> 1] >> (4 * (place[i] & 1)).to(torch.uint8)) & 15).double()
        out += [n, tail[:, 2 * i].repeat_interleave(32, 1), tail[:, 2 * i + 1].repeat_interleave(32, 1)]
    return out


def _half(w):
    """w to 11 bits, whatever its size."""
    f, e = torch.frexp(w)
    return torch.ldexp(torch.round(f * 2048) / 2048, e)


def _references(q, rows):
    """Outputs in 64 bits: right, with weights of 11 bits, with value sums 2^-15 short; and those sums."""
    nk, sk, mk, nv, sv, mv = rows
    p = torch.softmax(SCALE * q.double() @ (mk + sk * nk).T, -1)
    low = p @ mv
    right = p @ (sv * nv)
    rough = torch.empty_like(right)
    for g in range(4):
        c = slice(32 * g, 32 * g + 32)
        rough[:, c] = _half(p * sv[:, 32 * g]) @ nv[:, c]
    return right + low, rough + low, right * (1 - 2.0 ** -15) + low, right


def _wrong(x, right):
    return int((x != right).sum())


def _check(got, refs, dtype):
    exact, rough, short, sums = zip(*refs)
    right, rough, short = (torch.cat(r).to(dtype) for r in (exact, rough, short))
    got = torch.cat(got)
    yard = _wrong(rough, right)
    limit = yard / 4 + 5 * math.sqrt(yard / 4)
    assert yard > 60 and _wrong(short, right) > limit, (yard, _wrong(short, right))
    assert _wrong(got, right) <= limit, (_wrong(got, right), yard, right.numel())
    # and one by one: half a step, and before that what weights of 11 bits could be off by at worst
    off = torch.cat(sums) * 2.0 ** -11
    exact = torch.cat(exact)
    lim = off + torch.finfo(dtype).eps / 2 * (exact.abs() + off) + 2.0 ** -25
    assert bool(((got.double() - exact).abs() <= lim).all())


@TYPES
@pytest.mark.parametrize("T,Hkv,G,page", [(32768, 4, 4, 64), (131072, 2, 4, 128), (20011, 2, 8, 16), (32767, 8, 1, 48)])
def test_anchor_outputs_are_correctly_rounded(T, Hkv, G, page, dtype):
    g = _gen(T)
    pages, table = _store(g, T, Hkv, page)
    q = (1.5 * _randn(g, 1, Hkv * G, 128)).to(dtype)
    out, _, _ = api.decode_anchor_paged_q4(q, pages, table, page, _i32(T), T, SCALE, Hkv)
    assert api.device_status() == 0
    refs = [_references(q[0, h * G:h * G + G], _values(pages, table, T, h)) for h in range(Hkv)]
    _check([out[0, h * G:h * G + G] for h in range(Hkv)], refs, dtype)


@TYPES
@pytest.mark.parametrize("T,Hkv,G,page", [(32768, 4, 4, 64), (50001, 2, 8, 16)])
def test_reuse_outputs_are_correctly_rounded(T, Hkv, G, page, dtype):
    g = _gen(T + 1)
    pages, table = _store(g, T, Hkv, page)
    q = (1.5 * _randn(g, 1, Hkv * G, 128)).to(dtype)
    n = api.k_for_len(T)
    idx = torch.stack([torch.randperm(T, generator=g, device=DEV)[:n].sort().values for _ in range(Hkv)]).to(torch.int32)
    out, _ = api.decode_reuse_paged_q4(q, pages, table, page, _i32(T), idx[None].contiguous(), _i32(*([n] * Hkv)),
                                       _i32(*range(Hkv)), SCALE, Hkv)
    assert api.device_status() == 0
    refs = [_references(q[0, h * G:h * G + G], [x[idx[h].long()] for x in _values(pages, table, T, h)])
            for h in range(Hkv)]
    _check([out[0, h * G:h * G + G] for h in range(Hkv)], refs, dtype)

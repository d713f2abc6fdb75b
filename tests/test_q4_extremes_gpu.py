"""Values at the ends of bfloat16's range: groups whose scale is next to nothing are
quantised as exactly as others, and rows scaled by a power of two, up to what the
header allows, give outputs scaled by it, bit for bit."""
import numpy as np
import pytest
import torch

import oracle as O
from long_context_emitting_b200 import api, paging
from test_q4_gpu import DEV, SCALE, _filled, _gen, _i32, _np, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    api.device_status()
    yield
    assert api.device_status() == 0, "a test left a device status behind"


def _tiny_rows(rng):
    """Rows [n, 128] whose groups span 2^-133 (one step of bfloat16's subnormals) to 2^-112 in all."""
    rows = []
    for e in range(-133, -113):
        unit = 2.0 ** e
        for m in (0.0, -5.0, -15.0, 240.0, -2.0 ** 9):
            n = rng.integers(0, 16, (4, 32)).astype(np.float64)       # a grid of 15 steps
            n[:, 0], n[:, 1] = 0, 15
            half = n.copy()
            half[:, 2:] = np.floor(half[:, 2:]) + 0.5 if e > -133 else half[:, 2:]     # half-way codes
            half[:, 0], half[:, 1] = 0, 15
            wide = rng.integers(0, 241, (4, 32)).astype(np.float64) / (16 if e > -129 else 1)
            rows += [((x + m) * unit).reshape(128) for x in (n, half, np.minimum(wide, 15))]
            rows.append((np.where(rng.random((4, 32)) < 0.5, 0, 1) * unit).reshape(128))
            rows.append(np.full(128, m * unit))
    return np.stack(rows)


def test_cache_groups_of_tiny_scale():
    rng = np.random.default_rng(9)
    x = torch.from_numpy(_tiny_rows(rng)).to(torch.bfloat16).to(DEV).view(1, 1, -1, 128)
    n = x.shape[2]
    assert 0 < float(x.float().abs()[x != 0].min()) <= 2.0 ** -133
    for k, v in ((x, x.flip(2)), (-x, x.roll(7, 2))):
        want = O.q4_pack(_np(k), _np(v))[0, 0]
        scales = want[:, 128:].copy().view(np.uint16)[:, :4].astype(np.uint32) << 16
        s = scales.view(np.float32)
        assert ((0 < s) & (s < 2.0 ** -120)).sum() > 100 and (s >= 2.0 ** -120).sum() > 100 and s.min() == 0
        pages, table = paging.q4_store([n], 1, 16, DEV)
        api.kv_write_paged_q4(k.contiguous(), v.contiguous(), pages, table, 16, _i32(0))
        got = pages[table[0].long(), 0].reshape(-1, 160)[:n].cpu().numpy()
        bad = np.argwhere(got != want)
        assert not bad.size, (len(bad), bad[:4])
        # and back: minimum + scale * code, rounded once
        ko, vo = api.kv_read_paged_q4(pages, table, 16, _i32(0), None, n)
        for y, o in ((k, ko), (v, vo)):
            ref = torch.from_numpy(O.q4_values(*O.q4_quantise(_np(y)))).to(torch.bfloat16).to(DEV)
            assert torch.equal(o, ref)


def _scaled(pages, k_power, v_power):
    """The store with the scales and minima of K and V times powers of two (exact)."""
    out = pages.clone()
    tail = out[..., 128:].view(torch.bfloat16)
    tail[..., :8] = (tail[..., :8].double() * 2.0 ** k_power).to(torch.bfloat16)
    tail[..., 8:] = (tail[..., 8:].double() * 2.0 ** v_power).to(torch.bfloat16)
    return out


@pytest.mark.parametrize("T,G", [(4096, 4), (4096, 8), (131072, 1)])
@pytest.mark.parametrize("k_power,top", [(97, True), (-90, False)])
def test_decode_values_scaled_by_powers_of_two(T, G, k_power, top):
    """V up to 2^116 / T, or down to 2^-80; K times a power that the queries take back."""
    g = _gen(T + G)
    Hkv, page = 2, 128
    pages, table = _filled(g, (T,), Hkv, page)
    q = (1.5 * _randn(g, 1, Hkv * G, 128)).to(torch.bfloat16)
    v = api.kv_read_paged_q4(pages, table, page, _i32(0), None, T)[1]
    power = -80
    if top:
        power = int(np.floor(116 - np.log2(T) - np.log2(float(v.float().abs().max()))))
        assert power >= 96
    far, q_far = _scaled(pages, k_power, power), (q.double() * 2.0 ** -k_power).to(torch.bfloat16)
    assert torch.equal(q_far.double() * 2.0 ** k_power, q.double())
    idx = torch.arange(0, T, 9, device=DEV, dtype=torch.int32).repeat(1, Hkv, 1).contiguous()
    args = (_i32(T), idx, _i32(*([idx.shape[-1]] * Hkv)), _i32(*range(Hkv)), SCALE, Hkv)
    a = api.decode_anchor_paged_q4(q, pages, table, page, _i32(T), T, SCALE, Hkv)
    b = api.decode_anchor_paged_q4(q_far, far, table, page, _i32(T), T, SCALE, Hkv)
    c = api.decode_reuse_paged_q4(q, pages, table, page, *args)
    d = api.decode_reuse_paged_q4(q_far, far, table, page, *args)
    assert api.device_status() == 0
    for x, y in ((a, b), (c, d)):
        assert torch.equal(x[1], y[1])
        assert bool(y[0].isfinite().all()) and torch.equal(x[0].double() * 2.0 ** power, y[0].double())
    assert torch.equal(a[2], b[2])

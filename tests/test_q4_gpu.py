"""The operators around the 4-bit paged cache on the GPU, against the float64
oracle: head norms with rotation, quantising writes (byte for byte), reading
back (bit for bit), anchor and reuse attention, and a whole decode step.

Tolerances, derived from the roundings the kernels make:
  * a stored output is off by at most half a step, eps/2 of its type;
  * a logit (natural units) is an fp32 sum of 128 products and is off by at most
    delta = scale * 2^-19 * max_t sum_c |q_c| (15 s + |m|): 2^-24 per operation,
    with room for 32 of them;
  * a probability then moves by 2 delta (its own logit and the normaliser) and
    2^-20 (exponential and logarithm approximations, 2^-22 each, and sums);
  * in the attention outputs a weight p s may be rounded to half precision
    (2^-11) before it multiplies its code: at most 2^-11 sum_t p_t s_t n_t.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from long_context_emitting_b200 import api, paging, workload
from long_context_emitting_b200.schedule import PagedQ4DecodeSchedule, StepGraph
from test_q4_cpu import _rint_fraction

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda")
SCALE = api.default_scale()
BAD_INDEX, NONFINITE = 5, 6
TYPES = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


@pytest.fixture(autouse=True)
def _clean_status():
    api.device_status()
    yield
    assert api.device_status() == 0, "a test left a device status behind"


# ------------------------------------------------------- norms and rotation ----
def _check_rope(got, x, pos, inv, w, eps, inter, dtype):
    ref = O.norm_rope(_np(x), _np(pos), _np(inv), None if w is None else _np(w), eps, inter)
    # fp32: an angle's cosine is off by at most 2^-21, a norm by 2^-20, the products by a few 2^-24,
    # each relative to the row's largest rotated pair
    big = np.abs(O.norm_rope(np.abs(_np(x)), 0 * _np(pos), _np(inv), None if w is None else np.abs(_np(w)), eps, inter))
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + 2.0 ** -18 * (big + np.roll(big, 64, -1) + np.roll(big, 1, -1)
                                                                    + np.roll(big, -1, -1)) + 2.0 ** -25
    err = np.abs(_np(got) - ref)
    assert (err <= tol).all(), (err - tol).max()


@TYPES
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("B,N,Hq,Hkv,norm,far", [
    (1, 1, 1, 1, "both", 0), (3, 1, 32, 8, "both", 131071), (2, 3, 8, 8, "none", 5), (1, 4, 7, 3, "q", 0),
    (2, 77, 24, 6, "both", 2**30), (1, 515, 5, 1, "k", -1000), (1, 130, 64, 8, "none", 2**31 - 200)])
def test_norm_rope(B, N, Hq, Hkv, norm, far, inter, dtype):
    g = _gen(B * 1000 + N)
    qkv = (3 * _randn(g, B, N, Hq + 2 * Hkv, 128)).to(dtype)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
    pos = (torch.arange(N, device=DEV) + far).expand(B, N).to(torch.int32).contiguous()
    inv = 500000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float32) / 64)
    qw = (1 + 0.3 * _randn(g, 128)).to(dtype) if norm in ("both", "q") else None
    kw = (1 + 0.3 * _randn(g, 128)).to(dtype) if norm in ("both", "k") else None
    before = qkv.clone()
    qo, ko = api.qk_norm_rope(q, k, pos, inv, qw, kw, 1e-6, inter)
    assert torch.equal(qkv, before)
    _check_rope(qo, q, pos, inv, qw, 1e-6, inter, dtype)
    _check_rope(ko, k, pos, inv, kw, 1e-6, inter, dtype)
    # in place, through views of the packed rows: the same bits, V untouched
    api.qk_norm_rope(q, k, pos, inv, qw, kw, 1e-6, inter, q_out=q.transpose(1, 2), k_out=k.transpose(1, 2))
    assert torch.equal(q.transpose(1, 2), qo) and torch.equal(k.transpose(1, 2), ko)
    assert torch.equal(qkv[:, :, Hq + Hkv:], before[:, :, Hq + Hkv:])


def test_norm_rope_strides_and_edges():
    g = _gen(7)
    base = _randn(g, 5, 4, 2, 256).to(torch.bfloat16)      # heads of a wider row, tokens first
    q = base[:, :, :, 64:192].permute(1, 0, 2, 3)          # [4, 5, 2, 128], channels 64..191
    k = _randn(g, 1, 5, 1, 128).to(torch.bfloat16).expand(4, 5, 3, 128)   # broadcast input
    pos = torch.randint(0, 9999, (4, 5), generator=g, device=DEV, dtype=torch.int32)
    inv = torch.rand(64, generator=g, device=DEV)
    big = torch.full((4, 2, 7, 128), 9.0, device=DEV, dtype=torch.bfloat16)
    qo, ko = api.qk_norm_rope(q, k, pos, inv, q_out=big[:, :, 1:6])
    _check_rope(qo, q, pos, inv, None, 0, False, torch.bfloat16)
    _check_rope(ko, k, pos, inv, None, 0, False, torch.bfloat16)
    assert (big[:, :, 0] == 9).all() and (big[:, :, 6] == 9).all()
    # a row of zeros, a huge row, a row with a NaN: the others are not touched by it
    q = _randn(g, 1, 4, 1, 128).to(torch.bfloat16)
    q[0, 0] = 0
    q[0, 1] = 1e18
    q[0, 2, 0, 5] = float("nan")
    w = torch.ones(128, device=DEV, dtype=torch.bfloat16)
    p0 = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    qo, _ = api.qk_norm_rope(q, q, p0, inv, q_weight=w, k_weight=w)
    assert (qo[0, 0, 0] == 0).all() and (qo[0, 0, 1] == 1).all() and qo[0, 0, 2].isnan().all()
    _check_rope(qo[:, :, 3:], q[:, 3:], p0[:, 3:], inv, w, 1e-6, False, torch.bfloat16)
    # no tokens, no sequences
    for B, N in ((2, 0), (0, 3)):
        e = torch.empty(B, N, 2, 128, device=DEV, dtype=torch.bfloat16)
        qo, _ = api.qk_norm_rope(e, e, torch.empty(B, N, dtype=torch.int32, device=DEV), inv)
        assert qo.shape == (B, 2, N, 128)


# --------------------------------------------------------- write, read back ----
def _kinds(g, n, dtype):
    """Rows [n, 128] of the values a cache meets, by turns."""
    x = _randn(g, n, 128) * 2
    x[1::8] += 100                                              # an offset
    x[2::8] = torch.round(x[2::8] * 4) / 4                      # a grid: half-way codes
    x[3::8] = x[3::8, :1]                                       # constant rows
    x[4::8] = 0
    x[5::8, ::7] *= 50                                          # outlier channels
    x[6::8] = torch.randint(-15, 16, (x[6::8].shape[0], 128), generator=g, device=DEV) / 2
    x[7::8] *= 2.0 ** -12                                       # small; and tiny among large:
    x[7::16, ::3] = 1 - 2 * torch.randint(0, 2, x[7::16, ::3].shape, generator=g, device=DEV).float()
    x[7::16, 1::3] *= 2.0 ** -14
    return x.to(dtype)


@TYPES
@pytest.mark.parametrize("page,Hkv,N,start,count", [
    (16, 8, 1, (0, 15, 16, 4095), None), (64, 1, 3, (62, 0), (3, 0)), (48, 3, 4, (45, 1), (4, 3)),
    (128, 2, 130, (0, 127, 5), (130, 129, 0)), (16, 5, 37, (3,), None)])
def test_cache_write_and_read(page, Hkv, N, start, count, dtype):
    B = len(start)
    g = _gen(page + N)
    k = _kinds(g, B * Hkv * N, dtype).view(B, Hkv, N, 128)
    v = _kinds(g, B * N * Hkv, dtype).view(B, N, Hkv, 128).transpose(1, 2)   # token-major
    cnt = count or (N,) * B
    pages, table = paging.q4_store([s + c for s, c in zip(start, cnt)], Hkv, page, DEV, seed=N, spare_pages=2)
    pages.fill_(0xA5)
    want = pages.cpu().numpy()
    tab = table.cpu().numpy()
    rows = O.q4_pack(_np(k), _np(v))
    for b in range(B):
        for n in range(cnt[b]):
            t = start[b] + n
            want[tab[b, t // page], :, t % page] = rows[b, :, n]
    api.kv_write_paged_q4(k, v, pages, table, page, _i32(*start), None if count is None else _i32(*count))
    assert api.device_status() == 0
    got = pages.cpu().numpy()
    bad = np.argwhere(got != want)
    assert not bad.size, (len(bad), bad[:4])
    # read back: one rounding of minimum + scale * code (fp32 arithmetic is exact here but for one rounding)
    ko = torch.full((B, Hkv, N, 128), 7.0, dtype=dtype, device=DEV)
    vo = ko.clone()
    api.kv_read_paged_q4(pages, table, page, _i32(*start), None if count is None else _i32(*count), N, dtype, k=ko,
                         v=vo)
    for x, o in ((k, ko), (v, vo)):
        n, s, m = O.q4_quantise(_np(x))
        ref = O.q4_values(n, s, m)
        for b in range(B):
            e = np.abs(_np(o[b, :, :cnt[b]]) - ref[b, :, :cnt[b]])
            assert (e <= (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * np.abs(ref[b, :, :cnt[b]]) + 2.0 ** -25).all()
            assert (o[b, :, cnt[b]:] == 7).all()


def test_cache_codes_at_borders():
    """Values whose distance to the minimum is inexact in fp32 next to a half-way
    point: the code is that of exact arithmetic (checked with fractions)."""
    rows = []
    for e in (-30, -26, -60, -120):
        for m, hi in ((-1.5, 1.5), (-7.5, 7.5), (-3.75, 3.75), (-1.0, 14.0)):
            r = torch.zeros(128, dtype=torch.float64)
            r[::2], r[1::2] = m, hi
            # near each half-way point of the true step, from both sides, by a tiny amount
            tiny = 2.0 ** e
            r[2:32:4], r[34:64:4], r[66:96:4] = tiny, -tiny, 0.0
            rows.append(r)
    x = torch.stack(rows).to(torch.bfloat16).to(DEV).view(1, 1, -1, 128)
    pages, table = paging.q4_store([x.shape[2]], 1, 16, DEV)
    api.kv_write_paged_q4(x, x.flip(2), pages, table, 16, _i32(0))
    got = pages[table[0].long(), 0].reshape(-1, 160)[:x.shape[2]].cpu().numpy()
    (nk, sk, mk), (nv, sv, mv) = O.q4_unpack(got)
    for n, s, m, xs in ((nk, sk, mk, _np(x)[0, 0]), (nv, sv, mv, _np(x.flip(2))[0, 0])):
        for r in range(xs.shape[0]):
            for c in range(128):
                lo = min(xs[r, c // 32 * 32:c // 32 * 32 + 32])
                assert m[r, c // 32] == lo
                q = (Fraction(float(xs[r, c])) - Fraction(float(lo))) / Fraction(float(s[r, c // 32]))
                assert n[r, c] == _rint_fraction(q), (r, c)


@TYPES
def test_cache_nonfinite_and_bad_places(dtype):
    g = _gen(3)
    k, v = _randn(g, 2, 2, 20, 128).to(dtype), _randn(g, 2, 2, 20, 128).to(dtype)
    k[0, 1, 3, 40] = float("inf")
    v[1, 0, 5, 127] = float("nan")
    pages, table = paging.q4_store([20, 20], 2, 16, DEV)
    api.kv_write_paged_q4(k, v, pages, table, 16, _i32(0, 0))
    assert api.device_status() == NONFINITE
    ko, vo = api.kv_read_paged_q4(pages, table, 16, _i32(0, 0), None, 20, dtype)
    assert ko[0, 1, 3, 32:64].isnan().all() and vo[1, 0, 5, 96:].isnan().all()
    assert int(ko.isnan().sum()) == 32 and int(vo.isnan().sum()) == 32
    if dtype == torch.bfloat16:   # a finite range that overflows
        k[0, 1, 3, 40], v[1, 0, 5, 127] = 0, 0
        k[0, 0, 0, 0], k[0, 0, 0, 1] = 3.3e38, -3.3e38
        api.kv_write_paged_q4(k, v, pages, table, 16, _i32(0, 0))
        assert api.device_status() == NONFINITE
    # starts, counts and pages out of range: skipped, everything else as it was
    k, v = _randn(g, 4, 2, 20, 128).to(dtype), _randn(g, 4, 2, 20, 128).to(dtype)
    pages, table = paging.q4_store([20] * 4, 2, 16, DEV)
    for start, count in (((-1, 0, 0, 0), None), ((13, 0, 0, 0), None), ((0,) * 4, (21, 20, 20, 20)),
                         ((0,) * 4, (-1, 20, 20, 20)), ((2**31 - 5, 0, 0, 0), None)):
        pages.fill_(0x11)
        api.kv_write_paged_q4(k, v, pages, table, 16, _i32(*start), None if count is None else _i32(*count))
        assert api.device_status() == BAD_INDEX
        assert (pages[table[0].long()] == 0x11).all()
        ref = paging.q4_store([20] * 4, 2, 16, DEV)[0].fill_(0x11)
        api.kv_write_paged_q4(k[1:], v[1:], ref, table[1:], 16, _i32(0, 0, 0))
        assert torch.equal(pages, ref)
        ko = torch.full_like(k, 7.0)
        api.kv_read_paged_q4(pages, table, 16, _i32(*start), None if count is None else _i32(*count), 20, dtype, k=ko)
        assert api.device_status() == BAD_INDEX
        assert (ko[0] == 7).all() and not (ko[1:] == 7).all(-1).any()
    table[2, 1] = pages.shape[0]
    table[3, 0] = -1
    pages.fill_(0x11)
    api.kv_write_paged_q4(k, v, pages, table, 16, _i32(0, 0, 0, 0))
    assert api.device_status() == BAD_INDEX
    ko = torch.full_like(k, 7.0)
    api.kv_read_paged_q4(pages, table, 16, _i32(0, 0, 0, 0), None, 20, dtype, k=ko)
    assert api.device_status() == BAD_INDEX
    assert (ko[2, :, 16:] == 7).all() and (ko[3, :, :16] == 7).all()
    assert not (ko[2, :, :16] == 7).all(-1).any() and not (ko[3, :, 16:] == 7).all(-1).any()


# ---------------------------------------------------------------- attention ----
def _filled(g, lens, Hkv, page, seed=0, loud=False):
    """A store whose rows are quantised from random K/V; with ``loud`` some rows
    carry scales of very different size."""
    pages, table = paging.q4_store(lens, Hkv, page, DEV, seed=seed, spare_pages=3)
    k, v = _randn(g, *pages.shape[:3], 128), _randn(g, *pages.shape[:3], 128)
    k[..., ::17] *= 4
    if loud:
        v *= torch.pow(2.0, torch.randint(-20, 21, (*pages.shape[:3], 4, 1), generator=g, device=DEV).float()
                       ).expand(*pages.shape[:3], 4, 32).reshape(v.shape)
        v[..., 64:96] += 3
    for p in range(pages.shape[0]):     # through the identity table: page p is "sequence" p
        api.kv_write_paged_q4(k[p:p + 1].to(torch.bfloat16), v[p:p + 1].to(torch.bfloat16), pages,
                              _i32(p).view(1, 1), page, _i32(0))
    return pages, table


def _rows(pages, table, lens, page):
    """Per sequence: (codes, scales, minima) of K and of V, [Hkv, T, .]."""
    pg, tab = pages.cpu().numpy(), table.cpu().numpy()
    out = []
    for b, T in enumerate(lens):
        r = np.stack([pg[tab[b, t // page], :, t % page] for t in range(T)], 1) if T else \
            np.zeros((pages.shape[1], 0, 160), np.uint8)
        out.append(O.q4_unpack(r))
    return out


def _attend_ref(q, rows, scale):
    """One sequence and key head: q [G, 128], rows = ((n, s, m) of K, of V) -> reference and tolerances."""
    (nk, sk, mk), (nv, sv, mv) = rows
    K, V = O.q4_values(nk, sk, mk), O.q4_values(nv, sv, mv)
    x = scale * q @ K.T
    top = x.max(1, keepdims=True)
    e = np.exp(x - top)
    p = e / e.sum(1, keepdims=True)
    lse = (top + np.log(e.sum(1, keepdims=True)))[:, 0]
    reach = np.abs(q) @ np.repeat(15 * sk + np.abs(mk), 32, -1).T
    delta = abs(scale) * 2.0 ** -19 * reach.max(1)             # [G]
    out = p @ V
    steps = p @ O.q4_values(nv, sv, np.zeros_like(mv))
    drift = (2 * delta + 2.0 ** -20)[:, None]
    tol = drift * (p @ np.abs(V)) * 2 + 2.0 ** -11 * steps
    return out, lse, p, tol, delta, drift


def _check_out(got, out, tol, dtype, what):
    e = np.abs(_np(got) - out)
    lim = tol + torch.finfo(dtype).eps / 2 * (np.abs(out) + tol) + 2.0 ** -25
    assert (e <= lim).all(), (what, (e / lim).max(), e.max())


CASES = [  # lens, Hkv, G, page
    ((1, 15, 16, 17, 127, 129, 1000, 2051), 8, 4, 64),
    ((0, 1, 33, 0, 640), 2, 8, 16),
    ((2049, 31, 512), 3, 2, 48),
    ((5000,), 1, 1, 128),
    ((300,) * 5, 4, 4, 32),
]


@TYPES
@pytest.mark.parametrize("lens,Hkv,G,page", CASES, ids=[f"b{len(c[0])}h{c[1]}g{c[2]}p{c[3]}" for c in CASES])
def test_decode_q4_against_oracle(lens, Hkv, G, page, dtype):
    _decode_case(lens, Hkv, G, page, dtype, loud=False, qmul=1.5)


@TYPES
@pytest.mark.parametrize("qmul", [1.5, 60.0, 2.0 ** -12], ids=["q1", "q60", "qsmall"])
def test_decode_q4_loud_values(dtype, qmul):
    """Values whose groups differ by 2^40 in size, and sharp, ordinary and flat softmaxes."""
    _decode_case((700, 64, 5), 2, 4, 32, dtype, loud=True, qmul=qmul)


def _decode_case(lens, Hkv, G, page, dtype, loud, qmul):
    B, Hq, max_T = len(lens), Hkv * G, max(lens)
    g = _gen(sum(lens) + G)
    pages, table = _filled(g, lens, Hkv, page, seed=G, loud=loud)
    q = (qmul * _randn(g, B, Hq, 128)).to(dtype)
    ld = (max_T + 3) // 4 * 4 + 8
    pooled = torch.full((B, Hkv, ld), 5.0, device=DEV)
    out, lse, _ = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), max_T, SCALE, Hkv, pooled=pooled,
                                             ld_pooled=ld)
    assert api.device_status() == 0
    rows = _rows(pages, table, lens, page)
    wild = loud and dtype == torch.float16  # values beyond half precision's range saturate or vanish there
    for b, T in enumerate(lens):
        assert (pooled[b, :, T:] == 5).all()
        for h in range(Hkv):
            sl = slice(h * G, h * G + G)
            if T == 0:
                assert (out[b, sl] == 0).all() and (lse[b, sl] == -np.inf).all()
                continue
            part = [tuple(a[h] for a in r) for r in rows[b]]
            o, l, p, tol, delta, drift = _attend_ref(_np(q[b, sl]), part, SCALE)
            fits = np.abs(o) < (6e4 if wild else np.inf)
            _check_out(torch.where(torch.from_numpy(fits).to(DEV), out[b, sl], torch.zeros_like(out[b, sl])),
                       np.where(fits, o, 0), tol, dtype, f"anchor b={b} h={h}")
            assert (np.abs(_np(lse[b, sl]) - l) <= 2 * delta + 2.0 ** -22 * np.abs(l) + 2.0 ** -20).all()
            e = np.abs(_np(pooled[b, h, :T]) - p.mean(0))
            assert (e <= (drift * p).mean(0) + 1e-36).all(), (e / (p.mean(0) + 1e-36)).max()

    # reuse: a third of the tokens (at least one), another head's rows through the map, unused tail -1
    ks = [(T + 2) // 3 for T in lens]
    k_max = max(ks) + 3
    idx = np.full((B, Hkv, k_max), -1, dtype=np.int32)
    rng = np.random.default_rng(G)
    for b, T in enumerate(lens):
        for h in range(Hkv):
            idx[b, h, :ks[b]] = np.sort(rng.permutation(T)[:ks[b]])
    hm = rng.integers(0, Hkv, Hkv)
    ik = [k for k in ks for _ in range(Hkv)]
    out, lse = api.decode_reuse_paged_q4(q, pages, table, page, _i32(*lens), torch.from_numpy(idx).to(DEV), _i32(*ik),
                                         _i32(*hm.tolist()), SCALE, Hkv)
    assert api.device_status() == 0
    for b, T in enumerate(lens):
        for h in range(Hkv):
            sl = slice(h * G, h * G + G)
            if ks[b] == 0:
                assert (out[b, sl] == 0).all() and (lse[b, sl] == -np.inf).all()
                continue
            j = idx[b, hm[h], :ks[b]]
            part = [tuple(a[h][j] for a in r) for r in rows[b]]
            o, l, p, tol, delta, drift = _attend_ref(_np(q[b, sl]), part, SCALE)
            fits = np.abs(o) < (6e4 if wild else np.inf)
            _check_out(torch.where(torch.from_numpy(fits).to(DEV), out[b, sl], torch.zeros_like(out[b, sl])),
                       np.where(fits, o, 0), tol, dtype, f"reuse b={b} h={h}")
            assert (np.abs(_np(lse[b, sl]) - l) <= 2 * delta + 2.0 ** -22 * np.abs(l) + 2.0 ** -20).all()


def test_decode_q4_tail_rows_do_not_leak():
    """Slots behind a sequence's end hold NaN scales; they are never part of the result."""
    g = _gen(11)
    lens, Hkv, page = (37, 16, 1), 2, 16
    pages, table = _filled(g, lens, Hkv, page)
    q = _randn(g, 3, 8, 128).to(torch.bfloat16)
    want = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 37, SCALE, Hkv)
    mine = {int(p) for p in table[table >= 0]}
    for p in range(pages.shape[0]):
        if p not in mine:
            pages[p] = 0xFF
    for b, T in enumerate(lens):
        if T % page:
            pages[int(table[b, T // page]), :, T % page:] = 0xFF
    got = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 37, SCALE, Hkv)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    for b, T in enumerate(lens):
        assert torch.equal(want[2][b, :, :T], got[2][b, :, :T])


def test_decode_q4_nan_row_stays_in_its_head():
    g = _gen(12)
    lens, Hkv, page = (90, 90), 2, 32
    pages, table = _filled(g, lens, Hkv, page)
    q = _randn(g, 2, 8, 128).to(torch.bfloat16)
    want = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 90, SCALE, Hkv)
    pages[int(table[0, 1]), 1, 3, 128:].view(torch.bfloat16)[12] = float("nan")   # V minimum of group 0, token 35
    out, lse, pooled = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 90, SCALE, Hkv)
    assert out[0, 4:, :32].isnan().all() and not out[0, 4:, 32:].isnan().any()
    assert torch.equal(out[0, :4], want[0][0, :4]) and torch.equal(out[1], want[0][1])
    assert torch.equal(lse, want[1]) and torch.equal(pooled[..., :90], want[2][..., :90])
    pages[int(table[0, 1]), 1, 3, 128:].view(torch.bfloat16)[4] = float("nan")    # K minimum: the whole row's logit
    out, lse, _ = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 90, SCALE, Hkv)
    assert out[0, 4:].isnan().all() and lse[0, 4:].isnan().all()
    assert torch.equal(out[0, :4], want[0][0, :4]) and torch.equal(out[1], want[0][1])


def test_decode_q4_bad_pages_lengths_and_indices():
    g = _gen(13)
    lens, Hkv, page = (100, 64, 70), 2, 32
    pages, table = _filled(g, lens, Hkv, page)
    q = _randn(g, 3, 8, 128).to(torch.bfloat16)
    sl = _i32(*lens)
    want = api.decode_anchor_paged_q4(q, pages, table, page, sl, 100, SCALE, Hkv)
    bad = table.clone()
    bad[0, 1] = pages.shape[0]       # tokens 32..63 of sequence 0 are lost
    bad[1, 0] = -7
    ld = 104
    pooled = torch.full((3, Hkv, ld), 5.0, device=DEV)
    out, lse, _ = api.decode_anchor_paged_q4(q, pages, bad, page, sl, 100, SCALE, Hkv, pooled=pooled, ld_pooled=ld)
    assert api.device_status() == BAD_INDEX
    assert (pooled[0, :, 32:64] == 0).all() and (pooled[1, :, :32] == 0).all()
    assert torch.equal(out[2], want[0][2])
    rows = _rows(pages, table, lens, page)
    keep = np.r_[0:32, 64:100]
    for h in range(Hkv):
        o, l, p, tol, delta, _ = _attend_ref(_np(q[0, 4 * h:4 * h + 4]), [tuple(a[h][keep] for a in r) for r in rows[0]],
                                             SCALE)
        _check_out(out[0, 4 * h:4 * h + 4], o, tol, torch.bfloat16, "lost page")
    # lengths out of range: an empty sequence, flagged
    for T in (-1, 101):
        out, lse, _ = api.decode_anchor_paged_q4(q, pages, table, page, _i32(100, T, 70), 100, SCALE, Hkv)
        assert api.device_status() == BAD_INDEX
        assert (out[1] == 0).all() and (lse[1] == -np.inf).all() and torch.equal(out[0], want[0][0])
    # indices
    idx = torch.arange(20, device=DEV, dtype=torch.int32).repeat(3, Hkv, 1)
    ik, hm = _i32(*([20] * 6)), _i32(0, 1)
    ref, ref_l = api.decode_reuse_paged_q4(q, pages, table, page, sl, idx, ik, hm, SCALE, Hkv)
    worse = torch.cat([idx, torch.full_like(idx[..., :3], -1)], -1)
    worse[..., 20], worse[..., 22] = 2**31 - 1, 100
    out, lse = api.decode_reuse_paged_q4(q, pages, table, page, sl, worse, _i32(*([23] * 6)), hm, SCALE, Hkv)
    assert api.device_status() == BAD_INDEX
    # the same rows, perhaps split differently over warps: the tolerance of one set
    for b in range(3):
        for h in range(Hkv):
            o, l, p, tol, delta, _ = _attend_ref(_np(q[b, 4 * h:4 * h + 4]),
                                                 [tuple(a[h][:20] for a in r) for r in rows[b]], SCALE)
            _check_out(out[b, 4 * h:4 * h + 4], o, tol, torch.bfloat16, "bad indices")
            _check_out(ref[b, 4 * h:4 * h + 4], o, tol, torch.bfloat16, "good indices")
    for kw in (dict(ik=_i32(20, 20, 24, 20, 20, 20)), dict(ik=_i32(20, 20, -1, 20, 20, 20)), dict(sl=_i32(100, 200, 70)),
               dict(sl=_i32(100, -3, 70))):
        a = dict(ik=ik, sl=sl) | kw
        out, lse = api.decode_reuse_paged_q4(q, pages, table, page, a["sl"], idx, a["ik"], hm, SCALE, Hkv)
        assert api.device_status() == BAD_INDEX
        assert (out[1, :4] == 0).all() and (lse[1, :4] == -np.inf).all()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])
    out, lse = api.decode_reuse_paged_q4(q, pages, table, page, sl, idx, ik, _i32(0, 2), SCALE, Hkv)
    assert api.device_status() == BAD_INDEX
    assert (out[:, 4:] == 0).all() and torch.equal(out[:, :4], ref[:, :4])
    out, lse = api.decode_reuse_paged_q4(q, pages, table, page, sl, idx[..., :0], _i32(*([0] * 6)), hm, SCALE, Hkv)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_decode_q4_repeated_index_counts_twice():
    g = _gen(14)
    pages, table = _filled(g, (50,), 1, 16)
    q = _randn(g, 1, 4, 128).to(torch.bfloat16)
    idx = torch.tensor([[[3, 3, 9, 49, 49, 49]]], dtype=torch.int32, device=DEV)
    out, lse = api.decode_reuse_paged_q4(q, pages, table, 16, _i32(50), idx, _i32(6), _i32(0), SCALE, 1)
    j = idx[0, 0].cpu().numpy()
    part = [tuple(a[0][j] for a in r) for r in _rows(pages, table, (50,), 16)[0]]
    o, l, _, tol, delta, _ = _attend_ref(_np(q[0]), part, SCALE)
    _check_out(out[0], o, tol, torch.bfloat16, "repeated")
    assert (np.abs(_np(lse[0]) - l) <= 2 * delta + 2.0 ** -20).all()


def test_decode_q4_matches_read_back():
    """The cache read back in 16 bits and attended by the 16-bit call: the same
    within the roundings of the read (half a step per value)."""
    g = _gen(15)
    T, Hkv = 1500, 8
    pages, table = _filled(g, (T,), Hkv, 64)
    q = _randn(g, 1, 32, 128).to(torch.bfloat16)
    k, v = api.kv_read_paged_q4(pages, table, 64, _i32(0), None, T)
    out, lse, pooled = api.decode_anchor_paged_q4(q, pages, table, 64, _i32(T), T, SCALE, Hkv)
    ref, ref_l, ref_p = api.decode_anchor(q, k.view(-1), v.view(-1), torch.zeros(1, dtype=torch.int64, device=DEV),
                                          _i32(T), T, SCALE, Hkv)
    # half a bf16 step per key value, |logit error| <= scale 2^-9 sum |q||k|
    d = float(SCALE * 2.0 ** -9 * (q.float().abs().view(8, 4, 128) @ k[0].float().abs().transpose(1, 2)).max())
    assert float((lse - ref_l).abs().max()) <= d + 1e-4
    big = float(v.float().abs().max())
    assert float((out.float() - ref.float()).abs().max()) <= (2 * d + 2.0 ** -7) * big
    assert float((pooled / ref_p - 1).abs().max()) <= 3 * d


# ------------------------------------------------------------ a decode step ----
def _step_case(dtype, norm, seed=21):
    lens, Hq, Hkv, L, page = (513, 1, 0, 130), 8, 2, 3, 32
    g = _gen(seed)
    inv = 500000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float32) / 64)
    sch = PagedQ4DecodeSchedule(4, Hq, Hkv, lens, (0,), L, DEV, inv, dtype=dtype)
    layers, maps = [], {}
    for l in range(L):
        qkv = _randn(g, 4, 1, Hq + 2 * Hkv, 128).to(dtype)
        pages, table = _filled(g, lens, Hkv, page, seed=l)
        layers.append({"q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hkv], "v": qkv[:, :, Hq + Hkv:], "kv_pages": pages,
                       "block_table": table})
        if norm:
            layers[-1]["q_weight"] = (1 + 0.2 * _randn(g, 128)).to(dtype)
            layers[-1]["k_weight"] = (1 + 0.2 * _randn(g, 128)).to(dtype)
        maps[l] = torch.randint(0, Hkv, (Hkv,), generator=g, device=DEV, dtype=torch.int32)
    return sch, layers, maps, lens, page


@TYPES
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "plain"])
def test_q4_decode_step(dtype, norm):
    """Three layers (anchor, reuse, reuse) from projections to outputs, each
    operator checked on what the one before it produced."""
    sch, layers, maps, lens, page = _step_case(dtype, norm)
    outs = [torch.empty(4, sch.Hq, 128, dtype=dtype, device=DEV) for _ in layers]
    sch.step(layers, maps, outs)
    assert api.device_status() == 0
    G = sch.Hq // sch.Hkv
    for l, lay in enumerate(layers):
        w = lay.get("q_weight"), lay.get("k_weight")
        pos = sch.positions.view(4, 1)
        qr, kr = api.qk_norm_rope(lay["q"], lay["k"], pos, sch.inv_freq, w[0], w[1])
        _check_rope(qr, lay["q"], pos, sch.inv_freq, w[0], 1e-6, False, dtype)
        rows = _rows(lay["kv_pages"], lay["block_table"], lens, page)
        new = O.q4_pack(_np(kr[:, :, 0]), _np(lay["v"][:, 0]))
        for b, T in enumerate(lens):
            if T == 0:
                assert (outs[l][b] == 0).all()
                continue
            t = T - 1
            got = lay["kv_pages"][int(lay["block_table"][b, t // page]), :, t % page].cpu().numpy()
            assert np.array_equal(got, new[b])
            for h in range(sch.Hkv):
                part = [tuple(a[h] for a in r) for r in rows[b]]
                if l:   # reuse: the anchor's indices through the head map
                    j = sch.idx[b, int(maps[l][h]), :O.k_for_len(T)].cpu().numpy()
                    part = [tuple(a[j] for a in r) for r in part]
                o, _, _, tol, _, _ = _attend_ref(_np(qr[b, h * G:h * G + G, 0]), part, SCALE)
                _check_out(outs[l][b, h * G:h * G + G], o, tol, dtype, f"step l={l} b={b} h={h}")


def test_q4_decode_step_graph_and_stream():
    """The step captured as one graph and replayed, and run on a side stream: the
    same bits as run op by op."""
    sch, layers, maps, lens, page = _step_case(torch.bfloat16, True, seed=22)
    mk = lambda: [torch.empty(4, sch.Hq, 128, dtype=torch.bfloat16, device=DEV) for _ in layers]  # noqa: E731
    eager, graphed, side = mk(), mk(), mk()
    sch.step(layers, maps, eager)
    torch.cuda.synchronize()
    gr = StepGraph(lambda: sch.step(layers, maps, graphed))
    for o in graphed:
        o.zero_()
    gr.replay()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        sch.step(layers, maps, side)
    st.synchronize()
    assert api.device_status() == 0
    for a, b, c in zip(eager, graphed, side):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_decode_q4_two_streams_at_once():
    """Two calls in flight at the same time, each with its own workspace: the
    same bits as one after the other."""
    g = _gen(31)
    work = []
    for i, lens in enumerate(((3001, 77), (512, 4097))):
        pages, table = _filled(g, lens, 2, 64, seed=i)
        work.append((_randn(g, 2, 8, 128).to(torch.bfloat16), pages, table, 64, _i32(*lens), max(lens), SCALE, 2))
    want = [api.decode_anchor_paged_q4(*w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        got = []
        for w, s in zip(work, streams):
            with torch.cuda.stream(s):
                got.append(api.decode_anchor_paged_q4(*w))
        torch.cuda.synchronize()
        for a, b, w in zip(want, got, work):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
            for i, T in enumerate(w[4].tolist()):
                assert torch.equal(a[2][i, :, :T], b[2][i, :, :T])


def test_decode_q4_long_cache_offsets():
    """A store of more than 2^31 bytes and 2^32 code nibbles: the last pages are
    where they should be."""
    Hkv, page = 8, 64
    num = (1 << 32) // (Hkv * page * 160) + 40
    pages = torch.zeros(num, Hkv, page, 160, dtype=torch.uint8, device=DEV)
    T = 1000
    n = (T + page - 1) // page
    table = torch.arange(num - n, num, device=DEV, dtype=torch.int32).flip(0).view(1, n).contiguous()
    g = _gen(41)
    k, v = _randn(g, 1, Hkv, T, 128).to(torch.bfloat16), _randn(g, 1, Hkv, T, 128).to(torch.bfloat16)
    api.kv_write_paged_q4(k, v, pages, table, page, _i32(0))
    small = pages[num - n:].clone()
    t2 = table - (num - n)
    assert int(pages[:1000].max()) == 0
    q = _randn(g, 1, 32, 128).to(torch.bfloat16)
    a = api.decode_anchor_paged_q4(q, pages, table, page, _i32(T), T, SCALE, Hkv)
    b = api.decode_anchor_paged_q4(q, small, t2, page, _i32(T), T, SCALE, Hkv)
    idx = torch.arange(0, T, 7, device=DEV, dtype=torch.int32).repeat(1, Hkv, 1).contiguous()
    args = (_i32(T), idx, _i32(*([idx.shape[-1]] * Hkv)), _i32(*range(Hkv)), SCALE, Hkv)
    c = api.decode_reuse_paged_q4(q, pages, table, page, *args)
    d = api.decode_reuse_paged_q4(q, small, t2, page, *args)
    ka, va = api.kv_read_paged_q4(pages, table, page, _i32(0), None, T)
    kb, vb = api.kv_read_paged_q4(small, t2, page, _i32(0), None, T)
    assert api.device_status() == 0
    for x, y in ((a[0], b[0]), (a[1], b[1]), (a[2], b[2]), (c[0], d[0]), (c[1], d[1]), (ka, kb), (va, vb)):
        assert torch.equal(x, y)
    assert float((ka.float() - k.float()).abs().max()) < 0.5 and int(small.max()) > 0

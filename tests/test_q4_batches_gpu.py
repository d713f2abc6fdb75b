"""The 4-bit decode calls on batches that the device plans by itself: many short
sequences, a capacity far above the lengths, lengths that change under a captured
graph, and workspaces that hold old bytes.  The reference is the float64 oracle
through the same checks as the other tests of these calls, or the same call on
other ground, bit for bit."""
import numpy as np
import pytest
import torch

from long_context_emitting_b200 import api
from long_context_emitting_b200.schedule import StepGraph
from test_q4_gpu import BAD_INDEX, DEV, SCALE, _attend_ref, _check_out, _filled, _gen, _i32, _np, _randn, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    api.device_status()
    yield
    assert api.device_status() == 0, "a test left a device status behind"


def _check(q, pages, table, page, lens, Hkv, out, lse, pooled, only=None):
    G = q.shape[1] // Hkv
    rows = _rows(pages, table, lens, page)
    for b, T in enumerate(lens):
        if only is not None and b not in only:
            continue
        for h in range(Hkv):
            sl = slice(h * G, h * G + G)
            if T == 0:
                assert (out[b, sl] == 0).all() and (lse[b, sl] == -np.inf).all()
                continue
            o, l, p, tol, delta, drift = _attend_ref(_np(q[b, sl]), [tuple(a[h] for a in r) for r in rows[b]], SCALE)
            _check_out(out[b, sl], o, tol, q.dtype, f"b={b} h={h}")
            assert (np.abs(_np(lse[b, sl]) - l) <= 2 * delta + 2.0 ** -22 * np.abs(l) + 2.0 ** -20).all()
            e = np.abs(_np(pooled[b, h, :T]) - p.mean(0))
            assert (e <= (drift * p).mean(0) + 1e-36).all()


@pytest.mark.parametrize("Hkv,G,lo,hi,extra", [(2, 4, 0, 40, 0), (1, 8, 0, 3, 5000), (3, 2, 1, 90, 700), (8, 1, 0, 2, 64)])
def test_many_short_sequences(Hkv, G, lo, hi, extra):
    """More units than blocks, several units per block, empty ones between, and one long sequence."""
    rng = np.random.default_rng(hi)
    lens = [int(x) for x in rng.integers(lo, hi, 261)]
    lens[130] = hi + extra
    g = _gen(hi)
    pages, table = _filled(g, lens, Hkv, 16, seed=hi)
    q = (1.5 * _randn(g, len(lens), Hkv * G, 128)).to(torch.bfloat16)
    max_T = max(lens)
    ld = (max_T + 3) // 4 * 4
    pooled = torch.full((len(lens), Hkv, ld), 5.0, device=DEV)
    out, lse, _ = api.decode_anchor_paged_q4(q, pages, table, 16, _i32(*lens), max_T, SCALE, Hkv, pooled=pooled,
                                             ld_pooled=ld)
    assert api.device_status() == 0
    for b, T in enumerate(lens):
        assert (pooled[b, :, T:] == 5).all()
    _check(q, pages, table, 16, lens, Hkv, out, lse, pooled)


def test_capacity_far_above_the_lengths():
    """max_T is what the block table allows, the sequences are short: the same checks."""
    g = _gen(3)
    lens, Hkv, page = (33, 0, 700, 1), 4, 32
    pages, table = _filled(g, lens, Hkv, page)
    cap = 200000
    wide = torch.full((4, cap // page), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    q = _randn(g, 4, 16, 128).to(torch.float16)
    out, lse, pooled = api.decode_anchor_paged_q4(q, pages, wide, page, _i32(*lens), cap, SCALE, Hkv)
    assert api.device_status() == 0
    _check(q, pages, table, page, lens, Hkv, out, lse, pooled)
    for bad in ((33, -1, cap + 1, 1), (0, 0, 0, 0), (-5, -5, -5, -5)):
        out, lse, _ = api.decode_anchor_paged_q4(q, pages, wide, page, _i32(*bad), cap, SCALE, Hkv)
        assert api.device_status() == (BAD_INDEX if min(bad) < 0 else 0)
        for b, T in enumerate(bad):
            if not 0 < T <= cap:
                assert (out[b] == 0).all() and (lse[b] == -np.inf).all()


def test_lengths_that_change_under_a_graph():
    """The captured call plans on the device: replays with other lengths give what eager calls give."""
    g = _gen(4)
    full, Hkv, page = (900, 2100, 64, 513), 2, 64
    pages, table = _filled(g, full, Hkv, page)
    q = _randn(g, 4, 8, 128).to(torch.bfloat16)
    sl = _i32(*full)
    mk = lambda: (torch.zeros(4, 8, 128, dtype=torch.bfloat16, device=DEV), torch.zeros(4, 8, device=DEV),  # noqa: E731
                  torch.zeros(4, Hkv, 2100, device=DEV))
    o, l, p = mk()
    ws = api.workspace(api.decode_anchor_paged_q4_workspace_bytes(4, 8, Hkv, 2100), DEV)
    gr = StepGraph(lambda: api.decode_anchor_paged_q4(q, pages, table, page, sl, 2100, SCALE, Hkv, out=o, lse=l, pooled=p,
                                                      ld_pooled=2100, ws=ws))
    for lens in (full, (1, 2100, 0, 512), (900, 1, 1, 1), (0, 0, 0, 0), full):
        sl.copy_(_i32(*lens))
        p.zero_()
        gr.replay()
        torch.cuda.synchronize()
        eo, el, ep = mk()
        api.decode_anchor_paged_q4(q, pages, table, page, sl, 2100, SCALE, Hkv, out=eo, lse=el, pooled=ep, ld_pooled=2100)
        assert torch.equal(o, eo) and torch.equal(l, el) and torch.equal(p, ep)
        _check(q, pages, table, page, lens, Hkv, o, l, p)


@pytest.mark.parametrize("byte", [0x00, 0xFF, 0x7F])
def test_workspace_bytes_do_not_matter(byte):
    g = _gen(5)
    lens, Hkv, page = (300, 0, 77, 1500), 2, 16
    pages, table = _filled(g, lens, Hkv, page)
    q = _randn(g, 4, 16, 128).to(torch.bfloat16)
    want = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 1500, SCALE, Hkv)
    ws = api.workspace(api.decode_anchor_paged_q4_workspace_bytes(4, 16, Hkv, 1500), DEV).fill_(byte)
    got = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 1500, SCALE, Hkv, ws=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    for b, T in enumerate(lens):
        assert torch.equal(want[2][b, :, :T], got[2][b, :, :T])


def test_partial_stages_after_rows_of_nan():
    """A block whose earlier rows were NaN works on a partly filled stage of another sequence next: what
    is left in its shared memory does not reach the valid rows."""
    g = _gen(6)
    lens, Hkv, page, G = [20, 3] * 200, 1, 16, 4
    pages, table = _filled(g, lens, Hkv, page)
    q = _randn(g, len(lens), G, 128).to(torch.bfloat16)
    want = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 20, SCALE, Hkv)
    for b in range(0, len(lens), 2):    # every second sequence all NaN
        for pg in table[b][table[b] >= 0].tolist():
            pages[pg] = 0xFF
    got = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 20, SCALE, Hkv)
    assert got[0][0::2].isnan().all()
    assert torch.equal(want[0][1::2], got[0][1::2]) and torch.equal(want[1][1::2], got[1][1::2])
    for b in range(1, len(lens), 2):
        assert torch.equal(want[2][b, :, :3], got[2][b, :, :3])


@pytest.mark.parametrize("T,k", [(4000, 1), (4000, 31), (4000, 33), (4000, 129), (9000, 2049), (9000, 9000)])
def test_reuse_lengths(T, k):
    """Selections from one token to all, on one unit (clusters of 16) and many."""
    for B, Hkv in ((1, 1), (5, 8)):
        g = _gen(T + k + B)
        lens = [T] + [max(1, T // (3 * i)) for i in range(1, B)]
        pages, table = _filled(g, lens, Hkv, 64)
        q = _randn(g, B, Hkv * 4, 128).to(torch.bfloat16)
        ks = [min(k, t) for t in lens]
        idx = torch.full((B, Hkv, max(ks) + 5), -1, dtype=torch.int32, device=DEV)
        for b in range(B):
            for h in range(Hkv):
                idx[b, h, :ks[b]] = torch.randperm(lens[b], generator=g, device=DEV)[:ks[b]].to(torch.int32)  # any order
        ik = _i32(*[x for x in ks for _ in range(Hkv)])
        hm = _i32(*reversed(range(Hkv)))
        out, lse = api.decode_reuse_paged_q4(q, pages, table, 64, _i32(*lens), idx, ik, hm, SCALE, Hkv)
        assert api.device_status() == 0
        rows = _rows(pages, table, lens, 64)
        for b in range(B):
            for h in range(0, Hkv, 3):
                j = idx[b, Hkv - 1 - h, :ks[b]].cpu().numpy()
                o, l, _, tol, delta, _ = _attend_ref(_np(q[b, 4 * h:4 * h + 4]),
                                                     [tuple(a[h][j] for a in r) for r in rows[b]], SCALE)
                _check_out(out[b, 4 * h:4 * h + 4], o, tol, q.dtype, f"b={b} h={h}")
                assert (np.abs(_np(lse[b, 4 * h:4 * h + 4]) - l) <= 2 * delta + 2.0 ** -22 * np.abs(l) + 2.0 ** -20).all()

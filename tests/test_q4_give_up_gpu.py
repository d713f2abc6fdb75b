"""What the 4-bit anchor leaves when a block's bounded wait gives up: NaN for every
unit that the block had a part of, and never anything of an earlier call that the
workspace still holds.  The block gives up by order of a diagnostic entry point, so
nothing waits and nothing faults."""
import pytest
import torch

from long_context_emitting_b200 import api, binding
from long_context_emitting_b200.binding import Shape
from test_q4_gpu import DEV, SCALE, _filled, _gen, _i32, _randn

pytestmark = pytest.mark.gpu
TIMEOUT = binding.KASCADE_ERR_TIMEOUT


def _call(block, q, pages, table, page, lens, max_T, Hkv, ws):
    B, Hq, _ = q.shape
    ld = (max_T + 3) // 4 * 4
    out = torch.full((B, Hq, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, Hq), 3.0, device=DEV)
    pooled = torch.full((B, Hkv, ld), 3.0, device=DEV)
    rc = binding.load().kascade_selftest_anchor_q4_gives_up(
        block, Shape(B, Hq, Hkv, 128), q.data_ptr(), pages.data_ptr(), pages.shape[0], table.data_ptr(), table.shape[1],
        page, lens.data_ptr(), max_T, SCALE, out.data_ptr(), lse.data_ptr(), pooled.data_ptr(), ld, ws.data_ptr(),
        ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    return out, lse, pooled


@pytest.mark.parametrize("lens,Hkv,G", [((3000, 0, 900, 5000), 2, 4), ((17,) * 300, 2, 8), ((70000,), 1, 1)])
def test_units_of_a_block_that_gives_up_are_nan(lens, Hkv, G):
    g = _gen(51)
    B, page, max_T = len(lens), 64, max(lens)
    pages, table = _filled(g, lens, Hkv, page)
    q, other = (_randn(g, B, Hkv * G, 128).to(torch.bfloat16) for _ in range(2))
    ws = api.workspace(api.decode_anchor_paged_q4_workspace_bytes(B, Hkv * G, Hkv, max_T), DEV)
    sl = _i32(*lens)
    want = _call(10**9, q, pages, table, page, sl, max_T, Hkv, ws)    # no such block
    assert api.device_status() == 0
    assert not any(w.isnan().any() for w in want)
    hit = torch.zeros(B, Hkv, dtype=torch.bool, device=DEV)
    for block in list(range(0, 444, 37)) + [1, 2, 3, 443]:
        # an earlier call of other queries leaves complete parts in the workspace
        _call(10**9, other, pages, table, page, sl, max_T, Hkv, ws)
        assert api.device_status() == 0
        out, lse, pooled = _call(block, q, pages, table, page, sl, max_T, Hkv, ws)
        lost = lse.view(B, Hkv, G).isnan()
        assert api.device_status() == (TIMEOUT if lost.any() else 0)
        assert (lost.all(-1) == lost.any(-1)).all()
        lost = lost.all(-1)
        hit |= lost
        for b, T in enumerate(lens):
            for h in range(Hkv):
                sl_ = slice(h * G, h * G + G)
                if lost[b, h]:
                    assert T and out[b, sl_].isnan().all() and pooled[b, h, :T].isnan().all()
                else:
                    assert torch.equal(out[b, sl_], want[0][b, sl_]) and torch.equal(lse[b, sl_], want[1][b, sl_])
                    assert torch.equal(pooled[b, h, :T], want[2][b, h, :T])
                assert (pooled[b, h, T:] == 3).all()
    assert hit.any()


def test_the_next_call_is_whole_again():
    g = _gen(52)
    lens, Hkv, page = (700, 33), 2, 16
    pages, table = _filled(g, lens, Hkv, page)
    q = _randn(g, 2, 8, 128).to(torch.bfloat16)
    ws = api.workspace(api.decode_anchor_paged_q4_workspace_bytes(2, 8, Hkv, 700), DEV)
    want = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 700, SCALE, Hkv)
    lost = 0
    for block in range(40):    # the first ones hold no stage: their share is the start of the first unit
        hit = bool(_call(block, q, pages, table, page, _i32(*lens), 700, Hkv, ws)[1].isnan().any())
        assert api.device_status() == (TIMEOUT if hit else 0)
        lost += hit
        got = api.decode_anchor_paged_q4(q, pages, table, page, _i32(*lens), 700, SCALE, Hkv, ws=ws)
        assert api.device_status() == 0
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert lost > 4

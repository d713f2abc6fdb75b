"""Long runs of the overlapped kernels without a wait between them, over the same
buffers with new values each time: every result is that of the same calls run one
by one, bit for bit."""
import pytest
import torch

from long_context_emitting_b200 import api, paging
from long_context_emitting_b200.schedule import StepGraph
from test_q4_gpu import DEV, SCALE, _gen, _i32, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    api.device_status()
    yield
    assert api.device_status() == 0, "a test left a device status behind"


def _chain(rounds, dtype, B, N, Hq, Hkv, page, seed):
    """The calls of one round (norm -> write -> read -> write -> read, and with one token per sequence
    attention over the pages and over 16-bit rows), and the tensors that they leave."""
    g = _gen(seed)
    qkv = [_randn(g, B, N, Hq + 2 * Hkv, 128).to(dtype) for _ in range(rounds)]
    start = [200 + 64 * b for b in range(B)]
    lens = [s + N for s in start]
    max_T, k_max = max(lens), min(lens)
    pages, table = paging.q4_store(lens, Hkv, page, DEV, seed=seed)
    old = _randn(g, 2, B, Hkv, max(start), 128).to(dtype)
    api.kv_write_paged_q4(old[0], old[1], pages, table, page, _i32(*([0] * B)), _i32(*start))
    q, k = torch.empty(B, Hq, N, 128, dtype=dtype, device=DEV), torch.empty(B, Hkv, N, 128, dtype=dtype, device=DEV)
    inv = 500000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float32) / 64)
    pos = torch.arange(N, device=DEV, dtype=torch.int32).repeat(B, 1)
    first, sl = _i32(*start), _i32(*lens)
    wide = _randn(g, 2, B * Hkv * max_T * 128).to(dtype)     # 16-bit caches
    off = torch.arange(B, device=DEV, dtype=torch.int64) * (Hkv * max_T * 128)
    idx = torch.arange(k_max, device=DEV, dtype=torch.int32).repeat(B, Hkv, 1).contiguous()
    ik, hm = _i32(*([k_max] * B * Hkv)), _i32(*range(Hkv))
    ld = (max_T + 3) // 4 * 4
    ws = api.workspace(max(api.decode_anchor_paged_q4_workspace_bytes(B, Hq, Hkv, max_T),
                           api.decode_reuse_workspace_bytes(B, Hq, Hkv, k_max)), DEV)
    torch.cuda.synchronize()

    def calls(r, out):
        x = qkv[r]
        v = x[:, :, Hq + Hkv:].transpose(1, 2)
        norm = lambda: api.qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], pos, inv, q_out=q, k_out=k)  # noqa: E731
        yield norm
        yield lambda: api.kv_write_paged_q4(k, v, pages, table, page, first)
        yield lambda: api.kv_read_paged_q4(pages, table, page, first, None, N, dtype, k=out["k0"], v=out["v0"])
        yield lambda: api.kv_write_paged_q4(v, k, pages, table, page, first)
        yield lambda: api.kv_read_paged_q4(pages, table, page, first, None, N, dtype, k=out["k1"], v=out["v1"])
        if N > 1:
            return
        one = q.view(B, Hq, 128)
        yield lambda: api.decode_reuse(one, wide[0], wide[1], off, sl, idx, ik, hm, SCALE, Hkv, out=out["w"],
                                       lse=out["wl"], ws=ws)
        yield lambda: api.decode_anchor_paged_q4(one, pages, table, page, sl, max_T, SCALE, Hkv, out=out["a"],
                                                 lse=out["al"], pooled=out["p"], ld_pooled=ld, ws=ws)
        yield lambda: api.decode_reuse_paged_q4(one, pages, table, page, sl, idx, ik, hm, SCALE, Hkv, out=out["r"],
                                                lse=out["rl"])

    def outs():
        e = lambda *s, t=dtype: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
        f = torch.float32
        return {"k0": e(B, Hkv, N, 128), "v0": e(B, Hkv, N, 128), "k1": e(B, Hkv, N, 128), "v1": e(B, Hkv, N, 128),
                "a": e(B, Hq, 128), "al": e(B, Hq, t=f), "p": e(B, Hkv, ld, t=f), "r": e(B, Hq, 128),
                "rl": e(B, Hq, t=f), "w": e(B, Hq, 128), "wl": e(B, Hq, t=f)}

    return calls, outs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("B,N,Hq,Hkv,page", [(4, 1, 32, 8, 64), (16, 1, 16, 4, 16), (3, 700, 8, 8, 48)])
def test_rounds_without_a_wait(B, N, Hq, Hkv, page, dtype):
    rounds = 24
    calls, outs = _chain(rounds, dtype, B, N, Hq, Hkv, page, seed=B + N)

    def run(results):
        for r in range(rounds):
            for call in calls(r, results[r]):
                call()

    def same(results, want):
        torch.cuda.synchronize()
        for w, o in zip(want, results):
            for n in w:
                assert torch.equal(w[n], o[n]), n

    want, got = [outs() for _ in range(rounds)], [outs() for _ in range(rounds)]
    for r in range(rounds):
        for call in calls(r, want[r]):
            call()
            torch.cuda.synchronize()
    assert not torch.equal(want[0]["k0"], want[1]["k0"])
    for _ in range(3):
        run(got)
        same(got, want)
    graph = StepGraph(lambda: run(got))
    for _ in range(5):
        graph.replay()
        same(got, want)

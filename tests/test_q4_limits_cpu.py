"""Refusals of the 4-bit cache's calls that need no GPU: page stores whose rows
cannot be counted, read-back outputs that share memory."""
import pytest
import torch

from long_context_emitting_b200 import api, binding, paging
from long_context_emitting_b200.binding import Shape
from test_q4_cpu import HEAD_STRIDES, P, UNSUPPORTED, _bf, fake, lib  # noqa: F401


def test_stores_of_2_to_the_31_rows_are_refused(lib):  # noqa: F811
    s = Shape(2, 8, 8, 128)
    num, size = 1 << 22, 64          # times 8 heads: 2^31 rows
    need = lib.kascade_decode_anchor_paged_q4_workspace_bytes(s, 256)
    got = [
        lib.kascade_kv_write_paged_q4(s, 4, P, HEAD_STRIDES, P, HEAD_STRIDES, P, num, P, 4, size, P, None, None),
        lib.kascade_kv_read_paged_q4(s, 4, P, num, P, 4, size, P, None, P, 2 * P, None),
        lib.kascade_decode_anchor_paged_q4(s, P, P, num, P, 4, size, P, 256, 0.1, P, P, P, 256, P, need, None),
        lib.kascade_decode_reuse_paged_q4(s, P, P, num, P, 4, size, P, P, P, 16, P, 0.1, P, P, None),
    ]
    assert got == [UNSUPPORTED] * 4
    assert num * 8 * size == 2**31 and binding.Q4_ROW_BYTES * 2**31 > 300 << 30


def test_read_back_outputs_must_not_share_memory(fake):  # noqa: F811
    pages, table = paging.q4_store([40, 1], 2, 16, "cpu")
    z = torch.zeros(2, dtype=torch.int32)
    buf = _bf(2 * 2 * 2 * 5 * 128 + 128)
    n = 2 * 2 * 5 * 128
    api.kv_read_paged_q4(pages, table, 16, z, None, 5, k=buf[:n], v=buf[n:])
    for a, b in ((buf[:n], buf[:n]), (buf[:n], buf[n - 128:]), (buf[64:], buf[:n])):
        with pytest.raises(ValueError):
            api.kv_read_paged_q4(pages, table, 16, z, None, 5, k=a, v=b)


def test_norm_rope_output_overlaps(fake):  # noqa: F811
    """An output may be its own input's view and nothing else that overlaps."""
    buf = _bf(3, 2, 4, 8, 128)
    q, k = buf[0], _bf(2, 4, 2, 128)
    pos, inv = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(64)
    api.qk_norm_rope(q, k, pos, inv, q_out=q.transpose(1, 2))
    api.qk_norm_rope(q, k, pos, inv, q_out=buf[1].transpose(1, 2))
    flat = buf.view(-1)
    shifted = flat[128:128 + q.numel()].view(2, 4, 8, 128)
    over = buf[:, 0].unsqueeze(0).expand(2, 3, 4, 8, 128)[:, 0].transpose(1, 2)  # q's first sequence, twice
    for out in (shifted.transpose(1, 2), over):
        with pytest.raises(ValueError):
            api.qk_norm_rope(q, k, pos, inv, q_out=out)
    with pytest.raises(ValueError):   # k_out over q's rows
        api.qk_norm_rope(q, k, pos, inv, k_out=q[:, :, :2].transpose(1, 2))

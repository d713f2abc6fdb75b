"""Tensors whose dimensions of length 1 carry odd strides: the same results as their plain copies."""
import pytest
import torch

from long_context_emitting_b200 import api, paging
from test_q4_gpu import DEV, TYPES, _gen, _i32, _randn

pytestmark = pytest.mark.gpu


def _odd(x, dim):
    """x, 1 long in ``dim``, with the strides that a permuted tensor has there."""
    y = torch.empty(*(n for i, n in enumerate(x.shape) if i != dim), 1, dtype=x.dtype, device=x.device).movedim(-1, dim)
    y.copy_(x)
    assert y.stride(dim) == 1 and torch.equal(x, y)
    return y


@TYPES
@pytest.mark.parametrize("B,N,H,dim", [(3, 1, 4, 1), (1, 5, 4, 0), (3, 5, 1, 2), (1, 1, 1, 1)])
def test_odd_strides_where_nothing_is_strided(B, N, H, dim, dtype):
    g = _gen(B + 10 * N + 100 * H)
    q, k = (_randn(g, B, N, H, 128).to(dtype) for _ in range(2))
    pos = torch.arange(N, device=DEV, dtype=torch.int32).repeat(B, 1)
    inv = torch.rand(64, generator=g, device=DEV)
    want = api.qk_norm_rope(q, k, pos, inv)
    out = _odd(torch.zeros(B, N, H, 128, dtype=dtype, device=DEV), dim).transpose(1, 2)
    got = api.qk_norm_rope(_odd(q, dim), _odd(k, dim), pos, inv, q_out=out)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and got[0] is out
    pages, table = paging.q4_store([N] * B, H, 16, DEV)
    other = pages.clone()
    api.kv_write_paged_q4(want[0], want[1], pages, table, 16, _i32(*([0] * B)))
    api.kv_write_paged_q4(out, _odd(want[1].transpose(1, 2), dim).transpose(1, 2), other, table, 16, _i32(*([0] * B)))
    assert torch.equal(pages, other) and int(pages.max()) > 0
    assert api.device_status() == 0

"""Buffers that hold enough elements, but not where the call looks for them, are
refused; ones with room for more sequences, and flat ones, are taken."""
import pytest
import torch

from long_context_emitting_b200 import api, paging
from test_q4_cpu import _bf, fake  # noqa: F401


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_norm_rope_layouts(fake):  # noqa: F811
    q, k = _bf(2, 3, 8, 128), _bf(2, 3, 2, 128)
    inv = torch.zeros(64)
    for pos in (_i32(2, 3), _i32(6), _i32(5, 3), _i32(9)):
        api.qk_norm_rope(q, k, pos, inv)
    for pos in (_i32(2, 4), _i32(3, 2), _i32(2, 3, 2), _i32(1, 8)):
        with pytest.raises(ValueError, match="positions"):
            api.qk_norm_rope(q, k, pos, inv)
    one = q[:, :1]
    for pos in (_i32(2), _i32(2, 1), _i32(4), _i32(4, 1)):      # one token per sequence
        api.qk_norm_rope(one, k[:, :1], pos, inv)
    with pytest.raises(ValueError, match="positions"):
        api.qk_norm_rope(one, k[:, :1], _i32(2, 4), inv)
    pos = _i32(2, 3)
    for kw in (dict(inv_freq=torch.zeros(128)), dict(inv_freq=torch.zeros(2, 64)), dict(q_weight=_bf(256)),
               dict(k_weight=_bf(2, 128))):
        with pytest.raises(ValueError):
            api.qk_norm_rope(q, k, pos, **({"inv_freq": inv} | kw))


def test_read_back_layouts(fake):  # noqa: F811
    pages, table = paging.q4_store([40, 1], 2, 16, "cpu")
    z = _i32(2)
    api.kv_read_paged_q4(pages, table, 16, z, None, 5, k=_bf(3, 2, 5, 128), v=_bf(9999 * 128))
    for bad in (_bf(2, 2, 8, 128), _bf(2, 4, 5, 128), _bf(2, 2, 5, 256)):
        for kw in (dict(k=bad), dict(v=bad)):
            with pytest.raises(ValueError):
                api.kv_read_paged_q4(pages, table, 16, z, None, 5, **kw)
    with pytest.raises(ValueError):
        api.kv_read_paged_q4(pages, table, 16, z, _i32(2, 2), 5)


def test_attention_layouts(fake):  # noqa: F811
    lens = [40, 1]
    pages, table = paging.q4_store(lens, 2, 16, "cpu")
    q, sl = _bf(2, 8, 128), torch.tensor(lens, dtype=torch.int32)
    anchor = lambda **kw: api.decode_anchor_paged_q4(q, pages, table, 16, kw.pop("sl", sl), 40, 0.1, 2, **kw)  # noqa: E731
    anchor(out=_bf(3, 8, 128), lse=torch.zeros(3, 8), pooled=torch.zeros(3, 2, 40))
    anchor(pooled=torch.zeros(2, 2, 48), ld_pooled=48)
    anchor(pooled=torch.zeros(4096))
    for kw in (dict(pooled=torch.zeros(2, 2, 48)), dict(pooled=torch.zeros(2, 4, 40)), dict(out=_bf(2, 16, 128)),
               dict(lse=torch.zeros(2, 16)), dict(sl=_i32(2, 2))):
        with pytest.raises(ValueError):
            anchor(**kw)
    idx, ik, hm = _i32(2, 2, 7), _i32(4), torch.tensor([0, 1], dtype=torch.int32)
    reuse = lambda **kw: api.decode_reuse_paged_q4(q, pages, table, 16, sl, *(kw.get(n, d) for n, d in  # noqa: E731
                                                   (("idx", idx), ("ik", ik), ("hm", hm))), 0.1, 2)
    reuse()
    reuse(idx=_i32(4, 7), ik=_i32(2, 2))
    reuse(idx=_i32(3, 2, 7), ik=_i32(3, 2), hm=_i32(5))
    for kw in (dict(idx=_i32(2, 4, 7)), dict(ik=_i32(2, 4)), dict(hm=_i32(2, 2))):
        with pytest.raises(ValueError):
            reuse(**kw)


def test_rows_lie_where_memory_says_so():
    """Against the places of the elements themselves: a longer buffer is taken only if the call's rows start it."""
    import itertools

    for inner in ((), (3,), (2, 3), (2, 1, 4)):
        rows = 1
        for x in inner:
            rows *= x
        for n in range(1, 4):
            for shape in itertools.product(range(1, 6), repeat=n):
                t = torch.empty(shape)
                if api._rows_lie(t, inner):
                    # the dimensions after the first split a row of `inner`, or are one
                    rest = t[0].numel()
                    assert rows % rest == 0
    for t, inner, ok in ((_i32(5, 1), (), True), (_i32(5, 2), (), False), (_i32(8, 7), (2, 7), True),
                         (_i32(3, 2, 7), (2, 7), True), (_i32(3, 4, 7), (2, 7), False), (_i32(3, 7, 2), (2, 7), False),
                         (_i32(3, 2), (2, 7), False), (_i32(9), (2, 7), True), (_i32(4, 3, 1), (3,), True)):
        assert api._rows_lie(t, inner) == ok, (t.shape, inner)


def test_harmless_longer_buffers_are_taken(fake):  # noqa: F811
    q, k = _bf(2, 3, 8, 128), _bf(2, 3, 2, 128)
    api.qk_norm_rope(q, k, _i32(2, 3, 1), torch.zeros(1, 64))
    pages, table = paging.q4_store([40, 1], 2, 16, "cpu")
    api.kv_read_paged_q4(pages, table, 16, _i32(2), _i32(5, 1), 5, k=_bf(99, 128))
    q, sl = _bf(2, 8, 128), _i32(4, 1)
    api.decode_anchor_paged_q4(q, pages, table, 16, sl, 40, 0.1, 2, pooled=torch.zeros(9, 40))
    api.decode_reuse_paged_q4(q, pages, table, 16, sl, _i32(9, 7), _i32(7, 1), _i32(3, 1), 0.1, 2)

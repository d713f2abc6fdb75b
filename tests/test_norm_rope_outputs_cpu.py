"""Which outputs the norms and the rotation take: none that shares memory with
what the same call still reads or writes elsewhere."""
import itertools
import random

import pytest
import torch

from long_context_emitting_b200 import api
from test_q4_cpu import _bf, fake  # noqa: F401


def test_norm_rope_outputs_may_not_meet(fake):  # noqa: F811
    """An output over the other one's input, over the other output, or over itself is refused."""
    q, k = _bf(2, 4, 2, 128), _bf(2, 4, 2, 128)
    pos, inv = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(64)
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    api.qk_norm_rope(q, k, pos, inv, q_out=t(q), k_out=t(k))
    out = _bf(2, 2, 4, 128)
    twice = _bf(5, 128)[:4].expand(2, 2, 4, 128)
    for kw in ({"k_out": t(q)}, {"q_out": t(k)}, {"q_out": t(k), "k_out": t(q)}, {"q_out": out, "k_out": out},
               {"q_out": twice}, {"k_out": _bf(9, 128).as_strided((2, 2, 4, 128), (128, 128, 128, 1))}):
        with pytest.raises(ValueError, match="overlap"):
            api.qk_norm_rope(q, k, pos, inv, **kw)
    # One tensor for both inputs: read twice, so neither output may replace it.
    api.qk_norm_rope(q, q, pos, inv, q_out=out)
    for kw in ({"q_out": t(q)}, {"k_out": t(q)}):
        with pytest.raises(ValueError, match="overlap"):
            api.qk_norm_rope(q, q, pos, inv, **kw)


@pytest.mark.parametrize("B,N", [(1, 1), (1, 4), (3, 1), (2, 5)])
def test_norm_rope_outputs_inside_packed_rows(fake, B, N):  # noqa: F811
    """Views that interleave without a shared row are taken: in place in packed rows, also of padded
    sequences, over V's rows, and two outputs of one buffer."""
    rows = _bf(B, N + 2, 4 + 2 + 4, 128)[:, :N]
    q, k, v = rows.split((4, 2, 4), 2)
    pos, inv = torch.zeros(B, N, dtype=torch.int32), torch.zeros(64)
    t = lambda x: x.transpose(1, 2)  # noqa: E731
    api.qk_norm_rope(q, k, pos, inv, q_out=t(q), k_out=t(k))
    api.qk_norm_rope(q, k, pos, inv, q_out=t(v), k_out=t(k))
    both = _bf(B, 6, N, 128)
    api.qk_norm_rope(q, k, pos, inv, q_out=both[:, :4], k_out=both[:, 4:])
    for kw in ({"q_out": both[:, :4], "k_out": both[:, 3:5]}, {"q_out": t(rows[:, :, 1:5])},
               {"q_out": t(v), "k_out": t(v[:, :, :2])}, {"q_out": t(rows[:, :, 4:8]), "k_out": t(k)}):
        with pytest.raises(ValueError, match="overlap"):
            api.qk_norm_rope(q, k, pos, inv, **kw)


def test_rows_apart_against_every_row():
    """The search for rows that meet, against all pairs of rows of small views."""
    g = random.Random(5)
    verdicts = [0, 0]
    for _ in range(3000):
        dims = lambda: tuple((g.choice((0, 64, 128, 256, 384, 640, 1280, 8 * g.randrange(200))), g.randrange(1, 4))  # noqa: E731
                             for _ in range(3))
        xs = dims()
        ys = tuple((s, g.randrange(1, 4)) for s, _ in xs) if g.random() < 0.6 else dims()
        delta = 16 * g.randrange(-300, 300)
        first = lambda v: [2 * sum(i * s for i, (s, _) in zip(at, v))  # noqa: E731
                           for at in itertools.product(*(range(n) for _, n in v))]
        want = all(abs(delta + x - y) >= 256 for x in first(xs) for y in first(ys))
        assert api._rows_apart(delta, xs, ys) == want, (delta, xs, ys)
        verdicts[want] += 1
    assert min(verdicts) > 300

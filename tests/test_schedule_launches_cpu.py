"""Kernel launches counted for a step of each schedule."""
import torch

from long_context_emitting_b200.schedule import DecodeSchedule, PagedQ4DecodeSchedule, PrefillSchedule, launches_per_step


def test_launches_per_step():
    wide = DecodeSchedule(1, 8, 2, [500], (0, 3), 5, "cpu")
    q4 = PagedQ4DecodeSchedule(1, 8, 2, [500], (0, 3), 5, "cpu", torch.zeros(64))
    pre = PrefillSchedule(1, 8, 2, 256, (0,), 3, "cpu")
    assert launches_per_step(wide, None) == 2 * (2 + 1) + 3
    # every layer also normalises and appends
    assert launches_per_step(q4, None) == 2 * (2 + 1) + 3 + 5 * 2
    assert launches_per_step(None, pre) == (2 + 1) + 2
    assert launches_per_step(q4, pre) == launches_per_step(q4, None) + launches_per_step(None, pre)

"""Host checks of the diagnostic call of the 4-bit anchor: those of the call itself, and the block's number."""
from long_context_emitting_b200 import binding
from long_context_emitting_b200.binding import Shape
from test_q4_cpu import INVALID, OK, P, UNSUPPORTED, WS_SMALL


def test_gives_up_host_checks():
    def call(block=0, s=Shape(2, 32, 8, 128), q=P, wb=1 << 30):
        return binding.load().kascade_selftest_anchor_q4_gives_up(block, s, q, P, 8, P, 4, 64, P, 256, 0.1, P, P, P, 256, P,
                                                                  wb, None)
    assert call(block=-1) == INVALID and call(q=None) == INVALID and call(wb=0) == WS_SMALL
    assert call(s=Shape(2, 32, 8, 64)) == UNSUPPORTED and call(s=Shape(0, 32, 8, 128)) == OK

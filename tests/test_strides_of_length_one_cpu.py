"""The stride of a dimension that is 1 long has no meaning; PyTorch leaves any number
there.  Strides of longer dimensions are refused as before."""
import torch

from long_context_emitting_b200 import binding
from test_hostcall_cpu import INVALID, OK, _norm, _write

def _status(make, **kw):
    name, plain, _ = make(**kw)
    return getattr(binding.load(), "host_" + name)(0, *plain)


def test_strides_that_mean_something():
    x = torch.empty(2, 8, 128, 1).permute(0, 3, 1, 2)
    assert x.is_contiguous() and x.stride(1) == 1            # one token per sequence
    # the checks' own answer, without a launch: an empty batch is taken whatever its strides
    assert _status(_norm, B=0, qs=(3, 3, 3)) == OK and _status(_write, B=0, ks=(3, 3, 3)) == OK
    for kw in (dict(qs=(4, 4096, 128)), dict(qs=(16384, 1, 128)), dict(ks=(4096, 1024, 1)), dict(qos=(16384, 1, 128))):
        assert _status(_norm, **kw) == INVALID
    for kw in (dict(ks=(4, 1024, 128)), dict(vs=(1024, 1, 128))):
        assert _status(_write, **kw) == INVALID

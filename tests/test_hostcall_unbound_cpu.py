"""A call through the CPython module before the library's addresses are bound is an error, not a jump to nowhere."""
import subprocess
import sys

from long_context_emitting_b200 import binding

CODE = """
import importlib.util, sys
spec = importlib.util.spec_from_file_location("_hostcall", sys.argv[1])
m = importlib.util.module_from_spec(spec)
spec.loader.exec_module(m)
for name, n in (("norm_rope", 29), ("kv_write", 22), ("kv_read", 16), ("decode_anchor", 21), ("decode_reuse", 20)):
    try:
        getattr(m, name)(*[0] * n)
    except RuntimeError as e:
        assert "bind" in str(e)
    else:
        sys.exit(name)
"""


def test_calls_before_bind_raise():
    binding.load()
    from long_context_emitting_b200 import _hostcall
    r = subprocess.run([sys.executable, "-c", CODE, _hostcall.__file__], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)

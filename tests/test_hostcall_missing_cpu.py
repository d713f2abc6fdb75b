"""The library without its CPython module (no Python headers where it was built):
everything loads, and the calls that go through the module go through ctypes, with
the same status and the same refusals.  The module's file is the interpreter's own."""
import os
import subprocess
import sys
import sysconfig

import pytest

from long_context_emitting_b200 import binding, build
from test_hostcall_cpu import CASES, OK, _anchor, _norm, _read, _reuse, _write

WITHOUT = """
import sys
sys.modules["long_context_emitting_b200._hostcall"] = None      # importing it fails
from long_context_emitting_b200 import binding
lib = binding.load()
assert lib.kascade_k_for_len(4096) == 410
assert lib.host_kv_read(0, 0, 8, 8, 128, 4, None, 8, None, 4, 64, None, None, None, None, None) == 0
assert lib.host_kv_read(0, 2, 8, 8, 128, 4, None, 8, None, 4, 64, None, None, None, None, None) == 1
"""


def test_library_loads_without_the_module():
    root = os.path.dirname(os.path.dirname(os.path.abspath(binding.__file__)))
    r = subprocess.run([sys.executable, "-c", WITHOUT], capture_output=True, text=True, cwd=root)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("make,bad", CASES, ids=[f"{m.__name__[1:]}-{i}" for i, (m, _) in enumerate(CASES)])
def test_same_status_through_ctypes(make, bad, half):
    lib = binding.load()
    name, plain, _ = make(**bad)
    assert binding.ctypes_hostcall(lib, name)(half, *plain) == getattr(lib, "host_" + name)(half, *plain)


def test_same_refusals_through_ctypes():
    lib = binding.load()
    for make in (_norm, _write, _read, _anchor, _reuse):
        name, plain, _ = make(B=0)
        fn = binding.ctypes_hostcall(lib, name)
        assert fn(0, *plain) == OK
        for args in (plain, (0, *plain, 0), (), (0, "2", *plain[1:]), (0, 2.5, *plain[1:])):
            with pytest.raises(TypeError):
                fn(*args)
        for args in ((0, 1 << 31, *plain[1:]), (0, 0, *plain[1:5], 1 << 70, *plain[6:])):
            with pytest.raises(OverflowError):
                fn(*args)
    name, plain, _ = _reuse(B=0)
    with pytest.raises(TypeError):
        binding.ctypes_hostcall(lib, name)(0, *plain[:15], None, *plain[16:])   # the scale


def test_module_file_is_this_interpreters():
    from long_context_emitting_b200 import _hostcall
    assert os.path.basename(_hostcall.__file__) == "_hostcall" + sysconfig.get_config_var("EXT_SUFFIX")
    assert build.HOSTCALL == _hostcall.__file__
    assert build.hostcall_command("x")[0] == build.nvcc()


def test_build_state_without_headers(monkeypatch, tmp_path):
    """Without Python.h the library alone decides whether a build is up to date."""
    assert build.python_headers()
    monkeypatch.setattr(build, "HOSTCALL", str(tmp_path / "none.so"))
    assert not build.up_to_date()
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.python_headers() is None
    monkeypatch.setattr(build, "_inputs", lambda: [])
    assert build.up_to_date()

"""The CPython module through which the decode step's small entry points are called:
its arguments arrive where ctypes puts them, and what does not fit is refused."""
import pytest

from long_context_emitting_b200 import binding
from long_context_emitting_b200.binding import Shape, Strides

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
P = 0x10000  # a fake 16-byte aligned address, never read on the host


@pytest.fixture(scope="module")
def lib():
    return binding.load()


# (name, plain arguments after the half-precision flag, what ctypes takes for them)
def _norm(B=2, Hq=32, Hkv=8, d=128, N=4, q=P, qs=(16384, 4096, 128), k=2 * P, ks=(4096, 1024, 128), pos=P, inv=P, qw=P,
          kw=None, eps=1e-6, inter=0, qo=3 * P, qos=(16384, 4096, 128), ko=4 * P, kos=(4096, 1024, 128)):
    return ("norm_rope", (B, Hq, Hkv, d, N, q, *qs, k, *ks, pos, inv, qw, kw, eps, inter, qo, *qos, ko, *kos, None),
            (Shape(B, Hq, Hkv, d), N, q, Strides(*qs), k, Strides(*ks), pos, inv, qw, kw, eps, inter, qo, Strides(*qos), ko,
             Strides(*kos), None))


def _write(B=2, H=8, d=128, N=4, k=P, ks=(1024, 1024, 128), v=P, vs=(1024, 1024, 128), pages=P, num=8, table=P, per=4,
           size=64, start=P, count=None):
    return ("kv_write", (B, H, H, d, N, k, *ks, v, *vs, pages, num, table, per, size, start, count, None),
            (Shape(B, H, H, d), N, k, Strides(*ks), v, Strides(*vs), pages, num, table, per, size, start, count, None))


def _read(B=2, H=8, d=128, N=4, pages=P, num=8, table=P, per=4, size=64, start=P, count=None, k=P, v=2 * P):
    return ("kv_read", (B, H, H, d, N, pages, num, table, per, size, start, count, k, v, None),
            (Shape(B, H, H, d), N, pages, num, table, per, size, start, count, k, v, None))


def _anchor(B=2, Hq=32, Hkv=8, d=128, q=P, pages=P, num=8, table=P, per=4, size=64, sl=P, T=256, scale=0.1, out=P, lse=P,
            pooled=P, ld=256, ws=P, wb=16):
    return ("decode_anchor", (B, Hq, Hkv, d, q, pages, num, table, per, size, sl, T, scale, out, lse, pooled, ld, ws, wb, None),
            (Shape(B, Hq, Hkv, d), q, pages, num, table, per, size, sl, T, scale, out, lse, pooled, ld, ws, wb, None))


def _reuse(B=2, Hq=32, Hkv=8, d=128, q=P, pages=P, num=8, table=P, per=4, size=64, sl=P, idx=P, ik=P, k=16, hm=P,
           scale=0.1, out=P, lse=P):
    return ("decode_reuse", (B, Hq, Hkv, d, q, pages, num, table, per, size, sl, idx, ik, k, hm, scale, out, lse, None),
            (Shape(B, Hq, Hkv, d), q, pages, num, table, per, size, sl, idx, ik, k, hm, scale, out, lse, None))


# every field in turn is made wrong; each case ends in a host check, before any launch
CASES = [
    *[(_norm, b) for b in (dict(q=None), dict(k=None), dict(pos=None), dict(inv=P + 2), dict(qw=P + 8), dict(kw=P + 8),
                           dict(eps=-1.0), dict(eps=float("nan")), dict(qs=(16, 4, 128)), dict(ks=(8, 8, 4)),
                           dict(qs=(-8, 8, 8)), dict(qo=None), dict(qos=(16384, 4096, 0)), dict(ko=None),
                           dict(kos=(0, 1024, 128)), dict(kos=(4096, 0, 128)), dict(N=-1), dict(N=0), dict(B=0), dict(B=-1),
                           dict(Hq=0), dict(Hq=5000), dict(Hkv=5000), dict(d=64), dict(B=1 << 20, N=1 << 20))],
    *[(_write, b) for b in (dict(k=None), dict(v=None), dict(ks=(8, 12, 8)), dict(vs=(8, 8, 12)), dict(pages=P + 8),
                            dict(num=0), dict(table=P + 2), dict(per=0), dict(size=24), dict(start=None), dict(count=P + 2),
                            dict(N=-1), dict(N=0), dict(B=0), dict(H=0), dict(H=5000), dict(d=64), dict(num=1 << 22))],
    *[(_read, b) for b in (dict(pages=None), dict(num=-1), dict(table=None), dict(per=-3), dict(size=8), dict(start=None),
                           dict(count=P + 1), dict(k=None), dict(v=P), dict(v=P + 4), dict(N=0), dict(B=0), dict(H=0),
                           dict(d=256))],
    *[(_anchor, b) for b in (dict(), dict(q=P + 2), dict(pages=None), dict(num=0), dict(table=None), dict(per=3),
                             dict(size=40), dict(sl=None), dict(T=-1), dict(scale=float("inf")), dict(out=None),
                             dict(lse=P + 4), dict(pooled=None), dict(ld=252), dict(ld=258), dict(ws=None), dict(wb=0),
                             dict(Hq=24), dict(Hkv=0), dict(B=70000), dict(B=0), dict(d=64), dict(ld=(1 << 33) + 1))],
    *[(_reuse, b) for b in (dict(q=None), dict(pages=P + 8), dict(num=0), dict(table=None), dict(per=0), dict(size=17),
                            dict(sl=P + 1), dict(idx=None), dict(ik=None), dict(k=-1), dict(hm=None),
                            dict(scale=float("nan")), dict(out=None), dict(lse=P + 4), dict(Hq=24), dict(B=0),
                            dict(B=70000), dict(d=64))],
]


@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("make,bad", CASES, ids=[f"{m.__name__[1:]}-{i}" for i, (m, _) in enumerate(CASES)])
def test_same_status_as_ctypes(lib, make, bad, half):
    name, plain, struct = make(**bad)
    want = getattr(lib, binding.HOSTCALLS[name] + ("_f16" if half else ""))(*struct)
    assert want in (OK, INVALID, UNSUPPORTED, WS_SMALL)
    assert want != OK or 0 in plain[:5]     # nothing was launched
    assert getattr(lib, "host_" + name)(half, *plain) == want


def test_what_does_not_fit_is_refused(lib):
    for make in (_norm, _write, _read, _anchor, _reuse):
        name, plain, _ = make(B=0)
        fn = getattr(lib, "host_" + name)
        assert fn(0, *plain) == OK
        for args in (plain, (0, *plain, 0), (), (0, "2", *plain[1:]), (0, 2.5, *plain[1:])):
            with pytest.raises(TypeError):
                fn(*args)
        with pytest.raises(OverflowError):
            fn(0, 1 << 31, *plain[1:])
        with pytest.raises(OverflowError):
            fn(0, 0, *plain[1:5], 1 << 70, *plain[6:])
    name, plain, _ = _reuse(B=0)
    with pytest.raises(TypeError):
        lib.host_decode_reuse(0, *plain[:15], None, *plain[16:])   # the scale

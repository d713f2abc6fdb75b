"""The 4-bit cache and the head norms on the CPU: the oracle's definitions
against plain loops and exact fractions, the host checks of the entry points
(no GPU: every call here is refused or empty), and the Python layer's checks."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle as O
from long_context_emitting_b200 import api, binding, paging
from long_context_emitting_b200.binding import Shape, Strides
from long_context_emitting_b200.schedule import PagedQ4DecodeSchedule

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
P = 0x10000  # a fake 16-byte aligned address, never read on the host
HEAD_STRIDES = Strides(8 * 128, 8 * 128, 128)


@pytest.fixture(scope="module")
def lib():
    return binding.load()


# ------------------------------------------------------------------ oracle ----
def _bf16_grid(x, up):
    """Directed rounding to bfloat16 by stepping through its numbers."""
    b = torch.tensor(x, dtype=torch.float64).to(torch.bfloat16)
    while up and b.double().item() < x:
        b = torch.nextafter(b, torch.tensor(math.inf, dtype=torch.bfloat16))
    while not up and b.double().item() > x:
        b = torch.nextafter(b, torch.tensor(-math.inf, dtype=torch.bfloat16))
    return b.double().item()


@pytest.mark.parametrize("up", [True, False])
def test_oracle_bf16_toward(up):
    g = np.random.default_rng(0)
    xs = list(g.standard_normal(50)) + list(g.standard_normal(20) * 1e-40) + [0.0, 1.0, -1.0, 1 / 3, 1e30, -1e-39]
    for x in xs:
        assert O.bf16_toward(x, up) == _bf16_grid(x, up), x


def _rint_fraction(q: Fraction) -> int:
    f = math.floor(q)
    r = q - f
    return f + (1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2) else 0)


def test_oracle_quantise_against_fractions():
    g = np.random.default_rng(1)
    x = np.concatenate([g.standard_normal((4, 128)), np.round(g.standard_normal((4, 128)) * 8) / 2])
    n, s, m = O.q4_quantise(x)
    for r in range(x.shape[0]):
        for c in range(128):
            sg, mg = Fraction(float(s[r, c // 32])), Fraction(float(m[r, c // 32]))
            assert n[r, c] == _rint_fraction((Fraction(float(x[r, c])) - mg) / sg)
    assert n.min() >= 0 and n.max() <= 15
    # no value clips: every value is within half a scale
    assert (np.abs(O.q4_values(n, s, m) - x) <= np.repeat(s, 32, -1) / 2 * (1 + 1e-12)).all()


def test_oracle_pack_round_trip_and_places():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((3, 128)), g.standard_normal((3, 128))
    rows = O.q4_pack(k, v)
    (nk, sk, mk), (nv, sv, mv) = O.q4_unpack(rows)
    for x, n, s, m in ((k, nk, sk, mk), (v, nv, sv, mv)):
        n0, s0, m0 = O.q4_quantise(x)
        assert np.array_equal(n, n0) and np.array_equal(s, s0) and np.array_equal(m, m0)
    # channel 37 of K: group 1, lane 0, code 5 -> word 1, nibble 5; of V: word 2, half 1, nibble 1
    one = np.zeros((1, 128))
    one[0, 37] = 1.0
    row = O.q4_pack(one, one)[0]
    assert [i for i in range(128) if row[i]] == [4 + 2, 64 + 8 + 2] and row[6] == 0xf0 and row[64 + 10] == 0xf0
    # constants: code 0, scale 0
    assert not O.q4_pack(np.full((1, 128), 2.0), np.zeros((1, 128)))[0, :128].any()


def test_oracle_norm_rope_by_loops():
    g = np.random.default_rng(3)
    x, w = g.standard_normal((1, 2, 1, 128)), g.standard_normal(128)
    inv = 10000.0 ** (-np.arange(64) / 64)
    pos = np.array([[0, 7]])
    for inter in (False, True):
        got = O.norm_rope(x, pos, inv, w, 1e-6, inter)
        for n in range(2):
            y = x[0, n, 0] / math.sqrt(sum(t * t for t in x[0, n, 0]) / 128 + 1e-6) * w
            for i in range(64):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 64)
                z = complex(y[a], y[b]) * complex(math.cos(pos[0, n] * inv[i]), math.sin(pos[0, n] * inv[i]))
                assert abs(got[0, 0, n, a] - z.real) < 1e-12 and abs(got[0, 0, n, b] - z.imag) < 1e-12
    assert np.array_equal(O.norm_rope(x, pos, inv)[0, 0, 0], x[0, 0, 0])  # position 0 without a norm


# ------------------------------------------------------------- host checks ----
def test_norm_rope_host_checks(lib):
    s = Shape(2, 32, 8, 128)
    qs, ks = Strides(4 * 4096, 4096, 128), Strides(4 * 1024, 1024, 128)

    def call(s=s, N=4, q=P, qs=qs, k=2 * P, ks=ks, pos=P, inv=P, qw=P, eps=1e-6, qo=3 * P, qos=qs, ko=4 * P, kos=ks):
        return lib.kascade_qk_norm_rope(s, N, q, qs, k, ks, pos, inv, qw, None, eps, 0, qo, qos, ko, kos, None)

    for bad in (dict(q=None), dict(k=None), dict(pos=None), dict(inv=None), dict(qo=None), dict(ko=None),
                dict(q=P + 2), dict(qw=P + 8), dict(pos=P + 2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(N=-1), dict(qs=Strides(16, 4, 128)), dict(qs=Strides(-8, 8, 8)),
                dict(qos=Strides(4 * 4096, 4096, 0)), dict(kos=Strides(0, 1024, 128)), dict(qo=P, ko=P),
                dict(s=Shape(2, 0, 8, 128)), dict(s=Shape(-1, 32, 8, 128))):
        assert call(**bad) == INVALID, bad
    assert call(s=Shape(2, 32, 8, 64)) == UNSUPPORTED
    assert call(s=Shape(1 << 20, 32, 8, 128), N=1 << 20) == UNSUPPORTED
    assert call(N=0, q=None, k=None) == OK
    assert call(s=Shape(0, 32, 8, 128), q=None) == OK


def test_cache_host_checks(lib):
    s = Shape(2, 8, 8, 128)

    def write(s=s, N=4, k=P, st=HEAD_STRIDES, v=P, pages=P, num=8, table=P, per=4, size=64, start=P, count=None):
        return lib.kascade_kv_write_paged_q4(s, N, k, st, v, HEAD_STRIDES, pages, num, table, per, size, start, count,
                                             None)

    def read(s=s, N=4, pages=P, num=8, table=P, per=4, size=64, start=P, count=None, k=P, v=2 * P):
        return lib.kascade_kv_read_paged_q4_f16(s, N, pages, num, table, per, size, start, count, k, v, None)

    for bad in (dict(k=None), dict(v=None), dict(pages=None), dict(table=None), dict(start=None), dict(num=0),
                dict(per=0), dict(size=24), dict(size=0), dict(pages=P + 8), dict(k=P + 4), dict(table=P + 2),
                dict(count=P + 2), dict(st=Strides(8, 12, 8)), dict(N=-1), dict(s=Shape(2, 8, 0, 128))):
        assert write(**bad) == INVALID, bad
    for bad in (dict(k=None), dict(v=None), dict(v=P), dict(pages=None), dict(start=None), dict(size=8),
                dict(k=P + 4)):
        assert read(**bad) == INVALID, bad
    assert write(s=Shape(2, 8, 8, 64)) == UNSUPPORTED and read(s=Shape(2, 8, 5000, 128)) == UNSUPPORTED
    assert write(N=0, k=None) == OK and read(N=0, k=None) == OK and write(s=Shape(0, 8, 8, 128), k=None) == OK


def test_decode_q4_host_checks(lib):
    s = Shape(2, 32, 8, 128)

    def anchor(s=s, q=P, pages=P, num=8, table=P, per=4, size=64, sl=P, T=256, scale=0.1, out=P, pooled=P, ld=256,
               ws=P, wb=1 << 30):
        return lib.kascade_decode_anchor_paged_q4(s, q, pages, num, table, per, size, sl, T, scale, out, P, pooled, ld,
                                                  ws, wb, None)

    def reuse(s=s, q=P, pages=P, num=8, table=P, per=4, size=64, sl=P, idx=P, ik=P, k=16, hm=P, scale=0.1, out=P):
        return lib.kascade_decode_reuse_paged_q4(s, q, pages, num, table, per, size, sl, idx, ik, k, hm, scale, out, P,
                                                 None)

    for bad in (dict(q=None), dict(pages=None), dict(table=None), dict(sl=None), dict(out=None), dict(pooled=None),
                dict(ws=None), dict(q=P + 2), dict(pages=P + 8), dict(size=40), dict(num=0), dict(per=3),
                dict(ld=252), dict(ld=258), dict(scale=float("inf")), dict(T=-1), dict(s=Shape(2, 32, 0, 128))):
        assert anchor(**bad) == INVALID, bad
    for bad in (dict(q=None), dict(pages=None), dict(idx=None), dict(ik=None), dict(hm=None), dict(out=None),
                dict(k=-1), dict(scale=float("nan")), dict(size=17), dict(idx=P + 2)):
        assert reuse(**bad) == INVALID, bad
    for shape in (Shape(2, 32, 8, 64), Shape(2, 24, 8, 128), Shape(70000, 32, 8, 128)):
        assert anchor(s=shape) == UNSUPPORTED and reuse(s=shape) == UNSUPPORTED
    need = lib.kascade_decode_anchor_paged_q4_workspace_bytes(s, 256)
    assert need >= 2 * 8 * 256 * 4 * 4
    assert anchor(wb=need - 1) == WS_SMALL
    assert lib.kascade_decode_anchor_paged_q4_workspace_bytes(Shape(2, 32, 8, 64), 256) == 0
    empty = Shape(0, 32, 8, 128)
    assert anchor(s=empty, q=None) == OK and reuse(s=empty, q=None) == OK


# ----------------------------------------------------------- Python checks ----
class _FakeLib:
    def __getattr__(self, name):
        return (lambda *a: 256) if name.endswith("_workspace_bytes") else (lambda *a: 0)


@pytest.fixture
def fake(monkeypatch):
    def need(name, t, dtype):
        if t.dtype != dtype or not t.is_contiguous():
            raise ValueError(name)

    def rows(name, t, dtype, shape):
        if t.dtype != dtype or tuple(t.shape) != shape or (t.stride(-1) != 1 and t.numel()):
            raise ValueError(name)
    monkeypatch.setattr(api, "_lib", lambda: _FakeLib())
    monkeypatch.setattr(api, "_need_cuda", need)
    monkeypatch.setattr(api, "_need_rows", rows)
    monkeypatch.setattr(api, "_ws_bytes", lambda ws: ws.numel() * ws.element_size())
    monkeypatch.setattr(api, "_stream", lambda: 0)
    monkeypatch.setattr(api, "k_for_len", O.k_for_len)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_python_checks_norm_rope(fake):
    q, k = _bf(2, 3, 8, 128), _bf(2, 3, 2, 128)
    pos, inv = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(64)
    qo, ko = api.qk_norm_rope(q, k, pos, inv)
    assert qo.shape == (2, 8, 3, 128) and ko.shape == (2, 2, 3, 128)
    api.qk_norm_rope(q, k, pos, inv, q_out=q.transpose(1, 2), k_out=k.transpose(1, 2))  # in place
    packed = _bf(2, 3, 12, 128)
    pq, pk = packed[:, :, :8], packed[:, :, 8:10]
    api.qk_norm_rope(pq, pk, pos, inv, q_out=pq.transpose(1, 2), k_out=pk.transpose(1, 2))
    for bad in (dict(q_out=pk.transpose(1, 2).expand(2, 2, 3, 128)), dict(q_out=_bf(2, 3, 8, 128)),
                dict(q_weight=_bf(127)), dict(k_weight=torch.zeros(128)), dict(q_out=_bf(2, 8, 3, 128).half())):
        with pytest.raises(ValueError):
            api.qk_norm_rope(q, k, pos, inv, **bad)
    with pytest.raises(ValueError):  # shifted by one head: neither the same view nor apart
        api.qk_norm_rope(packed[:, :, :8], pk, pos, inv, q_out=packed[:, :, 1:9].transpose(1, 2))
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, k, pos[:1], inv)
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, k, pos, inv[:63])
    with pytest.raises(ValueError):
        api.qk_norm_rope(q, k[:, :2], pos, inv)
    with pytest.raises(TypeError):
        api.qk_norm_rope(q, k.half(), pos, inv)


def test_python_checks_cache_and_decode(fake):
    lens = [40, 1, 0]
    pages, table = paging.q4_store(lens, 2, 16, "cpu", spare_pages=2)
    assert pages.shape == (6, 2, 16, 160) and table.shape == (3, 3)
    assert table[2].tolist() == [-1, -1, -1] and table[1, 1] == -1
    used = table[table >= 0].tolist()
    assert len(set(used)) == len(used) == 4
    with pytest.raises(ValueError):
        paging.q4_store(lens, 2, 24, "cpu")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    k = _bf(3, 2, 5, 128)
    api.kv_write_paged_q4(k, k, pages, table, 16, i32(0, 0, 0), i32(5, 1, 0))
    a, b = api.kv_read_paged_q4(pages, table, 16, i32(0, 0, 0), None, 5)
    assert a.shape == b.shape == (3, 2, 5, 128)
    for bad in ((k, k[:, :, :4], pages, table, 16, i32(0, 0, 0)), (k, k, pages, table, 32, i32(0, 0, 0)),
                (k, k, pages, table[:2], 16, i32(0, 0, 0)), (k, k, pages, table, 16, i32(0, 0)),
                (k, k, pages[..., :159], table, 16, i32(0, 0, 0)), (k, k, pages, table, 16, i32(0, 0, 0), i32(1, 1))):
        with pytest.raises(ValueError):
            api.kv_write_paged_q4(*bad)
    with pytest.raises(TypeError):
        api.kv_read_paged_q4(pages, table, 16, i32(0, 0, 0), None, 5, torch.float32)
    with pytest.raises(ValueError):
        api.kv_read_paged_q4(pages, table, 16, i32(0, 0, 0), None, 5, k=_bf(3, 2, 4, 128))
    q, sl = _bf(3, 8, 128), i32(*lens)
    api.decode_anchor_paged_q4(q, pages, table, 16, sl, 40, 0.1, 2)
    idx, ik, hm = torch.zeros(3, 2, 7, dtype=torch.int32), torch.zeros(6, dtype=torch.int32), i32(0, 1)
    api.decode_reuse_paged_q4(q, pages, table, 16, sl, idx, ik, hm, 0.1, 2)
    with pytest.raises(ValueError):
        api.decode_anchor_paged_q4(q, pages, table, 16, sl[:2], 40, 0.1, 2)
    with pytest.raises(ValueError):
        api.decode_anchor_paged_q4(q, pages, table, 16, sl, 40, 0.1, 2, pooled=torch.zeros(3, 2, 39))
    with pytest.raises(TypeError):
        api.decode_anchor_paged_q4(q.float(), pages, table, 16, sl, 40, 0.1, 2)
    for bad in (dict(idx=idx[:2]), dict(ik=ik[:5]), dict(hm=hm[:1])):
        a = dict(idx=idx, ik=ik, hm=hm) | bad
        with pytest.raises(ValueError):
            api.decode_reuse_paged_q4(q, pages, table, 16, sl, a["idx"], a["ik"], a["hm"], 0.1, 2)


def test_schedule_passes_the_checks(fake):
    lens = [40, 1, 0]
    sch = PagedQ4DecodeSchedule(3, 8, 2, lens, (0,), 2, "cpu", torch.zeros(64))
    layers = []
    for l in range(2):
        qkv = _bf(3, 1, 12, 128)
        pages, table = paging.q4_store(lens, 2, 16, "cpu", seed=l)
        layers.append({"q": qkv[:, :, :8], "k": qkv[:, :, 8:10], "v": qkv[:, :, 10:], "kv_pages": pages,
                       "block_table": table, "q_weight": _bf(128)})
    sch.step(layers, {1: torch.zeros(2, dtype=torch.int32)}, [_bf(3, 8, 128), _bf(3, 8, 128)])
    assert sch.positions.tolist() == [39, 0, 0] and sch.count.tolist() == [1, 1, 0]


def test_cpu_tensors_are_refused():
    pages, table = paging.q4_store([4], 2, 16, "cpu")
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.qk_norm_rope(_bf(1, 1, 8, 128), _bf(1, 1, 2, 128), z, torch.zeros(64))
    with pytest.raises(ValueError):
        api.kv_write_paged_q4(_bf(1, 2, 1, 128), _bf(1, 2, 1, 128), pages, table, 16, z)
    with pytest.raises(ValueError):
        api.kv_read_paged_q4(pages, table, 16, z, None, 1)
    with pytest.raises(ValueError):
        api.decode_anchor_paged_q4(_bf(1, 8, 128), pages, table, 16, z, 4, 0.1, 2)

"""Host-side tests of the calls for the 4-bit cache, the many-token write and
the read-back that need no GPU: exports, geometry and the planner's choice, and
that validation answers before any CUDA call (the fake device addresses below
are never dereferenced)."""
import ctypes

import pytest

from gqa_decode_attention_sm_gb300 import _lib
from gqa_decode_attention_sm_gb300 import build as gbuild

OK, EINVAL, EDEV, EWS, EALIAS = 0, 1, 2, 3, 4
F16, BF16 = 0, 1
E2M1, I8, KV_BF16 = 4, 3, 1
Q, KV, LENS, OUT, WS, SC, BT = (0x10000000 * i for i in range(1, 8))


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


@pytest.mark.parametrize("B,C,want", [
    (1, 256, 1), (1, 512, 4), (1, 1024, 8), (1, 2048, 16), (1, 4096, 16), (1, 8192, 32), (1, 32768, 32),
    (4, 4096, 11), (8, 2048, 6), (32, 512, 1), (64, 32768, 8), (8, 131072, 57)])
def test_plan(lib, B, C, want):
    n = ctypes.c_int(0)
    assert lib.gqa_decode_plan_for(B, C, E2M1, 152, ctypes.byref(n)) == OK
    assert n.value == want


def test_geometry_and_launches(lib):
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    assert lib.gqa_decode_split_geometry(1000, 256, E2M1, ctypes.byref(a), ctypes.byref(b)) == OK
    assert (a.value, b.value) == (128, 8)  # 128-token tiles, as the 8-bit formats
    assert lib.gqa_decode_launch_count_for(1, 1024, E2M1, 1, 8, 152, ctypes.byref(a)) == OK and a.value == 1
    assert lib.gqa_decode_launch_count_for(64, 32768, E2M1, 3, 8, 152, ctypes.byref(a)) == OK and a.value == 2


def test_fp4_validation(lib):
    def call(**kw):
        a = dict(q=Q, kv=KV, sc=SC, lens=LENS, out=OUT, B=2, C=64, dt=BF16, qs=1.0, ks=1.0, vs=1.0, S=1, ws=WS, wsb=256)
        a.update(kw)
        return lib.gqa_decode_fp4kv(a["q"], a["kv"], a["sc"], a["lens"], a["out"], a["B"], a["C"], a["dt"], a["qs"],
                                    a["ks"], a["vs"], a["S"], a["ws"], a["wsb"], None)

    for kw in (dict(q=None), dict(kv=None), dict(sc=None), dict(lens=None), dict(out=None), dict(ws=None), dict(C=63),
               dict(sc=SC + 8), dict(kv=KV + 8), dict(dt=2), dict(qs=-1.0), dict(ks=0.0), dict(vs=float("nan")),
               dict(B=0), dict(S=257)):
        assert call(**kw) == EINVAL, kw
    assert call(S=4) == EWS
    assert call(out=SC + 64) == EALIAS and call(ws=KV) == EALIAS and call(out=KV + 4096) == EALIAS
    # the whole cache is 64 bytes a row: just behind it is free
    assert call(out=KV + 2 * 2 * 8 * 64 * 64, ws=None) == EINVAL
    f = lib.gqa_decode_split_stage
    assert f(Q, F16, KV, E2M1, LENS, OUT, 2, 64, 1.0, 1.0, 1.0, 1, WS, 256, None) == EINVAL
    v = lib.gqa_decode_verify
    assert v(Q, F16, KV, E2M1, None, LENS, OUT, 2, 64, 2, 1.0, 1.0, 1.0, 1, WS, 256, None) == EINVAL
    p = lib.gqa_decode_paged
    assert p(Q, F16, KV, E2M1, None, BT, 4, 16, 64, LENS, OUT, 2, 1, 1.0, 1.0, 1.0, 1, WS, 256, None) == EINVAL
    assert p(Q, F16, KV, E2M1, SC + 8, BT, 4, 16, 64, LENS, OUT, 2, 1, 1.0, 1.0, 1.0, 1, WS, 256, None) == EINVAL


P = [0x100000000 + i * 0x10000000 for i in range(16)]


def _write(lib, paged=False, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], qs=4096, ks=1024, vs=1024, qw=P[3], kw=P[4], dt=BF16, pos=P[5], sec=None, il=0,
             rows=P[6], slots=P[7], n=5, out=P[8], kv=P[9], fmt=KV_BF16, sc=None, B=2, C=64, eps=1e-6, th=1e6, k_=1.0,
             v_=1.0, ws=None, wsb=0, bt=P[10], maxp=4, nump=16, ps=64)
    a.update(kw)
    head = (a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["qw"], a["kw"], a["dt"], a["pos"],
            (ctypes.c_int * 3)(*a["sec"]) if a["sec"] else None, a["il"], a["rows"], a["slots"], a["n"], a["out"],
            a["kv"], a["fmt"], a["sc"])
    tail = (a["eps"], a["th"], a["k_"], a["v_"], a["ws"], a["wsb"], None)
    if paged:
        return lib.gqa_write_kv_paged(*head, a["bt"], a["B"], a["maxp"], a["nump"], a["ps"], *tail)
    return lib.gqa_write_kv(*head, a["B"], a["C"], *tail)


def test_write_validation(lib):
    assert _write(lib, n=0) == OK  # nothing to do, nothing looked at
    for kw in (dict(n=-1), dict(q=None), dict(pos=None), dict(rows=None), dict(slots=None), dict(out=None), dict(kv=None),
               dict(qw=None), dict(dt=3), dict(fmt=9), dict(fmt=0), dict(fmt=I8), dict(fmt=E2M1), dict(B=0), dict(C=0),
               dict(eps=-1.0), dict(th=0.5), dict(th=float("inf")), dict(k_=0.0), dict(v_=float("nan")),
               dict(q=P[0] + 8), dict(kv=P[9] + 2), dict(out=P[8] + 4), dict(qw=P[3] + 2), dict(pos=P[5] + 2),
               dict(qs=4088), dict(ks=1020), dict(vs=1028), dict(qs=-4096), dict(sec=(24, 20, 21)),
               dict(sec=(-2, 33, 33)), dict(sec=(20, 22, 22), il=1), dict(fmt=E2M1, sc=P[11], k_=1e-31),
               dict(fmt=E2M1, sc=P[11] + 1)):
        assert _write(lib, **kw) == EINVAL, kw
    assert _write(lib, ws=P[12], wsb=128) == EWS
    for kw in (dict(out=P[0]), dict(kv=P[1]), dict(out=P[9] + 4096), dict(out=P[3]), dict(kv=P[5] - 1024),
               dict(fmt=E2M1, sc=P[9] + 64), dict(fmt=E2M1, sc=P[2]), dict(ws=P[9], wsb=256), dict(out=P[7] - 512)):
        assert _write(lib, **kw) == EALIAS, kw
    # a strided projection reaches to its last token's heads, not further
    assert _write(lib, qs=6144, out=P[0] + 2 * (4 * 6144 + 4096)) != EALIAS
    assert _write(lib, qs=6144, out=P[0] + 2 * (4 * 6144 + 4088)) == EALIAS


def test_write_paged_validation(lib):
    for kw in (dict(bt=None), dict(bt=P[10] + 2), dict(ps=48), dict(ps=8), dict(ps=1 << 17), dict(maxp=0), dict(nump=0),
               dict(maxp=1 << 20, ps=2048), dict(rows=None), dict(B=0)):
        assert _write(lib, True, **kw) == EINVAL, kw
    assert _write(lib, True, out=P[10]) == EALIAS
    assert _write(lib, True, kv=P[10] - 4096) == EALIAS


def test_read_validation(lib):
    def call(paged=False, **kw):
        a = dict(kv=P[0], fmt=KV_BF16, sc=None, lens=P[1], st=None, out=P[2], dt=BF16, B=2, C=64, oc=64, k_=1.0, v_=1.0,
                 ws=None, wsb=0, bt=P[3], maxp=4, nump=16, ps=64)
        a.update(kw)
        if paged:
            return lib.gqa_read_kv_paged(a["kv"], a["fmt"], a["sc"], a["bt"], a["maxp"], a["nump"], a["ps"], a["lens"],
                                         a["st"], a["out"], a["dt"], a["B"], a["oc"], a["k_"], a["v_"], a["ws"],
                                         a["wsb"], None)
        return lib.gqa_read_kv(a["kv"], a["fmt"], a["sc"], a["lens"], a["st"], a["out"], a["dt"], a["B"], a["C"],
                               a["oc"], a["k_"], a["v_"], a["ws"], a["wsb"], None)

    for kw in (dict(kv=None), dict(lens=None), dict(out=None), dict(dt=2), dict(oc=0), dict(oc=(1 << 30) + 1),
               dict(fmt=5), dict(fmt=E2M1), dict(fmt=I8), dict(k_=-1.0), dict(B=70000), dict(C=0), dict(out=P[2] + 8),
               dict(kv=P[0] + 8), dict(lens=P[1] + 2), dict(st=P[4] + 1)):
        assert call(**kw) == EINVAL, kw
    assert call(ws=P[5], wsb=8) == EWS
    for kw in (dict(out=P[0]), dict(out=P[1] - 16), dict(st=P[2] + 64), dict(fmt=E2M1, sc=P[2]), dict(ws=P[2], wsb=256)):
        assert call(**kw) == EALIAS, kw
    assert call(True, out=P[3]) == EALIAS and call(True, ps=24) == EINVAL and call(True, bt=None) == EINVAL


def test_native_binding_judges_only_plain_arguments():
    import torch
    gbuild.build_native()
    from gqa_decode_attention_sm_gb300 import _native
    assert _native.torch_version == torch.__version__
    x = torch.zeros(2, 32, 128, dtype=torch.float16)
    for f, n in ((_native.write, 21), (_native.read, 12), (_native.attend, 13)):
        assert f(*[None] * n) is None and f() is None and f(*range(n)) is None
        assert f(1, True, *[x] * (n - 2)) is None       # CPU tensors are for the Python path to refuse
        assert f("address", *[x] * (n - 1)) is None

"""Decode attention over a 4-bit (e2m1) cache against its definition in 64 bits (GPU).

Every element of every output is compared with the formula evaluated in
float64 on the dequantised cache.  The bound, element by element:

  |got - ref| <= |ref| * eps(out) / 2  +  vmax * (2^-11 + N * 2^-25 + 2^-13)

eps(out) / 2 is the output's one rounding.  vmax is the largest |value| the
row can meet.  The softmax weights are rounded to fp16: half a step of a
normal one (2^-12 of it) in the numerator and in the denominator, together
2^-11 of vmax, and half a subnormal step (2^-25) for each of N tokens whose
weight is below 2^-14 (the denominator is at least about 1).  2^-13 covers
the scores: the FP32 dot product of 128 exact terms, its scaling, the maximum
taken off and ex2 are off by a few 2^-23 of the score's terms, below 2^-15 of
a weight at the magnitudes used here.
"""
import numpy as np
import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import _lib, api, inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
TD = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", params=["product", "checked"], autouse=True)
def library(request):
    """Every test runs on the product library and on the range-checked one."""
    from gqa_decode_attention_sm_gb300 import build as gbuild
    saved = _lib._lib
    _lib._lib = None
    if request.param == "checked":
        _lib._lib = _lib.load(gbuild.build_checked())
    else:
        gbuild.build()
        _lib.load()
    torch.cuda.init()
    yield request.param
    _lib._lib = saved


def definition(q, k, v, lens, q_scale=1.0):
    """q [B,T,32,128], k and v [B,8,C,128] in float64; [B,T,32,128]."""
    B, T = q.shape[:2]
    out = torch.zeros_like(q)
    for b in range(B):
        for j in range(T):
            n = min(int(lens[b]), k.shape[2]) - T + 1 + j
            if n < 1:
                continue
            s = torch.einsum("ghd,gtd->ght", q[b, j].view(8, 4, 128), k[b, :, :n]) * (q_scale / 128 ** 0.5)
            out[b, j] = torch.einsum("ght,gtd->ghd", torch.softmax(s, -1), v[b, :, :n]).reshape(32, 128)
    return out


def reference(t, q_scale=None):
    q = t["q"].double()
    q = q[:, None] if q.dim() == 3 else q
    k, v = (inputs.dequantise_e2m1(t["kv"][:, p], t["kv_scales"][:, p], s)
            for p, s in ((0, t["k_scale"]), (1, t["v_scale"])))
    # scales past the length are NaN on purpose: never part of the definition
    return definition(q, k, v, t["lens"].tolist(), t["q_scale"] if q_scale is None else q_scale).view(t["q"].shape)


def vmax(t):
    v = inputs.dequantise_e2m1(t["kv"][:, 1], t["kv_scales"][:, 1], t["v_scale"])
    return float(torch.nan_to_num(v, nan=0.0).abs().max())


def assert_close(out, t, ref=None):
    ref = reference(t) if ref is None else ref
    n = max(1, int(t["lens"].max()))
    err = (out.double() - ref).abs()
    bound = ref.abs() * (torch.finfo(out.dtype).eps / 2) + vmax(t) * (2 ** -11 + n * 2 ** -25 + 2 ** -13)
    assert torch.isfinite(out).all()
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3f} of the bound, err {float(err.max()):.3e}"
    # and together: a lost token or a wrong scale is far above the roundings
    assert float(err.square().mean().sqrt()) <= 0.02 * float(ref.square().mean().sqrt()) + 1e-12


def decode(t, num_splits=None, paged=0, ws=None, out=None):
    """One call; the way in depends on the shape (prepared, verify window or paged)."""
    q, T = t["q"], 1 if t["q"].dim() == 3 else t["q"].shape[1]
    B, C = q.shape[0], t["kv"].shape[3]
    sc = dict(k_scale=t["k_scale"], v_scale=t["v_scale"])
    S = num_splits or gq.plan(B, C, api.KV_E2M1)
    ws = torch.zeros(gq.workspace_size(B * T, C, S), dtype=torch.uint8, device=DEV) if ws is None else ws
    if paged:
        p = inputs.paginate(t, paged, extra_pages=2)
        out = gq.gqa_decode_paged(q, p["kv_pages"], p["block_table"], t["lens"], q_scale=t["q_scale"], num_splits=S,
                                  workspace=ws, kv_scales=p["kv_scale_pages"], out=out, **sc)
    elif T == 1:
        p = gq.prepare({"Q": q, "KV": t["kv"], "O": torch.empty_like(q) if out is None else out,
                        "sequence_lengths": t["lens"], "KV_SCALES": t["kv_scales"]}, q_scale=t["q_scale"],
                       num_splits=S, workspace=ws, **sc)
        out = gq.launch(p)
    else:
        out = gq.gqa_decode_verify(q, t["kv"], t["lens"], q_scale=t["q_scale"], kv_scales=t["kv_scales"],
                                   num_splits=S, workspace=ws, out=out, **sc)
    flags = gq.get_status(ws)
    assert not flags & (api.FLAG_BOUNDS | api.FLAG_WAIT_TIMEOUT), hex(flags)
    return out, flags


def make(B, C, lens, dtype="bf16", T=1, seed=5, **kw):
    w = inputs.custom(B, C, 1, kv_dtype="e2m1", q_dtype=dtype, nan_tail=True, q_len=T, **kw)
    return inputs.make(w, DEV, seed=seed, lens=lens)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("C,lens", [(2, [2, 1]), (64, [64, 5]), (130, [129, 130]), (1000, [999, 17]),
                                    (4096, [4096, 2049])])
def test_matches_the_definition(dtype, T, C, lens):
    t = make(2, C, [max(T, n) if C >= T else n for n in lens], dtype, T)
    out, flags = decode(t)
    assert_close(out, t)
    assert bool(flags & api.FLAG_LENGTH_CLAMPED) == bool((t["lens"] < T).any())


@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("grid,B,C,S", [("one piece and combine", 2, 2048, 16), ("cluster", 2, 1024, 4),
                                        ("balanced", 96, 1024, 4), ("one split", 3, 512, 1)])
@pytest.mark.parametrize("page", [0, 16, 256])
def test_every_grid_ragged(T, grid, B, C, S, page):
    rng = np.random.default_rng(B * 1000 + C + T + page)
    lens = rng.integers(0, C + 1, B)
    lens[0], lens[-1] = 0, C
    if B > 2:
        lens[1] = 1
    t = make(B, C, lens, "f16" if T % 2 else "bf16", T)
    out, flags = decode(t, S, page)
    assert_close(out, t)
    assert (out[0] == 0).all() and flags & api.FLAG_LENGTH_CLAMPED
    assert not flags & api.FLAG_PAGE_CLAMPED


def test_odd_pages_end_inside_a_tile_and_a_scale_pair():
    # an odd length in every page of 16 takes the scale that is loaded alone
    t = make(16, 256, list(range(1, 17)), "bf16", 1)
    assert_close(decode(t, 2, 16)[0], t)
    t = make(16, 256, [241 + i for i in range(16)][:15] + [255], "f16", 2)
    assert_close(decode(t, 2, 16)[0], t)


def test_planned_batch_long_rows():
    t = make(8, 16384, [16384, 16383, 8193, 1, 4097, 12345, 127, 129], "bf16", 1)
    assert_close(decode(t)[0], t)


@pytest.mark.parametrize("q_mag", [1e-7, 1e-2, 30.0, 1e5])
def test_any_magnitude_of_q(q_mag):
    # bf16 q is scaled by a power of two on its way to fp16; large scores make the softmax one-hot
    t = make(2, 300, [300, 7], "bf16", 1)
    t["q"] = (t["q"].float() * q_mag).to(torch.bfloat16)
    t["q_scale"] = min(1.0, 10.0 / q_mag)
    assert_close(decode(t)[0], t)


def test_every_code_and_every_scale():
    # all 16 codes and the e4m3 scales from the smallest subnormal to 448 meet in K and V
    g = torch.Generator(device=DEV).manual_seed(3)
    C = 512
    t = make(1, C, [C], "f16", 1)
    t["kv"] = torch.randint(0, 256, t["kv"].shape, generator=g, device=DEV, dtype=torch.int64).to(torch.uint8)
    t["kv_scales"] = torch.randint(0, 0x7F, t["kv_scales"].shape, generator=g, device=DEV).to(torch.uint8)
    t["k_scale"], t["v_scale"] = 2.0 ** -9, 3.0
    assert_close(decode(t)[0], t)
    t["kv_scales"][:] = 1  # 2^-9 everywhere
    t["k_scale"] = 1.0
    assert_close(decode(t)[0], t)
    # negative scales are numbers like the others
    t["kv_scales"] = torch.randint(0x81, 0xFE, t["kv_scales"].shape, generator=g, device=DEV).to(torch.uint8)
    t["k_scale"] = 2.0 ** -9
    assert_close(decode(t)[0], t)


def test_scales_join_once():
    # k_scale on the scores and v_scale on the output: powers of two move between
    # the tensor scale, the group scales and q_scale without changing a bit
    t = make(2, 700, [700, 333], "f16", 1)
    out = decode(t, 4)[0].clone()
    u = dict(t, k_scale=t["k_scale"] * 4, q_scale=0.25)
    assert torch.equal(decode(u, 4)[0], out)
    u = dict(t, v_scale=t["v_scale"] * 2)
    twice, got = 2 * out.float(), decode(u, 4)[0].float()
    # an fp16 output below 2^-14 is subnormal: x and 2x then round on the same
    # grid (step 2^-24), so 2 * round(x) is off by at most 2 * 2^-25 and
    # round(2x) by 2^-25; every normal output doubles exactly
    normal = out.float().abs() >= 2 ** -14
    assert torch.equal(got[normal], twice[normal])
    assert (got - twice)[~normal].abs().le(2 ** -24 + 2 ** -25).all()


def test_fp4kv_entry_and_float8_scales():
    t = make(3, 640, [640, 1, 77], "bf16", 1)
    ref = decode(t)[0]
    out = gq.gqa_decode_fp4kv(t["q"], t["kv"], t["kv_scales"].view(torch.float8_e4m3fn), t["lens"], t["k_scale"],
                              t["v_scale"])
    assert torch.equal(out, ref)


def test_runs_are_bitwise_alike_and_capturable():
    t = make(20, 2048, list(range(100, 2100, 97))[:20], "bf16", 1)
    p = gq.prepare({"Q": t["q"], "KV": t["kv"], "O": torch.empty_like(t["q"]), "sequence_lengths": t["lens"],
                    "KV_SCALES": t["kv_scales"]}, k_scale=t["k_scale"], v_scale=t["v_scale"])
    first = gq.launch(p).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gq.launch(p)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(p.out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq.launch(p)
    p.out.zero_()
    graph.replay()
    assert torch.equal(p.out, first)
    t["lens"].fill_(50)  # the lengths are read when the graph runs
    graph.replay()
    assert_close(p.out, t)


def test_bad_pages_are_clamped_and_flagged():
    t = make(2, 128, [128, 128], "bf16", 1)
    p = inputs.paginate(t, 64)
    table = p["block_table"].clone()
    table[1, 1] = 10 ** 6
    S = 1
    ws = torch.zeros(gq.workspace_size(2, 128, S), dtype=torch.uint8, device=DEV)
    out = gq.gqa_decode_paged(t["q"], p["kv_pages"], table, t["lens"], k_scale=t["k_scale"], v_scale=t["v_scale"],
                              num_splits=S, workspace=ws, kv_scales=p["kv_scale_pages"])
    flags = gq.get_status(ws)
    assert flags & api.FLAG_PAGE_CLAMPED and not flags & api.FLAG_BOUNDS
    assert_close(out[:1], {**t, "q": t["q"][:1], "kv": t["kv"][:1], "kv_scales": t["kv_scales"][:1],
                           "lens": t["lens"][:1]})


def test_unused_slots_and_neighbours_change_nothing():
    t = make(2, 512, [300, 511], "bf16", 1)
    out = decode(t, 4)[0].clone()
    for b, L in enumerate((300, 511)):
        t["kv"][b, :, :, L:] = 0x35
        t["kv_scales"][b, :, :, L:] = 0x78
    assert torch.equal(decode(t, 4)[0], out)


def test_refusals():
    t = make(2, 64, [64, 64], "bf16", 1)
    good = dict(q=t["q"], kv=t["kv"], kv_scales=t["kv_scales"], sequence_lengths=t["lens"])

    def call(**kw):
        a = {**good, **kw}
        return gq.gqa_decode_fp4kv(a.pop("q"), a.pop("kv"), a.pop("kv_scales"), a.pop("sequence_lengths"), **a)

    for kw in (dict(kv=t["kv"].view(torch.int8)), dict(kv=t["kv"][..., :32]), dict(kv_scales=t["kv_scales"][..., :4]),
               dict(kv_scales=t["kv_scales"].to(torch.bfloat16)), dict(kv_scales=t["kv_scales"].cpu()),
               dict(q=t["q"].float()), dict(kv=t["kv"].transpose(1, 2)), dict(out=t["q"].half())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(kv_scales=None)
    with pytest.raises(gq.GqaError, match="k_scale"):
        call(k_scale=0.0)
    with pytest.raises(gq.GqaError, match="multiple of 2"):
        call(kv=t["kv"][:, :, :, :63].contiguous(), kv_scales=t["kv_scales"][:, :, :, :63].contiguous())
    with pytest.raises(gq.GqaError, match="overlaps"):
        call(out=t["q"])
    p = gq.prepare({"Q": t["q"], "KV": t["kv"], "O": torch.empty_like(t["q"]), "sequence_lengths": t["lens"],
                    "KV_SCALES": t["kv_scales"]}, k_scale=1.0, v_scale=1.0)
    with pytest.raises(gq.GqaError, match="gqa_decode_fp4kv"):
        gq.split_stage(p)
    with pytest.raises((ValueError, gq.GqaError)):
        gq.gqa_decode_fp8kv(t["q"], t["kv"], t["lens"], 1.0, 1.0)


@pytest.mark.parametrize("T,page", [(1, 0), (3, 0), (1, 32), (2, 32)])
def test_the_native_binding_and_the_interpreted_one_are_alike(T, page, monkeypatch):
    assert api._native is not None, "the native binding is not built"
    t = make(3, 256, [256, 100, T], "bf16", T)
    native = decode(t, 4, page)[0]
    calls = []
    real = api._native
    monkeypatch.setattr(api, "_native", type("Spy", (), {"attend": lambda self, *a: calls.append(real.attend(*a)) or calls[-1]})())
    out = torch.empty_like(t["q"])
    assert torch.equal(decode(t, 4, page, out=out)[0], native)
    assert len(calls) == 1 and calls[0] is out  # with everything given, the native call is the one that runs
    monkeypatch.setattr(api, "_native", None)
    assert torch.equal(decode(t, 4, page)[0], native)

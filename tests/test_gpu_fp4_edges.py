"""Decode over a 4-bit cache where the softmax is far from even (GPU)."""
import math

import numpy as np
import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import api, inputs
from test_gpu_fp4 import DEV, assert_close, decode, library, make, reference  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,B,lens,S", [(1, 1, [8192], None), (1, 2, [8192, 8191], 1), (3, 2, [4096, 4001], 8),
                                        (4, 1, [2048], None), (2, 1, [8000], 3), (1, 40, [2048] * 40, 4)])
@pytest.mark.parametrize("nats", [8.0, 12.0, 16.0, 17.5, 19.0, 20.0])
def test_a_sink_takes_nothing_from_the_others(T, B, lens, S, nats):
    """One key far above the others, its value row 0: what is left is the sum of many small weights.  Each is
    rounded to fp16 once (2^-12 of it: at 2^15 of the largest it is a normal number down to 20 nats), all values
    are positive, so the whole is off by no more than that share; the scores' FP32 error (2^-20 at 20 nats of 128
    exact terms) and the output's rounding join it."""
    t = make(B, lens[0], lens, "f16", T, seed=50)
    t["kv_scales"][:, 0] = 0x08  # 2^-6
    t["kv_scales"][:, 1] = 0x38  # 1
    t["kv"][:, 1] &= 0x77        # no signs
    t["kv"][:, 0, :, 0] = 0x77   # the sink: 6 everywhere, scale 1
    t["kv_scales"][:, 0, :, 0] = 0x38
    t["kv"][:, 1, :, 0] = 0
    t["q"] = torch.ones_like(t["q"])
    t["k_scale"], t["v_scale"], t["q_scale"] = nats / (768 / math.sqrt(128)), 512.0 * math.exp(max(0, nats - 12)), 1.0
    out = decode(t, S)[0].double()
    ref = reference(t)
    assert (ref > 0).float().mean() > 0.99
    worst = ((out - ref).abs() / ref.clamp(min=1e-30)).max()
    assert worst <= 2 ** -11 + 2 ** -12 + 2 ** -14, float(worst)


@pytest.mark.parametrize("q_scale", [1e3, 1e6, 1e9, 1e12])
@pytest.mark.parametrize("T,lens,S", [(1, [1024], 1), (1, [1000, 513], 4), (3, [900, 1024], 2), (1, [1024] * 60, 4)])
def test_scores_past_the_range_of_float_differences(q_scale, T, lens, S):
    # the largest score is above the next by far more than its own rounding: one value row is the output
    t = make(len(lens), 1024, lens, "f16", T, seed=51)
    t["q_scale"] = q_scale
    ref = reference(t)
    assert_close(decode(t, S)[0], t, ref)


def test_a_draft_of_nan_reaches_only_the_queries_that_see_it():
    for T, page in ((2, 0), (3, 0), (4, 0), (3, 16)):
        t = make(2, 512, [300, 257], "bf16", T, seed=52)
        clean = decode(t, 2, page)[0].clone()
        for b, L in enumerate((300, 257)):
            t["kv_scales"][b, 1, 2, L - 1, 3] = 0x7F  # the last draft's value, dims 48 .. 63 of KV head 2
        out = decode(t, 2, page)[0]
        assert torch.equal(out[:, :-1], clean[:, :-1])
        last = torch.isnan(out[:, -1]).view(2, 8, 4, 8, 16)
        assert last[:, 2, :, 3].all()
        last[:, 2, :, 3] = False
        assert not last.any()
        # and in a key: the whole head of the queries that see it
        t = make(2, 512, [300, 257], "bf16", T, seed=52)
        for b, L in enumerate((300, 257)):
            t["kv_scales"][b, 0, 5, L - 2, 0] = 0x7F
        out = decode(t, 2, page)[0]
        assert torch.equal(out[:, :T - 2], clean[:, :T - 2])
        seen = torch.isnan(out[:, T - 2:]).view(2, -1, 8, 4, 128)
        assert seen[:, :, 5].all() and not seen[:, :, [0, 1, 2, 3, 4, 6, 7]].any()


@pytest.mark.parametrize("seed", range(20))
def test_random_scales_spreads_and_nan_drafts(seed):
    """Random codes and scales (of both signs, up to the whole e4m3 range), scores spread over 0.01 to 1e5, ragged and
    empty rows, windows, pages, splits; NaN scales behind the lengths and in drafts.  Element by element:
      |got - ref| <= |ref| eps / 2 + A (2^-11 + 2^-13 + 2 (e^d - 1)) + vmax N 2^-40
    A = sum p |v|: weights are rounded by 2^-12 of themselves (the denominator not), 2^-40 of the largest where they
    are subnormal; d = 2^-21 sum |q k|, the error of an FP32 score of 128 exact terms, its scaling and the maximum."""
    rng, g = np.random.default_rng(seed), torch.Generator(device=DEV).manual_seed(seed)
    dtype = [torch.float16, torch.bfloat16][rng.integers(2)]
    B, T, page = int(rng.choice([1, 2, 3, 5, 40])), int(rng.integers(1, 5)), int(rng.choice([0, 0, 16, 64]))
    C = int(np.exp(rng.uniform(np.log(2), np.log(4000 if B < 10 else 800))))
    C = -(-C // (page or 2)) * (page or 2)
    table = None
    if page:
        table = torch.randperm(B * C // page, generator=g, device=DEV).to(torch.int32).view(B, C // page).contiguous()
    units, rows = (B * C // page, page) if page else (B, C)
    kv = torch.randint(0, 256, (units, 2, 8, rows, 64), generator=g, device=DEV, dtype=torch.int64).to(torch.uint8)
    lo = int(rng.integers(0, 0x60))
    sc = torch.randint(lo, int(rng.integers(lo + 1, 0x7F)), (units, 2, 8, rows, 8), generator=g, device=DEV).to(torch.uint8)
    if rng.random() < 0.3:
        sc |= (torch.rand(sc.shape, generator=g, device=DEV) < 0.3).to(torch.uint8) * 0x80
    lens = torch.tensor(rng.integers(0, C + 1, B), dtype=torch.int32, device=DEV)
    lens[0] = C
    x = torch.stack([inputs.dequantise_e2m1(kv[:, p], sc[:, p], 1.0) for p in (0, 1)], 1)
    x = x if table is None else x[table.long()].movedim(1, 3).flatten(3, 4)
    q = (torch.randn((B, T, 32, 128), generator=g, device=DEV) * 2.0 ** float(rng.uniform(-8, 4))).to(dtype)
    size = float((x[:, 0].abs().mean() * q.double().abs().mean()).clamp(min=1e-30))
    ks = float(np.float32(2.0 ** float(rng.uniform(-20, 20))))
    qs = float(np.float32(10 ** float(rng.uniform(-2, 5)) / size / ks))
    vs = float(np.float32(min(2.0 ** float(rng.uniform(-20, 10)), 3e4 / float(x[:, 1].abs().max()))))
    drafts = []
    if not page:
        for b in range(B):
            L = int(lens[b])
            sc[b, :, :, L:] = 0x7F
            if L > T and rng.random() < 0.4:
                drafts.append((b, L - 1 - int(rng.integers(0, T)), int(rng.integers(8)), int(rng.integers(8))))
                sc[b, 1, drafts[-1][2], drafts[-1][1], drafts[-1][3]] = 0x7F
    S = int(rng.choice([1, 2, 3, 5, 8, 16]))
    ws = torch.zeros(gq.workspace_size(B * T, C, S), dtype=torch.uint8, device=DEV)
    how = dict(k_scale=ks, v_scale=vs, q_scale=qs, num_splits=S, workspace=ws, kv_scales=sc)
    out = gq.gqa_decode_paged(q, kv, table, lens, **how) if page else gq.gqa_decode_verify(q, kv, lens, **how)
    assert not gq.get_status(ws) & (api.FLAG_BOUNDS | api.FLAG_WAIT_TIMEOUT)
    for b in range(B):
        for j in range(T):
            L, got = int(lens[b]) - T + 1 + j, out[b, j].double().view(8, 4, 128)
            if L < 1:
                assert not got.any()
                continue
            qq, K, V = q[b, j].double().view(8, 4, 128), x[b, 0, :, :L] * ks, x[b, 1, :, :L] * vs
            p = torch.softmax(torch.einsum("ghd,gtd->ght", qq, K) * (qs / math.sqrt(128)), -1)
            d = torch.einsum("ghd,gtd->ght", qq.abs(), K.abs()).amax(-1, keepdim=True) * (qs / math.sqrt(128) * 2 ** -21)
            ref, A = torch.einsum("ght,gtd->ghd", p, V), torch.einsum("ght,gtd->ghd", p, V.abs())
            bound = (ref.abs() * (torch.finfo(dtype).eps / 2) + A * (2 ** -11 + 2 ** -13 + 2 * torch.expm1(d.clamp(max=5)))
                     + V.abs().amax(1)[:, None] * (L * 2 ** -40) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps)
            seen = torch.zeros_like(got, dtype=torch.bool)  # dims that a NaN reaches
            for _, slot, head, group in (n for n in drafts if n[0] == b and n[1] < L):
                seen[head, :, 16 * group:16 * group + 16] = True
            assert torch.isnan(got[seen]).all()
            assert ((got - ref).abs() <= bound)[~seen].all()

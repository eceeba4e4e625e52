"""Decode over a 4-bit cache where the softmax is far from even (GPU)."""
import math

import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import api, inputs
from test_gpu_fp4 import DEV, TD, assert_close, decode, library, make, reference

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

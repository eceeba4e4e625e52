"""Decode over a 4-bit cache where the softmax is far from even (GPU)."""
import math

import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import api, inputs
from test_gpu_fp4 import DEV, TD, assert_close, decode, library, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_scale", [1e3, 1e6, 1e9, 1e12])
@pytest.mark.parametrize("T,lens,S", [(1, [1024], 1), (1, [1000, 513], 4), (3, [900, 1024], 2), (1, [1024] * 60, 4)])
def test_scores_past_the_range_of_float_differences(q_scale, T, lens, S):
    # the largest score is above the next by far more than its own rounding: one value row is the output
    t = make(len(lens), 1024, lens, "f16", T, seed=51)
    t["q_scale"] = q_scale
    ref = reference(t)
    assert_close(decode(t, S)[0], t, ref)

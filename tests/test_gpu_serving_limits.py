"""The serving calls at the limits of what they take: values and scales that a query
does not see, infinite scores, weights of every kind, calls without a token (GPU).

Bounds as in test_gpu_serving.py, with what each test says of its own.
"""
import math

import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from test_gpu_serving import (D, DEV, HKV, HQ, TD, attend64, gen, kept64, library, new_cache,  # noqa: F401
                              paged, values)

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# ----------------------------------------- prompt attention: int8 scales apart


def int8_rows(q, K, V, sc, end, dtype):
    """(reference, bound) of one query token over int8 slots [0, end).

    A weight meets V times its V scale in fp16, and the running maximum counts the
    power of two above the largest V scale s that the query sees (2^-61 at least): the
    largest weight is held at 2^7 / (2 s) or more, and what lies on fp16's grid of 2^-24
    is off by 2^-25, so an output by 2^-25 * 2 s / 2^7 = 2^-31 s for each |code|."""
    half = torch.finfo(TD[dtype]).eps / 2
    ref, a, e = attend64(q, K, V, end)
    s = max(float(sc[:, :end].double().abs().max()), 2.0 ** -61)
    codes = torch.where(sc[:, :end] == 0, 127.0, (V[:, :end].abs().amax(-1) / sc[:, :end].double().abs())).sum(1).max()
    return ref, half * ref.abs() + (half + 2 * e + 2 ** -18) * a + torch.finfo(TD[dtype]).tiny * half + 2 ** -31 * s * float(codes)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("n,L", [(70, 300), (3, 128), (129, 257), (40, 20000)])
def test_prefill_hidden_int8_scales(library, n, L, page, dtype):  # noqa: F811
    """A V scale (or a K scale) of a token that a query does not see never reaches it,
    whatever it is: infinite, NaN, or 2^30 or 2^100 times the others'."""
    C = -(-L // 64) * 64
    for what in (INF, -INF, NAN, 2.0 ** 30, 2.0 ** 100):
        kv, sc = new_cache("i8", 1, C, 3)
        at = sorted({max(L - n + k, 1) for k in (1, n // 3, n // 2, n - 2, n - 1)})
        sc[0, 1, :, at] = what
        if not 1 < abs(what) < INF:
            sc[0, 0, 5, at] = what  # one head's keys too
        sc[0, :, :, L:] = NAN
        K, V = (values(kv[0, p], sc[0, p], "i8", 1.0) for p in (0, 1))
        q = torch.randn((n, HQ, D), generator=gen(4), device=DEV).to(TD[dtype])
        starts, lens = torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV)
        if page:
            pool, psc, table = paged(kv, sc, page, 1, C)
            out = gq.gqa_prefill_paged(q, pool, table, starts, lens, kv_scales=psc)
        else:
            out = gq.gqa_prefill(q, kv, starts, lens, kv_scales=sc)
        for j in sorted({0, *(t + d - (L - n) for t in at for d in (-1, 0)), n - 1}):
            if not 0 <= j < n:
                continue
            end = L - n + j + 1
            if any(t < end for t in at) and not math.isfinite(what):
                assert not torch.isfinite(out[j].float()).any(), f"{what}: query {j} does not see its own scale"
                continue
            if any(t < end for t in at) and what == 2.0 ** 100 and dtype == "f16":
                continue  # past fp16's largest number
            ref, bound = int8_rows(q[j], K, V, sc[0, 1], end, dtype)
            if not float(ref.abs().max()) < torch.finfo(TD[dtype]).max / 2:
                continue
            err = (out[j].double() - ref).abs()
            assert (err <= bound).all(), f"{what}: query {j}, worst {float((err / bound).max()):.3f} of the bound"

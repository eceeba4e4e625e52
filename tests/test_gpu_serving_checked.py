"""The serving kernels' own range checks (GPU): with the extents they compare against cut
short every call reports it, and with the true ones none does.

Every access of a call whose checks fire is redirected into its real buffers, so
nothing leaves them; that call's outputs are not looked at.
"""
import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import _lib, api
from test_gpu_serving import D, DEV, HKV, HQ, TD, draft_inputs, gen, new_cache, paged, scale_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def checked():
    from gqa_decode_attention_sm_gb300 import build as gbuild
    saved = _lib._lib
    _lib._lib = None
    _lib._lib = _lib.load(gbuild.build_checked())
    yield _lib._lib
    _lib._lib = saved


def zeros(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype, device=DEV)


def prefill(s, page):
    out, ws = torch.zeros_like(s["q"]), zeros(gq.prefill_workspace_size())
    how = dict(k_scale=s["ks"], v_scale=s["vs"], out=out, workspace=ws)
    if page:
        gq.gqa_prefill_paged(s["q"], s["pool"], s["table"], s["starts"], s["lens"], kv_scales=s["psc"], **how)
    else:
        gq.gqa_prefill(s["q"], s["kv"], s["starts"], s["lens"], kv_scales=s["sc"], **how)
    return ws, [out]


def weights(s, page):
    B, C = s["kv"].shape[0], s["kv"].shape[3]
    ws, w = zeros(gq.weights_workspace_size(B, C, 2)), zeros(B, HKV, C, dtype=torch.float32)
    q = s["q"][:2 * B].view(B, 2, HQ, D)
    how = dict(k_scale=s["ks"], workspace=ws)
    if page:
        gq.accumulate_weights_paged(q, s["pool"], s["table"], s["lens"], w, kv_scales=s["psc"], **how)
    else:
        gq.accumulate_weights(q, s["kv"], s["lens"], w, kv_scales=s["sc"], **how)
    return ws, [w]


def evict(s, page):
    B, C = s["kv"].shape[0], s["kv"].shape[3]
    keep = C // 3
    ws, w = zeros(gq.evict_workspace_size(B, keep)), s["w"].clone()
    lens, kept = s["lens"].clone(), zeros(B, HKV, keep, dtype=torch.int32)
    if page:  # in place
        pool, psc = s["pool"].clone(), None if s["psc"] is None else s["psc"].clone()
        gq.evict_kv_paged(pool, s["table"], lens, w, keep, 9, 4, kept=kept, kv_scales=psc, workspace=ws)
        return ws, [pool.view(torch.uint8), lens, w, kept]
    out, osc = new_cache(s["fmt"], B, keep + 5, 70)
    ow, ol = zeros(B, HKV, keep + 1, dtype=torch.float32), zeros(B, dtype=torch.int32)
    gq.evict_kv(s["kv"], lens, w, keep, 9, 4, out=out, out_scales=osc, out_lengths=ol, out_weights=ow, kept=kept,
                kv_scales=s["sc"], workspace=ws)
    return ws, [out.view(torch.uint8), ol, ow, kept]


@pytest.mark.parametrize("C", [640, 20480])  # weights on chip and in two launches, both kernels that choose
@pytest.mark.parametrize("call", [prefill, weights, evict])
@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8", "e2m1"])
def test_cut_extents_make_the_checks_fire(checked, fmt, page, call, C):
    B = 2
    kv, sc = new_cache(fmt, B, C, 71)
    s = dict(fmt=fmt, kv=kv, sc=sc, lens=torch.tensor([C - 7, C], dtype=torch.int32, device=DEV))
    s["ks"], s["vs"] = scale_of(fmt)
    s["q"] = torch.randn((90, HQ, D), generator=gen(72), device=DEV).to(TD["bf16"])
    s["starts"] = torch.tensor([0, 20, 90], dtype=torch.int32, device=DEV)
    s["w"] = torch.rand((B, HKV, C), generator=gen(73), device=DEV)
    if page:
        s["pool"], s["psc"], s["table"] = paged(kv, sc, page, B, C, 74)
    ws, first = call(s, page)
    assert gq.get_status(ws) == 0
    cache, scales = (s["pool"], s["psc"]) if page else (kv, sc)
    cuts = [(cache.numel() * cache.element_size() // 2, 0)]
    if scales is not None:
        cuts.append((0, scales.numel() * scales.element_size() // 2))
    for cut in cuts:
        try:
            assert checked.gqa_decode_debug_cut_extents(*cut) == 0
            ws, _ = call(s, page)
            torch.cuda.synchronize()
        finally:
            assert checked.gqa_decode_debug_cut_extents(0, 0) == 0
        flags = gq.get_status(ws)
        assert flags == api.FLAG_BOUNDS, hex(flags)
    ws, again = call(s, page)
    assert gq.get_status(ws) == 0
    for a, b in zip(first, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (3, 4, 1001), (65, 32, 70), (2, 3, 200003)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_stay_in_bounds(checked, B, T, V, dtype):
    p, d, u, q, lens = draft_inputs(B, T, V, dtype, seed=75)
    for probs in (q, None):
        ws = zeros(256)
        gq.verify_drafts(p, d, u, draft_probs=probs, sequence_lengths=lens.clone(), workspace=ws)
        assert gq.get_status(ws) == 0

"""Validation, sizes and exports of the serving calls (CPU: every call below is refused
before any CUDA call)."""
import ctypes

import pytest

from gqa_decode_attention_sm_gb300 import _lib, api
from gqa_decode_attention_sm_gb300 import build as gbuild


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return _lib.load()


# made-up addresses, far from one another; no call gets as far as using one
A = [(k + 1) << 40 for k in range(16)]
OK, INVALID, SMALL, ALIAS = 0, 1, 3, 4
BF16, F16 = 1, 0


def prefill(lib, **change):
    a = dict(q=A[0], dtype=BF16, kv=A[1], fmt=1, scales=None, starts=A[2], lens=A[3], out=A[4], tokens=8, batch=2,
             capacity=64, q_scale=1.0, k_scale=1.0, v_scale=1.0, ws=A[5], ws_bytes=1 << 30, stream=None)
    a.update(change)
    return lib.gqa_prefill(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), INVALID), (dict(tokens=(1 << 27) + 1), INVALID), (dict(starts=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(kv=None), INVALID),
    (dict(batch=0), INVALID), (dict(batch=65536), INVALID), (dict(capacity=0), INVALID), (dict(dtype=2), INVALID),
    (dict(fmt=0), INVALID), (dict(fmt=5), INVALID), (dict(fmt=3), INVALID), (dict(fmt=4, scales=A[6] + 4), INVALID),
    (dict(q=A[0] + 8), INVALID), (dict(out=A[4] + 2), INVALID), (dict(lens=A[3] + 1), INVALID),
    (dict(q_scale=-1.0), INVALID), (dict(q_scale=float("inf")), INVALID), (dict(k_scale=0.0), INVALID),
    (dict(v_scale=float("nan")), INVALID), (dict(ws=None), INVALID), (dict(ws=A[5] + 8), INVALID),
    (dict(ws_bytes=4096), SMALL), (dict(out=A[0]), ALIAS), (dict(out=A[1] + 1024), ALIAS), (dict(ws=A[1]), ALIAS),
    (dict(ws=A[4]), ALIAS), (dict(capacity=1 << 30, batch=64), INVALID)])
def test_prefill_validation(lib, change, status):
    assert prefill(lib, **change) == status


def test_prefill_nothing_to_do(lib):
    assert prefill(lib, tokens=0, q=None, out=None) == OK


@pytest.mark.parametrize("page,pages,per", [(8, 4, 4), (48, 4, 4), (131072, 4, 4), (16, 0, 4), (16, 4, 0), (65536, 4, 1 << 20)])
def test_paged_geometry(lib, page, pages, per):
    assert lib.gqa_prefill_paged(A[0], BF16, A[1], 1, None, A[6], per, pages, page, A[2], A[3], A[4], 8, 2, 1.0, 1.0, 1.0,
                                 A[5], 1 << 30, None) == INVALID
    assert lib.gqa_accumulate_weights_paged(A[0], BF16, A[1], 1, None, A[6], per, pages, page, A[3], A[4], 2, 1, 1.0, 1.0, 1,
                                            A[5], 1 << 30, None) == INVALID
    assert lib.gqa_evict_kv_paged(A[1], 1, None, A[6], per, pages, page, A[3], A[4], None, 0, None, None, A[7], 2, 0, 16, 0,
                                  0, A[5], 1 << 30, None) == INVALID


def drafts(lib, **change):
    a = dict(probs=A[0], pb=400, pt=100, dprobs=A[1], db=300, dt=100, type=2, drafts=A[2], u=A[3], lens=A[4], out_lens=A[5],
             tokens=A[6], accepted=A[7], batch=2, window=4, vocab=100, ws=None, ws_bytes=0, stream=None)
    a.update(change)
    return lib.gqa_verify_drafts(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(batch=0), INVALID), (dict(window=0), INVALID), (dict(window=33), INVALID), (dict(vocab=0), INVALID),
    (dict(vocab=(1 << 24) + 1), INVALID), (dict(probs=None), INVALID), (dict(drafts=None), INVALID),
    (dict(u=None), INVALID), (dict(tokens=None), INVALID), (dict(accepted=None), INVALID), (dict(lens=None), INVALID),
    (dict(out_lens=None), INVALID), (dict(type=3), INVALID), (dict(pt=99), INVALID), (dict(pb=399), INVALID),
    (dict(pb=0), INVALID), (dict(db=299), INVALID), (dict(dt=1 << 60), INVALID), (dict(probs=A[0] + 2), INVALID),
    (dict(ws=A[8], ws_bytes=8), SMALL), (dict(tokens=A[0]), ALIAS), (dict(accepted=A[6] + 16), ALIAS),
    (dict(out_lens=A[3]), ALIAS), (dict(ws=A[7], ws_bytes=256), ALIAS), (dict(out_lens=A[4] + 4), ALIAS)])
def test_drafts_validation(lib, change, status):
    assert drafts(lib, **change) == status


def weights(lib, **change):
    a = dict(q=A[0], dtype=BF16, kv=A[1], fmt=1, scales=None, lens=A[2], weights=A[3], batch=2, capacity=64, q_len=1,
             q_scale=1.0, k_scale=1.0, add=1, ws=A[4], ws_bytes=1 << 30, stream=None)
    a.update(change)
    return lib.gqa_accumulate_weights(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(q_len=0), INVALID), (dict(q_len=5), INVALID), (dict(lens=None), INVALID), (dict(weights=None), INVALID),
    (dict(weights=A[3] + 4), INVALID), (dict(dtype=F16), INVALID), (dict(k_scale=-1.0), INVALID),
    (dict(ws_bytes=300), SMALL), (dict(weights=A[1]), ALIAS), (dict(ws=A[3]), ALIAS), (dict(ws=A[0]), ALIAS)])
def test_weights_validation(lib, change, status):
    assert weights(lib, **change) == status


def evict(lib, **change):
    a = dict(kv=A[0], fmt=1, scales=None, lens=A[1], weights=A[2], out=A[3], out_scales=None, out_lens=A[4], out_weights=A[5],
             kept=A[6], batch=2, capacity=64, out_capacity=32, wcap=32, keep=32, recent=8, first=4, ws=A[7],
             ws_bytes=1 << 30, stream=None)
    a.update(change)
    return lib.gqa_evict_kv(*a.values())


@pytest.mark.parametrize("change,status", [
    (dict(keep=0), INVALID), (dict(keep=(1 << 30) + 1), INVALID), (dict(first=-1), INVALID), (dict(recent=29), INVALID),
    (dict(lens=None), INVALID), (dict(weights=None), INVALID), (dict(kept=None), INVALID), (dict(out_lens=None), INVALID),
    (dict(out=None), INVALID), (dict(out_capacity=31), INVALID), (dict(wcap=31), INVALID), (dict(fmt=3, scales=A[8]), INVALID),
    (dict(out=A[3] + 8), INVALID), (dict(kept=A[6] + 2), INVALID), (dict(ws_bytes=256), SMALL), (dict(out=A[0]), ALIAS),
    (dict(out_weights=A[2]), ALIAS), (dict(out_lens=A[1]), ALIAS), (dict(kept=A[4]), ALIAS), (dict(ws=A[6]), ALIAS),
    (dict(out=None, out_lens=None, out_weights=None, kept=A[1]), ALIAS),
    (dict(out=None, out_lens=None, out_weights=None, ws=A[0] + 256), ALIAS)])
def test_evict_validation(lib, change, status):
    assert evict(lib, **change) == status


def test_sizes(lib):
    assert lib.gqa_prefill_workspace_size() > 256
    assert lib.gqa_weights_workspace_size(2, 64, 4) >= 256 + 2 * 8 * 64 * 16 * 4
    assert lib.gqa_weights_workspace_size(0, 64, 1) == lib.gqa_weights_workspace_size(2, 64, 5) == 0
    assert lib.gqa_weights_workspace_size(64, 1 << 30, 4) > 1 << 41  # (past 32 bits)
    assert lib.gqa_evict_workspace_size(2, 100) > 256
    assert lib.gqa_evict_workspace_size(2, 0) == lib.gqa_evict_workspace_size(65536, 1) == 0
    with pytest.raises(ValueError):
        api.weights_workspace_size(1, 0)
    with pytest.raises(ValueError):
        api.evict_workspace_size(1, -1)


def test_messages(lib):
    evict(lib, recent=29)
    assert b"first and recent" in lib.gqa_last_error()
    assert isinstance(ctypes.string_at(lib.gqa_last_error()), bytes)

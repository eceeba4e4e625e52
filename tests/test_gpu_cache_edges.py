"""Cache writes at the edges of their number formats, against their definitions in 64 bits (GPU)."""
import math

import numpy as np
import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import _lib, api, inputs
from test_gpu_cache_io import (D, DEV, HKV, TD, check_heads, check_written, gen, library, new_cache,  # noqa: F401
                               page_table, rotated, rows_at, run_write, same_codes, tokens)

pytestmark = pytest.mark.gpu


def check_e2m1(got, gsc, plane, x, scale):
    """Codes and scales of one plane against exact x [N, 8, 128]; a group with a NaN has the NaN scale, whatever
    its codes."""
    codes, scales = inputs.quantise_e2m1(x, scale)
    nan = torch.isnan(x).unflatten(-1, (8, 16)).any(-1)
    assert ((gsc[:, plane] & 0x7F) == 0x7F)[nan].all(), "a NaN is kept as the group's NaN scale"
    assert torch.equal(gsc[:, plane][~nan], scales[~nan]), f"{int((gsc[:, plane] != scales)[~nan].sum())} scales"
    a, b = (c.unflatten(-1, (8, 8))[~nan] for c in (got[:, plane], codes))
    assert same_codes(a, b), f"{int((a != b).sum())} bytes of {a.numel()}"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [40, 1000])  # keys in doubt settled at once, and from the list
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
def test_small_groups_in_large_heads(dtype, n, norm, sparse):
    """Groups 1 to 2e-6 of their head's largest, with exact zeros and both signs: the FP32 error of the head is then
    up to several steps of a group's codes.  Sparse: a group holds zeros and both signs of one size alone, whose
    codes are far from every border but the one between the two signs of a zero.  Positions 0 to 3 (the definition's
    own angles are then good to 2^-51)."""
    t = tokens(n, 1, n, TD[dtype], seed=40)
    t["pos"] = (torch.arange(n, device=DEV) % 4).to(torch.int32)
    size = torch.tensor([1, 1e-4, 2e-5, 1e-5, 1e-6, 1e-6, 1e-6, 1e-6], device=DEV).repeat_interleave(16)
    big = 1000.0
    x = torch.randn((n, HKV, D), generator=gen(41), device=DEV)
    if sparse:
        x = torch.sign(x)
    x = torch.where(torch.rand((n, HKV, D), generator=gen(42), device=DEV) < 0.6, torch.zeros_like(x), x) * size * big
    x[..., 64:] = 0  # (pairs (i, i + 64) turn into one another)
    t["k"] = x.to(TD[dtype])
    t["kw"] = torch.ones_like(t["kw"])
    ks = float(np.float32((big if not norm else 8.0) / (6 * 448)))
    q_out, kv, sc, before, table, flags = run_write(t, "e2m1", 1, n, norm=norm, ks=ks, vs=1.0)
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    check_e2m1(got, gsc, 0, rotated(t["k"], t["kw"] if norm else None, t["pos"]), ks)


@pytest.mark.parametrize("n", [12, 1200])
@pytest.mark.parametrize("norm", [False, True])
def test_infinite_keys_saturate_and_nan_is_kept(n, norm):
    t = tokens(n, 1, n, torch.bfloat16, seed=43)
    t["pos"] = (1 + torch.arange(n, device=DEV) % 7).to(torch.int32)
    for k in range(0, n, 12):
        t["k"][k, 0, 5] = math.inf
        t["k"][k + 1, 3, 100] = -math.inf
        t["k"][k + 2, 7, 40] = math.nan
        t["k"][k + 3, 1, 2], t["k"][k + 3, 1, 66] = math.inf, math.inf  # a pair: inf - inf among them
        t["k"][k + 4, 2, 1], t["k"][k + 4, 2, 90] = math.nan, math.inf
        t["k"][k + 5] = math.nan
    q_out, kv, sc, before, table, flags = run_write(t, "e2m1", 1, n, norm=norm, ks=10 / 1024, vs=9 / 1024)
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    check_e2m1(got, gsc, 0, rotated(t["k"], t["kw"] if norm else None, t["pos"]), 10 / 1024)
    check_e2m1(got, gsc, 1, t["v"].double(), 9 / 1024)


@pytest.mark.parametrize("n", [12, 1200])
def test_nan_values_are_kept(n):
    t = tokens(n, 1, n, torch.bfloat16, seed=44)
    for k in range(0, n, 12):
        t["v"][k, 0, 5] = math.nan
        t["v"][k + 1, 3, 100], t["v"][k + 1, 3, 101] = -math.inf, math.nan
        t["v"][k + 2, 4] = math.nan
    q_out, kv, sc, before, table, flags = run_write(t, "e2m1", 1, n, ks=10 / 1024, vs=9 / 1024)
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    check_e2m1(got, gsc, 0, rotated(t["k"], t["kw"], t["pos"]), 10 / 1024)
    check_e2m1(got, gsc, 1, t["v"].double(), 9 / 1024)
    back = gq.read_kv(kv, torch.tensor([n], dtype=torch.int32, device=DEV), k_scale=10 / 1024, v_scale=9 / 1024,
                      kv_scales=sc)[0, 1].transpose(0, 1)[t["slots"].long()]
    assert torch.isnan(back[0, 0, :16]).all() and not torch.isnan(back[0, 0, 16:]).any()


def test_values_whose_quotient_is_next_to_the_largest_float():
    # 2^118 / (6 v_scale) just below 2^128: rounded up to a short number it would be infinite
    f = np.float32
    found = None
    for k in range(1, 2000):
        vs = f(f(2.0 ** -10) / f(6)) + f(k - 1000) * f(2.0 ** -36)
        d6 = f(6) * f(vs)
        inv = f(1) / d6
        with np.errstate(over="ignore"):
            q = f(2.0 ** 118) * inv
        if np.isfinite(q) and q.view(np.uint32) >= 0x7F7FFFC0:
            found = float(f(vs))
            break
    assert found is not None
    t = tokens(4, 1, 4, torch.bfloat16, seed=45)
    t["v"][0, 0, 0], t["v"][1, 1, 17] = 2.0 ** 118, -2.0 ** 118
    q_out, kv, sc, before, table, flags = run_write(t, "e2m1", 1, 4, ks=1.0, vs=found)
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    check_e2m1(got, gsc, 1, t["v"].double(), found)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1", "e4m3", "i8"])
@pytest.mark.parametrize("mag,eps", [(1e30, 1e-6), (3e36, 1e-6), (1e-25, 0.0), (1e-36, 0.0), (1e-12, 1e-24),
                                     (1e-30, 1e-30), (1e-12, 1e-38)])
@pytest.mark.parametrize("n", [40, 1000])
def test_norms_whose_squares_leave_fp32(fmt, mag, eps, n):
    t = tokens(n, 1, n, torch.bfloat16, seed=46, mag=mag / 20)
    t["pos"] = (torch.arange(n, device=DEV) % 1000).to(torch.int32)
    t["v"] = torch.randn(t["v"].shape, generator=gen(49), device=DEV).to(torch.bfloat16)  # (values have no norm)
    q_out, kv, sc, before, table, flags = run_write(t, fmt, 1, n, ks=10 / 1024, vs=1.0, eps=eps)
    check_heads(q_out, rotated(t["q"], t["qw"], t["pos"], eps=eps))
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    z = rotated(t["k"], t["kw"], t["pos"], eps=eps)
    if fmt == "e2m1":
        check_e2m1(got, gsc, 0, z, 10 / 1024)
    else:
        check_written(fmt, torch.bfloat16, got, gsc, z, t["v"], 10 / 1024, 1.0)


@pytest.mark.parametrize("scale", [0.01, 0.02, 0.7, 1.3, 41.0, 2.0 ** -5])
def test_e4m3_values_are_products_with_the_reciprocal(scale):
    """Every finite fp16 value, written by both entries: the FP32 product with the FP32 reciprocal, rounded to e4m3
    (no value further from value / scale than half a step and the two FP32 roundings)."""
    bits = torch.arange(65536, device=DEV).to(torch.int32).to(torch.int16).view(torch.float16)
    v = bits[torch.isfinite(bits)]
    n = -(-v.numel() // (HKV * D))
    v = torch.cat((v, torch.zeros(n * HKV * D - v.numel(), dtype=v.dtype, device=DEV))).view(n, HKV, D)
    t = tokens(n, 1, n, torch.float16, seed=47)
    t["v"] = v
    q_out, kv, sc, before, table, flags = run_write(t, "e4m3", 1, n, ks=1.0, vs=scale)
    got, _, _ = rows_at(kv, None, None, 0, t["rows"], t["slots"])
    inv = np.float32(1) / np.float32(scale)
    want = (v.float() * float(inv)).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(got[:, 1], want.view(torch.uint8))
    x = torch.clamp(v.double() / float(np.float32(scale)), -448, 448)
    back = got[:, 1].contiguous().view(torch.float8_e4m3fn).double()
    assert ((back - x).abs() <= torch.clamp(x.abs() * (2 ** -4 + 2 ** -22), min=2 ** -10 * (1 + 2 ** -18))).all()
    # the append step takes one token a row
    kv2, _ = new_cache("e4m3", n, 8)
    slots = torch.zeros(n, dtype=torch.int32, device=DEV)
    gq.append_kv(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], slots, kv2, k_scale=1.0, v_scale=scale)
    assert torch.equal(kv2[:, 1, :, 0], got[:, 1])


@pytest.mark.parametrize("what", ["write", "write scales", "read", "decode", "decode scales"])
def test_cut_extents_make_the_checks_fire(library, what):  # noqa: F811
    """The checked library's range checks see an access past extents that are cut short (and keep it inside the
    real buffers); with the true extents the same call is clean.  The product library has no checks to cut."""
    lib = _lib.load()
    n = 512
    t = tokens(n, 2, 256, torch.bfloat16, seed=48)
    kv, sc = new_cache("e2m1", 2, 256)
    table, units = page_table(2, 256, 16)
    pages, page_sc = new_cache("e2m1", units, 16)
    lens = torch.tensor([256, 255], dtype=torch.int32, device=DEV)
    how = dict(k_scale=0.01, v_scale=0.01)

    def run(paged):
        ws = torch.zeros(gq.workspace_size(2, 256, 2), dtype=torch.uint8, device=DEV)
        a = (t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"])
        if what.startswith("write"):
            if paged:
                gq.write_kv_paged(*a, pages, table, kv_scales=page_sc, workspace=ws, **how)
            else:
                gq.write_kv(*a, kv, kv_scales=sc, workspace=ws, **how)
        elif what == "read":
            if paged:
                gq.read_kv_paged(pages, table, lens, kv_scales=page_sc, workspace=ws, **how)
            else:
                gq.read_kv(kv, lens, kv_scales=sc, workspace=ws, **how)
        elif paged:
            gq.gqa_decode_paged(t["q"][:2], pages, table, lens, num_splits=2, workspace=ws, kv_scales=page_sc, **how)
        else:
            gq.gqa_decode_fp4kv(t["q"][:2], kv, sc, lens, num_splits=2, workspace=ws, **how)
        return gq.get_status(ws)

    for paged, codes, scales in ((False, kv, sc), (True, pages, page_sc)):
        cut = (0, scales.numel() // 2) if what.endswith("scales") else (codes.numel() // 2, 0)
        if library == "product":
            assert lib.gqa_decode_debug_cut_extents(*cut) == 1
            continue
        before = codes.clone()
        try:
            assert lib.gqa_decode_debug_cut_extents(*cut) == 0
            flags = run(paged)
        finally:
            assert lib.gqa_decode_debug_cut_extents(0, 0) == 0
        assert flags & api.FLAG_BOUNDS and not flags & api.FLAG_WAIT_TIMEOUT, hex(flags)
        if what.startswith("write"):  # nothing behind the cut is written
            assert torch.equal(codes[codes.shape[0] // 2 + 1:], before[codes.shape[0] // 2 + 1:])
            assert torch.equal(codes[-1], before[-1])
        assert not run(paged) & api.FLAG_BOUNDS


@pytest.mark.parametrize("seed", range(20))
def test_random_sizes_zeros_and_specials(seed):
    # groups of a head up to 2^60 apart (fp16: 2^14), zeros, powers of two (ties), infinities and NaN; positions below
    # 64, where the definition's angles are good to 2^-47
    rng, g = np.random.default_rng(seed), gen(seed + 60)
    dtype = [torch.float16, torch.bfloat16][rng.integers(2)]
    n = int(np.exp(rng.uniform(0, np.log(2500))))
    t = tokens(n, 1, n, dtype, seed=seed)
    t["pos"] = torch.randint(0, int(rng.integers(1, 64)), (n,), generator=g, device=DEV).to(torch.int32)
    wide, middle = (14, 0.0) if dtype == torch.float16 else (60, float(rng.uniform(-60, 60)))
    for name, heads in (("q", 32), ("k", 8), ("v", 8)):
        e = middle - torch.rand((n, heads, 8, 1), generator=g, device=DEV) * (wide * float(rng.random()))
        x = torch.randn((n, heads, 8, 16), generator=g, device=DEV) * torch.exp2(e)
        x[torch.rand(x.shape, generator=g, device=DEV) < float(rng.choice([0, 0.3, 0.9]))] = 0
        if rng.random() < 0.3:
            x = torch.exp2(torch.round(torch.log2(x.abs().clamp(min=1e-38)))) * torch.sign(x)
        if rng.random() < 0.4:
            x[torch.rand(x.shape, generator=g, device=DEV) < 1e-3] = float(rng.choice([math.inf, -math.inf, math.nan]))
        t[name] = x.flatten(2).to(dtype).contiguous()
    norm, eps = bool(rng.random() < 0.6), float(rng.choice([1e-6, 0.0, 1e-20, 1.0]))
    z = rotated(t["k"], t["kw"] if norm else None, t["pos"], eps=eps)
    scale = []
    for x in (z, t["v"].double()):
        top = torch.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0).abs().max() * 2.0 ** float(rng.uniform(-3, 3)) / 2688
        scale.append(float(np.float32(min(2.0 ** 99, max(2.0 ** -99, float(top))))))
    q_out, kv, sc, before, table, flags = run_write(t, "e2m1", 1, n, norm=norm, ks=scale[0], vs=scale[1], eps=eps)
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    check_e2m1(got, gsc, 0, z, scale[0])
    check_e2m1(got, gsc, 1, t["v"].double(), scale[1])
    zq = rotated(t["q"], t["qw"] if norm else None, t["pos"], eps=eps)
    heads = torch.isfinite(zq).all(-1) & (zq.abs().amax(-1) < torch.finfo(dtype).max / 2)
    check_heads(q_out[heads], zq[heads])
    assert torch.isnan(q_out[torch.isnan(zq)]).all()


@pytest.mark.parametrize("fmt", ["bf16", "e2m1", "i8"])
@pytest.mark.parametrize("n", [60, 2000])
def test_padding_may_hold_anything(fmt, n):
    # the tokens of slot -1 are NaN, infinite and huge: the others are what they are without them
    t = tokens(n, 1, n, torch.bfloat16, seed=55)
    pad = torch.rand(n, generator=gen(56), device=DEV) < 0.5
    t["pos"] = (torch.arange(n, device=DEV) % 5000).to(torch.int32)
    for name in "qkv":
        junk = torch.randint(-32768, 32768, t[name].shape, generator=gen(57), device=DEV).to(torch.int16)
        t[name][pad] = junk.view(torch.bfloat16)[pad]
    t["slots"][pad] = -1
    t["pos"][pad] = torch.randint(-2 ** 31, 2 ** 31 - 1, (int(pad.sum()),), generator=gen(58), device=DEV).to(torch.int32)
    q_out, kv, sc, before, table, flags = run_write(t, fmt, 1, n, ks=10 / 1024, vs=9 / 1024)
    assert flags == api.FLAG_SLOT_CLAMPED
    check_heads(q_out[~pad], rotated(t["q"], t["qw"], t["pos"])[~pad])
    got, gsc, (r, s) = rows_at(kv, sc, None, 0, t["rows"][~pad], t["slots"][~pad])
    check_written(fmt, torch.bfloat16, got, gsc, rotated(t["k"], t["kw"], t["pos"])[~pad], t["v"][~pad], 10 / 1024, 9 / 1024)
    before[0][r, :, :, s] = got
    assert torch.equal(before[0].view(torch.uint8), kv.view(torch.uint8))


def test_threads_on_their_own_streams():
    # calls release the interpreter: four threads at once, each with its own cache, theta and stream
    import threading
    n, C = 96, 128
    jobs, errors = [], []
    for k in range(4):
        t = tokens(n, 1, C, torch.bfloat16, seed=70 + k)
        kv, sc = new_cache("e2m1", 1, C, seed=k)
        jobs.append((t, kv, sc, 1e4 * (k + 1)))

    def chain(t, kv, sc, theta):
        how = dict(k_scale=0.01, v_scale=0.01, kv_scales=sc)
        lens = torch.tensor([C], dtype=torch.int32, device=DEV)
        q = gq.write_kv(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv, rope_theta=theta, **how)
        ws = torch.zeros(gq.workspace_size(1, C, 2), dtype=torch.uint8, device=DEV)
        out = gq.gqa_decode_fp4kv(q[:1], kv, sc, lens, 0.01, 0.01, out=torch.empty_like(q[:1]), num_splits=2, workspace=ws)
        back = gq.read_kv(kv, lens, out=torch.zeros((1, 2, HKV, C, D), dtype=torch.float16, device=DEV), **how)
        return q, kv.clone(), sc.clone(), out, back

    want = [chain(*j) for j in jobs]
    torch.cuda.synchronize()

    def work(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = chain(*jobs[k])
                    stream.synchronize()
                    assert all(torch.equal(a, b) for a, b in zip(got, want[k]))
                    with pytest.raises(gq.GqaError, match="rope_theta"):  # the message is the thread's own
                        chain(*jobs[k][:3], 0.25 * (k + 1) if k < 3 else -1.0)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors, errors


def test_the_largest_batch_and_page(library):  # noqa: F811
    # 65535 rows of 16 slots: the last rows' grid coordinates
    B, C, n = 65535, 16, 64
    kv = torch.zeros((B, 2, HKV, C, 64), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((B, 2, HKV, C, 8), dtype=torch.uint8, device=DEV)
    t = tokens(n, 1, n, torch.bfloat16, seed=80)
    t["rows"] = (B - 1 - torch.arange(n, device=DEV) // C).to(torch.int32)
    t["slots"] = (torch.arange(n, device=DEV) % C).to(torch.int32)
    ws = torch.zeros(gq.workspace_size(B, C, 1), dtype=torch.uint8, device=DEV)
    how = dict(k_scale=0.01, v_scale=0.01, kv_scales=sc)
    gq.write_kv(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv, workspace=ws, **how)
    got, gsc, _ = rows_at(kv, sc, None, 0, t["rows"], t["slots"])
    check_written("e2m1", torch.bfloat16, got, gsc, rotated(t["k"], t["kw"], t["pos"]), t["v"], 0.01, 0.01)
    lens = torch.full((B,), C, dtype=torch.int32, device=DEV)
    back = gq.read_kv(kv, lens, out=torch.ones((B, 2, HKV, C, D), dtype=torch.bfloat16, device=DEV), workspace=ws, **how)
    assert not back[:B - n // C].any()
    tail = torch.stack([inputs.dequantise_e2m1(kv[B - n // C:, p], sc[B - n // C:, p], 1.0) for p in (0, 1)], 1)
    assert torch.equal(back[B - n // C:], (tail.float() * float(np.float32(0.01))).bfloat16())
    q = torch.randn((B, 32, D), generator=gen(81), device=DEV).to(torch.bfloat16)
    out = gq.gqa_decode_fp4kv(q, kv, sc, lens, 0.01, 0.01, num_splits=1, workspace=ws)
    assert not out[:B - n // C].any()
    assert gq.get_status(ws) == 0
    x = back[-1].double()
    s = torch.einsum("ghd,gtd->ght", q[-1].double().view(8, 4, D), tail[-1, 0] * 0.01) / math.sqrt(D)
    ref = torch.einsum("ght,gtd->ghd", torch.softmax(s, -1), tail[-1, 1] * 0.01).reshape(32, D)
    assert ((out[-1].double() - ref).abs() <= ref.abs() * 2 ** -8 + x[1].abs().max() * 2 ** -10).all()
    del kv, sc, back, q, out
    # pages of 65536 slots, the last slots of the second page of a row
    P = 65536
    kv, sc = new_cache("e2m1", 3, P, seed=82)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    t["rows"].zero_()
    t["slots"] = (2 * P - n + torch.arange(n, device=DEV)).to(torch.int32)
    gq.write_kv_paged(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv, table, k_scale=0.01,
                      v_scale=0.01, kv_scales=sc, workspace=ws)
    got, gsc, _ = rows_at(kv, sc, table, P, t["rows"], t["slots"])
    check_written("e2m1", torch.bfloat16, got, gsc, rotated(t["k"], t["kw"], t["pos"]), t["v"], 0.01, 0.01)
    lens = torch.tensor([2 * P], dtype=torch.int32, device=DEV)
    out = gq.read_kv_paged(kv, table, lens, starts=lens - 2 * n, out=torch.zeros((1, 2, HKV, 2 * n, D), dtype=torch.float16,
                           device=DEV), k_scale=0.01, v_scale=0.01, kv_scales=sc, workspace=ws)
    x = torch.stack([inputs.dequantise_e2m1(kv[0, p, :, -2 * n:], sc[0, p, :, -2 * n:], 1.0) for p in (0, 1)])
    assert torch.equal(out[0], (x.float() * float(np.float32(0.01))).half())
    assert gq.get_status(ws) == 0

"""The serving calls at the limits of what they take: values and scales that a query
does not see, infinite scores, weights of every kind, calls without a token (GPU).

Bounds as in test_gpu_serving.py, with what each test says of its own.
"""
import math
import threading

import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from test_gpu_serving import (D, DEV, HKV, HQ, TD, attend64, draft_inputs, gen, kept64, library,  # noqa: F401
                              new_cache, paged, run_together, serving_state, together_buffers, values)

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


# ------------------------------------------------ prompt attention: large values


@pytest.mark.parametrize("n,L", [(70, 300), (40, 20000), (5, 129)])
def test_prefill_largest_bf16_values(library, n, L):  # noqa: F811
    """bf16 values up to the type's largest: weights are held at 1 or less, so a row's
    sum of weight * |V| stays what FP32 holds."""
    kv, _ = new_cache("bf16", 1, L, 5)
    q = torch.randn((n, HQ, D), generator=gen(6), device=DEV).to(torch.bfloat16)
    starts, lens = torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([L], dtype=torch.int32, device=DEV)
    half = 2.0 ** -8
    big = torch.finfo(torch.bfloat16).max
    for what in ("one", "all"):
        x = kv.clone()
        if what == "one":
            x[0, 1, :, 3] = big
            x[0, 1, :, L - n + 1, ::2] = -big
        else:
            x[0, 1] *= 2.0 ** 108  # (20000 * 2^108 * 5 < 2^127)
        out = gq.gqa_prefill(q, x, starts, lens)
        for j in (0, 1, n // 2, n - 1):
            ref, a, e = attend64(q[j], x[0, 0].double(), x[0, 1].double(), L - n + j + 1)
            assert float(ref.abs().max()) < big / 2
            err = (out[j].double() - ref).abs()
            assert (err <= half * ref.abs() + (half + 2 * e + 2 ** -18) * a).all(), f"{what}: query {j}"


# --------------------------------------------- calls without a token, and flags


@pytest.mark.parametrize("starts,lens", [([10, 0, 0], [5, 5]), ([0, 0, 0], [-1, 5]), ([0, 0, 0], [5, 65]),
                                         ([4, 4, 3], [9, 9]), ([20, 20, 20], [9, 9])])
def test_prefill_flags_without_tokens(library, starts, lens):  # noqa: F811
    """What is out of contract is told also where no row has a token."""
    kv, _ = new_cache("bf16", 2, 64, 8)
    q = torch.randn((12, HQ, D), generator=gen(9), device=DEV).to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    ws = torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    gq.gqa_prefill(q, kv, torch.tensor(starts, **i32), torch.tensor(lens, **i32), out=out, workspace=ws)
    assert gq.get_status(ws) == gq.api.FLAG_LENGTH_CLAMPED
    assert (out == 3.0).all()
    gq.gqa_prefill(q, kv, torch.zeros(3, **i32), torch.tensor([5, 0], **i32), out=out, workspace=ws)
    assert gq.get_status(ws) == 0


# ------------------------------------------------- weight sums: infinite scores


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "bf16")])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("C", [300, 40000])  # on chip and in two launches
def test_weights_of_minus_infinity(library, fmt, dtype, T, C):  # noqa: F811
    """A score of minus infinity gives its slot no weight and leaves the others theirs,
    wherever it lies: a lane's first slot, a whole slab of a warp, or the last."""
    L = C - 3
    g = gen(12)
    q = torch.randn((1, T, HQ, D), generator=g, device=DEV).to(TD[dtype])
    q[..., 0] = 1.0 + torch.rand(q.shape[:-1], generator=g, device=DEV).to(TD[dtype])
    for at in ([0], [0, 8], list(range(16)), list(range(32)), [5, 17, 100, L - T], list(range(130, 290)), [L // 2]):
        kv, sc = new_cache(fmt, 1, C, 13)
        if fmt == "i8":
            sc[0, 0, :, at] = INF
            kv[0, 0, :, at] = 0
            kv[0, 0, :, at, 0] = -1
            # (0 * inf is no number in the values; codes 0 add nothing to the score)
        else:
            kv[0, 0, :, at, 0] = -INF
        lens = torch.tensor([L], dtype=torch.int32, device=DEV)
        got = gq.accumulate_weights(q, kv, lens, torch.zeros((1, HKV, C), device=DEV), kv_scales=sc, add=False)
        K = torch.nan_to_num(values(kv[:, 0], None if sc is None else sc[:, 0], fmt, 1.0)[0], nan=0.0, neginf=0.0)
        w, e = (torch.zeros((HKV, L), dtype=torch.float64, device=DEV) for _ in range(2))
        for j in range(T):
            end = L - T + 1 + j
            k = K[:, :end].repeat_interleave(4, 0)
            s = torch.einsum("hd,htd->ht", q[0, j].double(), k) / math.sqrt(128.0)
            m = torch.einsum("hd,htd->ht", q[0, j].double().abs(), k.abs()).amax(-1, keepdim=True) / math.sqrt(128.0)
            ds = 2 ** -16 * m + 2 ** -22 * s.abs().amax(-1, keepdim=True)
            s[:, [t for t in at if t < end]] = -INF
            x = torch.softmax(s, -1)
            w[:, :end] += x.view(HKV, 4, end).sum(1)
            e[:, :end] += (x * (2 * ds + 2 ** -19)).view(HKV, 4, end).sum(1)
        assert not got[0][:, at].any()
        assert ((got[0, :, :L].double() - w).abs() <= e + 2 ** -126).all()


def test_weights_of_minus_infinity_alone(library):  # noqa: F811
    """A query whose scores are all minus infinity gives no weight (its softmax has no
    value), and a NaN score among them still makes NaN of the row's."""
    for C in (40, 40000):
        kv, _ = new_cache("f16", 2, C, 14)
        kv[:, 0, 2, :, 0] = -INF
        kv[1, 0, 2, C // 2, 0] = NAN
        q = torch.rand((2, HQ, D), generator=gen(15), device=DEV).half() + 0.5
        lens = torch.full((2,), C, dtype=torch.int32, device=DEV)
        w = gq.accumulate_weights(q, kv, lens, torch.full((2, HKV, C), 2.0, device=DEV))
        assert (w[0, 2] == 2.0).all()
        assert torch.isnan(w[1, 2, C // 2]) and not (w[1, 2] > 2.0).any()
        others = [h for h in range(HKV) if h != 2]
        # (2 + w is rounded to FP32: by 2^-22 of itself, a head's sum by no more)
        total = (w[:, others].double() - 2.0).sum(-1)
        assert ((total - 4.0).abs() <= C * 2.0 ** -22 + 4 * 2.0 ** -12).all()


# ------------------------------------------------------ eviction: kinds of weights


@pytest.mark.parametrize("C", [300, 1024, 3000, 8000, 9000])
def test_evict_as_many_numbers_as_needed(library, C):  # noqa: F811
    """Weights of both signs, and NaN, with as many numbers as are needed, one fewer, one more."""
    first, recent, L = 4, 9, C - 5
    hi = L - recent
    keep = C // 3
    need = keep - first - recent
    g = gen(C)
    for extra in (0, -1, 1):
        w = torch.randn((2, HKV, C), generator=g, device=DEV)
        w[0, 1] = -w[0, 1].abs()                       # negative ones of every size
        w[0, 2] = -1.0                                 # one negative value
        w[0, 3] = w[0, 3].sign()                       # two values
        w[0, 4] = torch.where(w[0, 4] > 0, INF, -INF)
        w[0, 5] = torch.where(w[0, 5] > 0, 0.0, -0.0)
        w[0, 6] = w[0, 6].abs()
        w[0, 7] = (w[0, 7] * 1e4).floor() * 1e-45      # subnormal, both signs
        w[1] *= 10.0 ** torch.randint(-30, 30, (HKV, C), generator=g, device=DEV)
        for b in range(2):
            for h in range(HKV):
                between = torch.randperm(hi - first, generator=g, device=DEV) + first
                w[b, h, between[need + extra:]] = NAN
        kv, _ = new_cache("f16", 2, C, 16)
        lens = torch.full((2,), L, dtype=torch.int32, device=DEV)
        out, ol = torch.zeros((2, 2, HKV, keep, D), dtype=torch.float16, device=DEV), torch.zeros_like(lens)
        ws = torch.zeros(gq.evict_workspace_size(2, keep), dtype=torch.uint8, device=DEV)
        kept = torch.full((2, HKV, keep), -9, dtype=torch.int32, device=DEV)
        gq.evict_kv(kv, lens, w, keep, recent, first, out=out, out_lengths=ol, kept=kept, workspace=ws)
        assert gq.get_status(ws) == 0
        for b in range(2):
            for h in range(HKV):
                want = kept64(w[b, h].tolist(), L, keep, recent, first)
                same = kept[b, h].tolist() == want  # (no diff of long lists)
                assert same, f"row {b} head {h}, {need + extra} numbers for {need}"
                assert torch.equal(out[b, :, h], kv[b, :, h][:, want])


# -------------------------------------------------- sizes past what an int holds


def test_sizes_past_an_int(library):  # noqa: F811
    kv, _ = new_cache("bf16", 1, 64, 60)
    lens = torch.tensor([64], dtype=torch.int32, device=DEV)
    w = torch.zeros((1, HKV, 64), device=DEV)
    for bad in (dict(recent=2 ** 32 + 2), dict(first=2 ** 32), dict(recent=-2 ** 32 + 1), dict(first=2 ** 31)):
        with pytest.raises(ValueError, match="2\\^31"):
            gq.evict_kv(kv, lens, w, 10, **bad)
        with pytest.raises(ValueError, match="2\\^31"):
            gq.evict_kv_paged(kv, torch.zeros((1, 1), dtype=torch.int32, device=DEV), lens, w, 10, **bad)
    for bad in (dict(recent=1.5), dict(first="1")):
        with pytest.raises(TypeError):
            gq.evict_kv(kv, lens, w, 10, **bad)
    assert int(lens) == 64
    with pytest.raises(ValueError, match="2\\^31"):
        gq.evict_kv(kv, lens, w, 2 ** 32 + 8)
    with pytest.raises(ValueError, match="2\\^31"):  # (8 GB)
        gq.verify_drafts(torch.zeros((1, 1, 2 ** 32 + 5), dtype=torch.float16, device=DEV),
                         torch.zeros((1, 0), dtype=torch.int32, device=DEV), torch.zeros((1, 1), device=DEV))
    torch.cuda.empty_cache()


# -------------------------------------------------- drafts: lengths and large sums


def test_drafts_lengths_below_zero(library):  # noqa: F811
    """max(length - (T - 1) + n, 0) of any int, without overflow."""
    p, d, u, q, _ = draft_inputs(6, 4, 50, "f32", seed=80)
    low = -2 ** 31
    lens = torch.tensor([low, low + 1, low + 2, -1, 0, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    tokens, accepted = gq.verify_drafts(p, d, u, draft_probs=q, sequence_lengths=lens)
    assert lens[:4].tolist() == [0] * 4
    assert int(lens[4]) == 0 and int(lens[5]) == 2 ** 31 - 1 - 3 + int(accepted[5])


# ----------------------------------------------------------------- largest sizes


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_drafts_largest_vocabulary(library, dtype):  # noqa: F811
    """2^24 tokens, and terms of 2^38 units each (their sum is 2^62)."""
    V = 1 << 24
    d, u = torch.zeros((3, 0), dtype=torch.int32, device=DEV), torch.tensor([[0.0], [0.3], [1 - 2.0 ** -24]], device=DEV)
    p = torch.ones((3, 1, V), dtype=TD[dtype], device=DEV)
    tokens, accepted = gq.verify_drafts(p, d, u)
    assert tokens[:, 0].tolist() == [int(math.floor(float(x) * 2 ** 24)) for x in u]
    p = torch.rand((3, 1, V), generator=gen(81), device=DEV).to(TD[dtype])
    tokens, _ = gq.verify_drafts(p, d, u)
    w = (p[:, 0].float().clamp(0, 1).double() * 2.0 ** 38).round().long()
    upto = w.cumsum(1)
    for b in range(3):
        target = int(upto[b, -1]) * int(math.floor(float(u[b, 0]) * 2 ** 24)) >> 24
        assert int(tokens[b, 0]) == int(torch.searchsorted(upto[b], target, right=True))


def test_drafts_rows_far_apart(library):  # noqa: F811
    """Rows 2^32 elements apart, at an odd 16-bit offset."""
    V, apart = 3001, 2 ** 32 + 1
    p, d, u, q, lens = draft_inputs(2, 3, V, "f16", seed=88)
    want = gq.verify_drafts(p, d, u, draft_probs=q, sequence_lengths=lens.clone())
    far = torch.empty(apart + 4 * V, dtype=torch.float16, device=DEV)  # 8 GB
    wide = far.as_strided((2, 3, V), (apart, V + 2, 1), 1)
    wide.copy_(p)
    got = gq.verify_drafts(wide, d, u, draft_probs=q, sequence_lengths=lens)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del far, wide
    torch.cuda.empty_cache()


def test_prefill_many_tokens(library):  # noqa: F811
    """More than 2^31 elements of q and out (4.9 GB each)."""
    B, n = 600, 1000
    kv = torch.randn((1, 2, HKV, n, D), generator=gen(89), device=DEV).to(torch.bfloat16)
    pool = torch.zeros((2 * 16, 2, HKV, 64, D), dtype=torch.bfloat16, device=DEV)
    for k in range(16):  # (every row has the same pages)
        part = kv[0, :, :, 64 * k:64 * (k + 1)]
        pool[k, :, :, :part.shape[2]] = part
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(16, **i32).repeat(B, 1)
    q = torch.empty((B * n, HQ, D), dtype=torch.bfloat16, device=DEV)
    for b in range(B):
        q[b * n:(b + 1) * n] = torch.randn((n, HQ, D), generator=gen(b), device=DEV).to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    gq.gqa_prefill_paged(q, pool, table, torch.arange(0, B * n + 1, n, **i32), torch.full((B,), n, **i32), out=out, workspace=ws)
    assert gq.get_status(ws) == 0
    half = 2.0 ** -8
    K, V = kv[0, 0].double(), kv[0, 1].double()
    for t in (0, n - 1, 524287, 524288, 524289, B * n - n, B * n - 1):
        ref, a, e = attend64(q[t], K, V, t % n + 1)
        assert ((out[t].double() - ref).abs() <= half * ref.abs() + (half + 2 * e + 2 ** -18) * a + 2 ** -126).all(), t
    del q, out
    torch.cuda.empty_cache()


@pytest.mark.parametrize("C", [65536, 400032])  # above 393216 slots the weights are read again each time
def test_evict_long_rows(library, C):  # noqa: F811
    kv, _ = new_cache("e4m3", 1, C, 82)
    w = torch.rand((1, HKV, C), generator=gen(83), device=DEV)
    w[0, 1] = (w[0, 1] * 8).floor()  # ties over all of the row
    w[0, 2, ::3] = NAN
    w[0, 3] -= 0.5
    L, keep, recent, first = C - 77, C // 5, 300, 7
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    out = torch.zeros((1, 2, HKV, keep, D), dtype=torch.uint8, device=DEV)
    ol, ow = torch.zeros_like(lens), torch.zeros((1, HKV, keep), device=DEV)
    ws = torch.zeros(gq.evict_workspace_size(1, keep), dtype=torch.uint8, device=DEV)
    kept = gq.evict_kv(kv, lens, w, keep, recent, first, out=out, out_lengths=ol, out_weights=ow, workspace=ws)
    assert gq.get_status(ws) == 0 and int(ol) == keep
    key = torch.where(torch.isnan(w[0, :, :L]), -INF, w[0, :, :L])
    key[:, :first] = INF
    key[:, L - recent:] = INF
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :keep]
    want = torch.sort(order, dim=-1).values
    assert torch.equal(kept[0].long(), want)
    assert torch.equal(out[0], kv[0].gather(2, want[None, :, :, None].expand(2, HKV, keep, D)))
    assert torch.equal(ow[0].view(torch.int32), w[0].gather(1, want).view(torch.int32))
    # in place: the same slots
    gq.evict_kv(kv, lens, w, keep, recent, first, kept=kept, workspace=ws)
    assert gq.get_status(ws) == 0 and int(lens) == keep and torch.equal(kept[0].long(), want)
    assert torch.equal(kv[:, :, :, :keep], out)


def test_evict_keep_past_the_capacity(library):  # noqa: F811
    """More slots asked for than the cache has: all stay."""
    kv, _ = new_cache("bf16", 2, 50, 84)
    w = torch.rand((2, HKV, 50), generator=gen(85), device=DEV)
    lens = torch.tensor([50, 17], dtype=torch.int32, device=DEV)
    out, ol = torch.zeros((2, 2, HKV, 130, D), dtype=torch.bfloat16, device=DEV), torch.zeros_like(lens)
    ow = torch.full((2, HKV, 140), 5.0, device=DEV)
    kept = gq.evict_kv(kv, lens, w, 120, 100, 20, out=out, out_lengths=ol, out_weights=ow)
    before, old = kv.clone(), w.clone()
    same = gq.evict_kv(kv, lens, w, 120, 100, 20)
    assert torch.equal(kept, same) and torch.equal(kv, before) and torch.equal(w, old) and lens.tolist() == [50, 17]
    for b, n in enumerate((50, 17)):
        assert kept[b].tolist() == [list(range(n)) + [-1] * (120 - n)] * HKV and int(ol[b]) == n
        assert torch.equal(out[b, :, :, :n], kv[b, :, :, :n]) and not out[b, :, :, n:].any()
        assert torch.equal(ow[b, :, :n], w[b, :, :n]) and not ow[b, :, n:].any()


def test_prefill_padding_in_front(library):  # noqa: F811
    """The first chunk may start behind padding."""
    kv, _ = new_cache("f16", 2, 200, 86)
    q = torch.randn((100, HQ, D), generator=gen(87), device=DEV).half()
    i32 = dict(dtype=torch.int32, device=DEV)
    lens = torch.tensor([150, 199], **i32)
    ws = torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, 3.0)
    gq.gqa_prefill(q, kv, torch.tensor([13, 50, 90], **i32), lens, out=out, workspace=ws)
    assert gq.get_status(ws) == 0 and (out[:13] == 3.0).all() and (out[90:] == 3.0).all()
    want = gq.gqa_prefill(q[13:90].contiguous(), kv, torch.tensor([0, 37, 77], **i32), lens)
    assert torch.equal(out[13:90], want)


# ------------------------------------------------------------------ fresh threads


def in_thread(f):
    """f() in a thread that has made no call of the GPU before; what it raised."""
    raised = []

    def run():
        try:
            f()
        except Exception as e:  # noqa: BLE001
            raised.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return raised


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_first_call_of_a_thread(library, fmt):  # noqa: F811
    """Each call as a thread's first work on the GPU, with every buffer given, so that
    nothing before it gives the thread a context."""
    s = serving_state(fmt)
    ws = together_buffers(s)
    fill = ws["kv"].clone()  # (slots past the new length keep it)
    want = [x.clone() for x in run_together(s, ws)]
    B = s["B"]
    ks, vs = (0.4, 0.7) if fmt == "e2m1" else (1.0, 1.0)
    q = s["q"].view(B, -1, HQ, D)[:, :2].contiguous()
    torch.cuda.synchronize()
    calls = [
        lambda: gq.gqa_prefill(s["q"], s["kv"], s["starts"], s["lens"], k_scale=ks, v_scale=vs, kv_scales=s["sc"], out=ws["out"],
                               workspace=ws["prefill"]),
        lambda: gq.accumulate_weights(q, s["kv"], s["lens"], ws["w"], k_scale=ks, kv_scales=s["sc"], add=False,
                                      workspace=ws["weights"]),
        lambda: gq.verify_drafts(ws["p"], ws["d"], ws["u"], draft_probs=ws["dq"], sequence_lengths=s["lens"],
                                 out_lengths=ws["len1"], tokens=ws["tokens"], accepted=ws["accepted"]),
        lambda: gq.evict_kv(s["kv"], ws["len1"], ws["w"], 100, 16, 4, out=ws["kv"], out_scales=ws["sc"],
                            out_lengths=ws["len2"], out_weights=ws["w2"], kept=ws["kept"], kv_scales=s["sc"],
                            workspace=ws["evict"]),
    ]
    for x in (ws["out"], ws["w"], ws["tokens"], ws["accepted"], ws["len1"], ws["kept"], ws["len2"], ws["w2"]):
        x.zero_()
    ws["kv"].copy_(fill)
    torch.cuda.synchronize()
    for call in calls:
        assert not in_thread(call)
    got = [ws["out"], ws["w"], ws["tokens"], ws["accepted"], ws["len1"], ws["kept"], ws["kv"], ws["len2"], ws["w2"]]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_threads_at_once(library):  # noqa: F811
    """Four threads, each on a stream and with buffers of its own, all calls many times."""
    s = serving_state("bf16")
    want = [x.clone() for x in run_together(s, together_buffers(s))]
    buffers = [together_buffers(s) for _ in range(4)]
    torch.cuda.synchronize()
    raised, barrier = [], threading.Barrier(4)

    def work(ws):
        try:
            stream = torch.cuda.Stream()
            barrier.wait(30)
            with torch.cuda.stream(stream):
                for _ in range(25):
                    run_together(s, ws)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            raised.append(e)
    threads = [threading.Thread(target=work, args=(ws,)) for ws in buffers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not raised
    for ws in buffers:
        got = [ws["out"], ws["w"], ws["tokens"], ws["accepted"], ws["len1"], ws["kept"], ws["kv"], ws["len2"], ws["w2"]]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for name in ("prefill", "weights", "evict"):
            assert gq.get_status(ws[name]) == 0


# ------------------------------------------------- block tables past the length


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("fmt", ["bf16", "i8", "e2m1"])
def test_table_entries_past_the_length(library, fmt, page):  # noqa: F811
    """Entries that no slot in use needs may hold anything: they are neither read from nor told."""
    B, C = 3, 1024
    kv, sc = new_cache(fmt, B, C, 90)
    pool, psc, table = paged(kv, sc, page, B, C, 91)
    lens = torch.tensor([1, 3 * page + 1, 2 * page], dtype=torch.int32, device=DEV).clamp(max=C)
    wild = table.clone()
    for b, L in enumerate(lens.tolist()):
        wild[b, -(-L // page):] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31, 10 ** 6], dtype=torch.int32,
                                               device=DEV).repeat(C)[:C // page - -(-L // page)]
    n = [1, 20, 33]
    n[2] = min(n[2], int(lens[2]))
    i32 = dict(dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, n[0], n[0] + n[1], sum(n)], **i32)
    q = torch.randn((sum(n), HQ, D), generator=gen(92), device=DEV).to(torch.bfloat16)
    w0, keep = torch.rand((B, HKV, C), generator=gen(93), device=DEV), 2 * page - 3
    got = []
    for t in (table, wild):
        ws = [torch.zeros(k, dtype=torch.uint8, device=DEV) for k in (
            gq.prefill_workspace_size(), gq.weights_workspace_size(B, C, 1), gq.evict_workspace_size(B, keep))]
        out = gq.gqa_prefill_paged(q, pool, t, starts, lens, kv_scales=psc, workspace=ws[0])
        w = gq.accumulate_weights_paged(q[:B], pool, t, lens, w0.clone(), kv_scales=psc, workspace=ws[1])
        p2, s2, l2 = pool.clone(), None if psc is None else psc.clone(), lens.clone()
        kept = gq.evict_kv_paged(p2, t, l2, w, keep, 5, 2, kv_scales=s2, workspace=ws[2])
        assert [gq.get_status(x) for x in ws] == [0, 0, 0]
        got.append([out, w, kept, p2.view(torch.uint8), l2])
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------- types of the bytes


def test_float8_types(library):  # noqa: F811
    """A cache of torch.float8_e4m3fn, and e2m1 scales of it, as the same bytes in uint8."""
    i32 = dict(dtype=torch.int32, device=DEV)
    lens, starts = torch.tensor([200, 77], **i32), torch.tensor([0, 30, 100], **i32)
    q = torch.randn((100, HQ, D), generator=gen(95), device=DEV).to(torch.bfloat16)
    for fmt in ("e4m3", "e2m1"):
        kv, sc = new_cache(fmt, 2, 200, 94)
        w0 = torch.rand((2, HKV, 200), generator=gen(96), device=DEV)
        got = []
        for as8 in (False, True):
            f8 = torch.float8_e4m3fn
            x = kv.view(f8) if as8 and fmt == "e4m3" else kv
            s = sc.view(f8) if as8 and sc is not None else sc
            out = gq.gqa_prefill(q, x, starts, lens, kv_scales=s)
            w = gq.accumulate_weights(q[:2], x, lens, w0.clone(), kv_scales=s)
            y, ys = torch.zeros_like(x[:, :, :, :50]), None if s is None else torch.zeros_like(s[:, :, :, :50])
            ol = torch.zeros_like(lens)
            kept = gq.evict_kv(x, lens, w, 50, 5, 2, out=y, out_scales=ys, out_lengths=ol, kv_scales=s)
            got.append([out, w, y.view(torch.uint8), kept, ol] + ([] if ys is None else [ys.view(torch.uint8)]))
            if as8 and fmt == "e4m3":
                with pytest.raises(ValueError):
                    gq.evict_kv(x, lens, w, 50, 5, 2, out=torch.zeros_like(kv[:, :, :, :50]), out_lengths=ol)
        for a, b in zip(*got):
            assert torch.equal(a, b)

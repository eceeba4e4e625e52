"""Prompt attention, draft verification, weight sums and eviction against their
definitions in 64 bits (GPU), on the product and on the range-checked library.

Bounds, each derived from the arithmetic and not from a run:
  scores    the products of 16-bit values are exact in FP32; 128 of them are added,
            each addition off by 2^-23 of the sum of their magnitudes m at most (the
            tensor cores cut where FP32 rounds), so |ds| <= 2^-16 m, and the scaling
            adds 2^-22 |s|
  weights   exp(s - max) / sum is off by 2 |ds| (its own score and the sum's) and
            2^-19 (exp2, the sum, the division)
  outputs   those, half a step of q's type for the weight where it meets V, all times
            sum of weight * |V|, and half a step of the output's type.  Where the weights
            are fp16 (any cache but a bf16 one) they lie on the grid of 2^-24 below its
            normal numbers: off by 2^-25 at most, where the largest weight is 2^7 or more
            (the running maximum never lies above the row's), so the outputs by 2^-32
            times the sum of |V| over the slots.  int8: the weights are held times the V
            scales, with the largest one's power of two above it in the maximum, so by
            2^-31 times the largest scale times the sum of |codes|
  tokens, lengths, kept slots and moved rows: equal
"""
import math

import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import _lib

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
TD = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HQ, HKV, D = 32, 8, 128
SCALE = {"e4m3": (0.03125, 0.046875), "e2m1": (0.4, 0.7)}


@pytest.fixture(scope="module", params=["product", "checked"], autouse=True)
def library(request):
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


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def new_cache(fmt, units, rows, seed=0):
    g = gen(seed + 17)
    shape = (units, 2, HKV, rows, 64 if fmt == "e2m1" else D)
    if fmt in TD:
        return torch.randn(shape, generator=g, device=DEV).to(TD[fmt]), None
    if fmt == "e4m3":
        return (4 * torch.randn(shape, generator=g, device=DEV)).to(torch.float8_e4m3fn).view(torch.uint8), None
    if fmt == "i8":
        kv = torch.randint(-127, 128, shape, generator=g, device=DEV).to(torch.int8)
        return kv, (0.002 + 0.02 * torch.rand(shape[:4], generator=g, device=DEV)).to(torch.bfloat16)
    kv = torch.randint(0, 256, shape, generator=g, device=DEV).to(torch.uint8)
    sc = (0.5 * torch.rand((*shape[:4], 8), generator=g, device=DEV)).to(torch.float8_e4m3fn).view(torch.uint8)
    return kv, sc


def values(kv, sc, fmt, scale):
    """Rows in 64 bits."""
    if fmt in TD:
        return kv.double()
    if fmt == "e4m3":
        return kv.view(torch.float8_e4m3fn).double() * scale
    if fmt == "i8":
        return kv.double() * sc.double()[..., None]
    level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    level = torch.cat((level, -level))
    x = torch.stack((level[(kv & 15).long()], level[(kv >> 4).long()]), -1).flatten(-2)
    return x * sc.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1) * scale


def paged(kv, sc, page, batch, capacity, seed=0):
    """The cache in shuffled pages with spare ones: (pages, scale pages, block table)."""
    per = capacity // page
    n = batch * per
    order = torch.randperm(n + 3, generator=gen(seed + 5), device=DEV)[:n]

    def scatter(x):
        if x is None:
            return None
        x = x.unflatten(3, (per, page)).movedim(3, 1).flatten(0, 1)  # [B * per, 2, 8, page, ...]
        out = torch.zeros((n + 3, *x.shape[1:]), dtype=x.dtype, device=DEV)
        out[order] = x
        return out
    return scatter(kv), scatter(sc), order.to(torch.int32).view(batch, per).contiguous()


def scale_of(fmt):
    return SCALE.get(fmt, (1.0, 1.0))


def check_flags(ws, library, want=0):
    assert gq.get_status(ws) == want


# ------------------------------------------------------------------ prefill


def attend64(q, K, V, end):
    """One query token's heads over slots [0, end): output, sum of weight * |V|, score error bound."""
    o, a, e = (torch.zeros((HQ, D), dtype=torch.float64, device=DEV) for _ in range(3))
    if end > 0:
        k, v = (x[:, :end].repeat_interleave(4, 0) for x in (K, V))
        s = torch.einsum("hd,htd->ht", q.double(), k) / math.sqrt(128.0)
        m = torch.einsum("hd,htd->ht", q.double().abs(), k.abs()).amax(-1) / math.sqrt(128.0)
        w = torch.softmax(s, -1)
        o, a = torch.einsum("ht,htd->hd", w, v), torch.einsum("ht,htd->hd", w, v.abs())
        e = (2 ** -16 * m + 2 ** -22 * s.abs().amax(-1))[:, None].expand(HQ, D)
    return o, a, e


def prefill_case(fmt, dtype, rows, capacity, page=0, seed=0, pad=3, q_scale=1.0, mag=1.0, sample=None, edit=None):
    """rows: (n, length) of each batch row."""
    B = len(rows)
    kv, sc = new_cache(fmt, B, capacity, seed)
    ks, vs = scale_of(fmt)
    if edit:
        edit(kv, sc)
    K, V = (values(kv[:, p], None if sc is None else sc[:, p], fmt, s) for p, s in ((0, ks), (1, vs)))
    n = [r[0] for r in rows]
    starts = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32, device=DEV)
    lens = torch.tensor([r[1] for r in rows], dtype=torch.int32, device=DEV)
    N = sum(n)
    q = (mag * torch.randn((N + pad, HQ, D), generator=gen(seed + 1), device=DEV)).to(TD[dtype])
    out = torch.full_like(q, 7.0)
    ws = torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    how = dict(q_scale=q_scale, k_scale=ks, v_scale=vs, out=out, workspace=ws)
    if page:
        pool, pool_sc, table = paged(kv, sc, page, B, capacity, seed)
        gq.gqa_prefill_paged(q, pool, table, starts, lens, kv_scales=pool_sc, **how)
    else:
        gq.gqa_prefill(q, kv, starts, lens, kv_scales=sc, **how)
    torch.cuda.synchronize()
    assert (out[N:] == 7.0).all(), "rows behind the last chunk changed"
    half = torch.finfo(TD[dtype]).eps / 2
    tiny = torch.finfo(TD[dtype]).tiny
    at = 0
    for b, (nb, L) in enumerate(rows):
        picks = range(nb) if sample is None or nb <= sample else sorted({0, nb - 1, *torch.randint(
            0, nb, (sample,), generator=torch.Generator().manual_seed(seed + b)).tolist()})
        for j in picks:
            ref, a, e = attend64(q[at + j] * q_scale, K[b], V[b], L - nb + j + 1)
            grid = 0.0 if fmt == "bf16" else 2 ** -31 * L * float(127 * sc[b, 1].abs().max() if fmt == "i8" else V[b].abs().max())
            bound = half * ref.abs() + (half + 2 * e + 2 ** -18) * a + tiny * half + grid
            err = (out[at + j].double() - ref).abs()
            assert (err <= bound).all(), \
                f"row {b} query {j}: worst {float((err / bound).max()):.3f} of the bound, {float(err.max()):.3e}"
        at += nb
    return ws


FORMATS = [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f16"), ("i8", "bf16"), ("i8", "f16"),
           ("e2m1", "bf16"), ("e2m1", "f16")]


@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("fmt,dtype", FORMATS)
def test_prefill_formats(library, fmt, dtype, page):
    rows = [(1, 1), (5, 5), (0, 17), (33, 100), (64, 64), (70, 384), (3, 384), (129, 257)]
    ws = prefill_case(fmt, dtype, rows, 384, page)
    check_flags(ws, library)


@pytest.mark.parametrize("rows", [
    [(1, 1)], [(1, 2000)], [(2, 130)], [(31, 31)], [(32, 128)], [(33, 129)], [(63, 640)], [(64, 1000)], [(65, 1001)],
    [(127, 127)], [(128, 255)], [(300, 300)], [(0, 0), (0, 5), (7, 9)], [(1, 1)] * 40, [(17, 1024)],
    [(513, 2049), (0, 2049), (1, 1), (700, 700), (256, 1999)]])
@pytest.mark.parametrize("fmt", ["f16", "bf16", "i8"])
def test_prefill_sizes(library, fmt, rows):
    prefill_case(fmt, "bf16" if fmt == "bf16" else "f16", rows, 2049, sample=40)


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("f16", "f16"), ("e2m1", "bf16")])
def test_prefill_long(library, fmt, dtype):
    # few tokens over a long row, many over a medium one: rows cut into pieces and merged
    prefill_case(fmt, dtype, [(40, 40000), (1500, 6000), (2, 30001)], 40000, sample=10, seed=3)
    prefill_case(fmt, dtype, [(100, 32768)], 32768, page=256, sample=10, seed=4)


# ------------------------------------------------------------------- drafts


def drafts64(p, d, u, q, lens):
    """The definition with whole numbers of the interpreter."""
    B, T, V = p.shape
    tokens, accepted, out = [], [], []
    for b in range(B):
        taken, row = [], None
        for j in range(T - 1):
            t = int(d[b, j])
            if not 0 <= t < V:
                break
            qd = 1.0 if q is None else float(q[b, j, t])
            if float(u[b, j]) * qd < float(p[b, j, t]):
                taken.append(t)
                row = None
            else:
                row = torch.zeros(V, device=p.device) if q is None else q[b, j].float()
                if q is None:
                    row[t] = math.inf
                break
        pn = p[b, len(taken)].float()

        def whole(x):
            x = torch.nan_to_num(x, nan=0.0).clamp(0, 1)
            return (x.double() * 2.0 ** 38).round().long().tolist()
        w = whole(pn) if row is None else whole(pn - row)
        if not any(w):
            w = whole(pn)
        total, k = sum(w), int(min(max(math.floor(float(u[b, -1]) * 2 ** 24), 0), 2 ** 24 - 1))
        target, acc, pick = (total * k) >> 24, 0, -1
        for i, x in enumerate(w):
            acc += x
            if acc > target:
                pick = i
                break
        n = len(taken)
        tokens.append(taken + [pick] + [-1] * (T - 1 - n))
        accepted.append(n)
        out.append(max(int(lens[b]) - (T - 1) + n, 0))
    return tokens, accepted, out


def draft_inputs(B, T, V, dtype, seed=0, sharp=2.5):
    g = gen(seed)
    p = torch.softmax(sharp * torch.randn((B, T, V), generator=g, device=DEV), -1)
    q = torch.softmax(torch.log(p[:, :T - 1].clamp(min=1e-30)) + 0.8 * torch.randn((B, T - 1, V), generator=g, device=DEV), -1)
    e = -torch.log1p(-torch.rand((B, T - 1, V), generator=g, device=DEV))
    d = (q / e.clamp(min=1e-30)).argmax(-1).to(torch.int32) if T > 1 else torch.zeros((B, 0), dtype=torch.int32, device=DEV)
    u = torch.rand((B, T), generator=g, device=DEV)
    return p.to(TD[dtype]), d.contiguous(), u, q.to(TD[dtype]), torch.randint(T, 999, (B,), generator=g, device=DEV, dtype=torch.int32)


def check_drafts(p, d, u, q, lens):
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    new = torch.zeros_like(lens)
    tokens, accepted = gq.verify_drafts(p, d, u, draft_probs=q, sequence_lengths=lens, out_lengths=new, workspace=ws)
    want = drafts64(p, d, u, q, lens)
    assert accepted.tolist() == want[1]
    assert tokens.tolist() == want[0]
    assert new.tolist() == want[2]
    return gq.get_status(ws)


@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,V", [(1, 4, 32000), (3, 2, 1), (5, 3, 2), (9, 4, 37), (4, 1, 1000), (2, 8, 4097), (7, 5, 50001),
                                   (3, 32, 300), (2, 3, 200003)])
def test_drafts(library, B, T, V, dtype, greedy):
    p, d, u, q, lens = draft_inputs(B, T, V, dtype, seed=V + T)
    if T > 2:
        d[0, 1] = -1
    assert check_drafts(p, d, u, None if greedy else q, lens) == 0


def test_drafts_strided_and_in_place(library):
    p, d, u, q, lens = draft_inputs(6, 4, 1003, "f32", seed=5)
    wide = torch.full((6, 4, 1024), 9.0, device=DEV)
    wide[..., :1003] = p
    wide_q = torch.full((6, 5, 1029), 9.0, device=DEV)
    wide_q[:, 1:4, 2:1005] = q
    want = drafts64(p, d, u, q, lens)
    tokens, accepted = gq.verify_drafts(wide[..., :1003], d, u, draft_probs=wide_q[:, 1:4, 2:1005], sequence_lengths=lens)
    assert tokens.tolist() == want[0] and accepted.tolist() == want[1] and lens.tolist() == want[2]


def test_drafts_edges(library):
    V = 5000
    p, d, u, q, lens = draft_inputs(12, 4, V, "f32", seed=6)
    p[0, :, :] = 0
    p[0, :, 4999] = 1.0      # a target that is sure of the last token
    p[1] = float("nan")      # nothing to draw from
    p[2, 0] = q[2, 0]        # p = q: a refusal leaves nothing beside q
    u[2, 0] = 0.99999994
    q[2, 0, d[2, 0]] *= 1.5
    p[3, :, 7] = float("nan")
    q[4] = 0                 # a draft that its model never draws
    u[5] = 0
    u[6] = 1 - 2 ** -24
    d[7, 0] = -1             # no draft at all
    d[8, 2] = -5
    p[9] = 0
    p[9, :, 3] = 2 ** -39    # below half a unit (ties to even: 0)
    p[10] = 1e-12
    lens[11] = 2             # shorter than what is taken back
    assert check_drafts(p, d, u, q, lens) == 0
    d[0, 0] = V
    assert check_drafts(p, d, u, q, lens) == gq.api.FLAG_SLOT_CLAMPED


# ------------------------------------------------------------------ weights


def weights64(q, K, L, T):
    """[8, L] sums and their score error bounds."""
    w, e = torch.zeros((HKV, L), dtype=torch.float64, device=DEV), torch.zeros((HKV, L), dtype=torch.float64, device=DEV)
    for j in range(T):
        n = L - T + 1 + j
        if n < 1:
            continue
        k = K[:, :n].repeat_interleave(4, 0)
        s = torch.einsum("hd,htd->ht", q[j].double(), k) / math.sqrt(128.0)
        m = torch.einsum("hd,htd->ht", q[j].double().abs(), k.abs()).amax(-1, keepdim=True) / math.sqrt(128.0)
        x = torch.softmax(s, -1)
        ds = 2 ** -16 * m + 2 ** -22 * s.abs().amax(-1, keepdim=True)
        w[:, :n] += x.view(HKV, 4, n).sum(1)
        e[:, :n] += (x * (2 * ds + 2 ** -19)).view(HKV, 4, n).sum(1)
    return w, e


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("fmt,dtype", FORMATS)
def test_weights(library, fmt, dtype, T, page):
    B, C = 5, 640
    kv, sc = new_cache(fmt, B, C, 2)
    ks, _ = scale_of(fmt)
    lens = torch.tensor([640, 1, 0, 129, 333], dtype=torch.int32, device=DEV)
    q = torch.randn((B, T, HQ, D), generator=gen(3), device=DEV).to(TD[dtype])
    K = values(kv[:, 0], None if sc is None else sc[:, 0], fmt, ks)
    old = torch.rand((B, HKV, C), generator=gen(4), device=DEV)
    ws = torch.zeros(gq.weights_workspace_size(B, C, T), dtype=torch.uint8, device=DEV)
    how = dict(k_scale=ks, workspace=ws)
    for add in (True, False):
        acc = old.clone()
        if page:
            pool, psc, table = paged(kv, sc, page, B, C)
            gq.accumulate_weights_paged(q, pool, table, lens, acc, kv_scales=psc, add=add, **how)
        else:
            gq.accumulate_weights(q[:, 0].contiguous() if T == 1 else q, kv, lens, acc, kv_scales=sc, add=add, **how)
        for b, L in enumerate(lens.tolist()):
            assert torch.equal(acc[b, :, L:], old[b, :, L:])
            w, e = weights64(q[b], K[b], L, T)
            if add:
                w = w + old[b, :, :L].double()
                e = e + 2 ** -24 * w
            assert ((acc[b, :, :L].double() - w).abs() <= e + 2 ** -126).all()
    want = gq.api.FLAG_LENGTH_CLAMPED  # a row without a slot for each query
    assert gq.get_status(ws) == want


@pytest.mark.parametrize("fmt,dtype,B,C", [("bf16", "bf16", 1, 70001), ("e4m3", "bf16", 3, 9000), ("e2m1", "f16", 40, 258)])
def test_weights_sizes(library, fmt, dtype, B, C):
    kv, sc = new_cache(fmt, B, C, 5)
    ks, _ = scale_of(fmt)
    lens = torch.randint(4, C + 1, (B,), generator=gen(6), device=DEV, dtype=torch.int32)
    q = torch.randn((B, 2, HQ, D), generator=gen(7), device=DEV).to(TD[dtype])
    acc = torch.zeros((B, HKV, C), device=DEV)
    gq.accumulate_weights(q, kv, lens, acc, k_scale=ks, kv_scales=sc)
    for b in range(0, B, max(1, B // 5)):
        L = int(lens[b])
        K = values(kv[b, 0], None if sc is None else sc[b, 0], fmt, ks)
        w, e = weights64(q[b], K, L, 2)
        assert ((acc[b, :, :L].double() - w).abs() <= e + 2 ** -126).all()
        assert not acc[b, :, L:].any()


# ----------------------------------------------------------------- eviction


def kept64(w, L, keep, recent, first):
    """The kept slots of one head, by sorting."""
    if L <= keep:
        return list(range(L))
    vals = [-math.inf if x != x else x for x in w]
    isnan = [x != x for x in w]
    rest = sorted(range(first, L - recent), key=lambda t: (isnan[t], -vals[t], t))[:keep - first - recent]
    return sorted(list(range(first)) + rest + list(range(L - recent, L)))


def evict_inputs(fmt, B, C, seed=0, ties=True):
    kv, sc = new_cache(fmt, B, C, seed)
    w = torch.exp(2 * torch.randn((B, HKV, C), generator=gen(seed + 1), device=DEV)) / C
    if ties:  # sums of few values, zeros among them
        w = torch.where(torch.rand(w.shape, generator=gen(seed + 2), device=DEV) < 0.3, (w * C).floor() / C, w)
    return kv, sc, w


def check_evicted(fmt, kv, sc, w, lens, keep, recent, first, got_kv, got_sc, got_w, got_lens, kept, clean_w=True):
    for b, L in enumerate(lens.tolist()):
        n = min(L, keep)
        assert int(got_lens[b]) == n
        for h in range(HKV):
            at = kept64(w[b, h, :L].tolist(), L, keep, recent, first)
            assert kept[b, h].tolist() == at + [-1] * (keep - n)
            at = torch.tensor(at, dtype=torch.long, device=DEV)
            assert torch.equal(got_kv[b, :, h, :n].view(torch.uint8), kv[b, :, h][:, at].view(torch.uint8))
            if sc is not None:
                assert torch.equal(got_sc[b, :, h, :n], sc[b, :, h][:, at])
            if got_w is not None:
                assert torch.equal(got_w[b, h, :n], w[b, h, at])
                assert not got_w[b, h, n:L if not clean_w else None].any()


EVICTIONS = [  # batch, capacity, lengths, keep, recent, first
    (1, 1024, [1024], 512, 32, 4),
    (3, 300, [300, 0, 77], 77, 0, 0),
    (2, 200, [200, 133], 1, 0, 0),
    (2, 200, [199, 2], 1, 1, 0),
    (2, 640, [640, 500], 100, 60, 40),
    (1, 640, [639], 638, 5, 2),
    (2, 9000, [9000, 4097], 2050, 100, 1),
    (1, 40000, [39999], 10000, 7, 3),
]


@pytest.mark.parametrize("B,C,lens,keep,recent,first", EVICTIONS)
@pytest.mark.parametrize("fmt", ["f16", "e4m3", "i8", "e2m1"])
def test_evict_into_another(library, fmt, B, C, lens, keep, recent, first):
    if fmt != "f16" and C > 10000:
        pytest.skip("one format is enough for the long row")
    kv, sc, w = evict_inputs(fmt, B, C, seed=keep)
    before = [x.clone() for x in (kv, w)]
    lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, out_sc = new_cache(fmt, B, keep + 3, seed=99)
    fill = out.clone()
    out_w, out_lens = torch.full((B, HKV, keep + 5), 3.0, device=DEV), torch.full_like(lens, -1)
    ws = torch.zeros(gq.evict_workspace_size(B, keep), dtype=torch.uint8, device=DEV)
    kept = gq.evict_kv(kv, lens, w, keep, recent=recent, first=first, out=out, out_scales=out_sc, out_lengths=out_lens,
                       out_weights=out_w, kv_scales=sc, workspace=ws)
    assert gq.get_status(ws) == 0
    assert torch.equal(kv.view(torch.uint8), before[0].view(torch.uint8)) and torch.equal(w, before[1])
    check_evicted(fmt, kv, sc, w, lens, keep, recent, first, out, out_sc, out_w, out_lens, kept)
    for b, n in enumerate(out_lens.tolist()):
        assert torch.equal(out[b, :, :, n:].view(torch.uint8), fill[b, :, :, n:].view(torch.uint8))


@pytest.mark.parametrize("B,C,lens,keep,recent,first", EVICTIONS)
@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_evict_in_place(library, fmt, B, C, lens, keep, recent, first):
    kv, sc, w = evict_inputs(fmt, B, C, seed=keep + 1)
    lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    new_kv, new_sc, new_w, new_lens = (None if x is None else x.clone() for x in (kv, sc, w, lens))
    ws = torch.zeros(gq.evict_workspace_size(B, keep), dtype=torch.uint8, device=DEV)
    kept = gq.evict_kv(new_kv, new_lens, new_w, keep, recent=recent, first=first, kv_scales=new_sc, workspace=ws)
    assert gq.get_status(ws) == 0
    check_evicted(fmt, kv, sc, w, lens, keep, recent, first, new_kv, new_sc, new_w, new_lens, kept, clean_w=False)
    for b, L in enumerate(lens.tolist()):  # slots past the old length, and past the new one in the cache, as they were
        n = min(L, keep)
        assert torch.equal(new_w[b, :, L:], w[b, :, L:])
        assert torch.equal(new_kv[b, :, :, n:].view(torch.uint8), kv[b, :, :, n:].view(torch.uint8))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("fmt,page", [("bf16", 16), ("i8", 64), ("e2m1", 32)])
def test_evict_paged(library, fmt, page, in_place):
    B, C, keep, recent, first = 3, 64 * 20, 333, 40, 2
    kv, sc, w = evict_inputs(fmt, B, C, seed=7)
    lens = torch.tensor([C, 300, 1001], dtype=torch.int32, device=DEV)
    per = -(-keep // page)
    room = new_cache(fmt, B, C + per * page, seed=8)
    room[0][:, :, :, :C] = kv
    if sc is not None:
        room[1][:, :, :, :C] = sc
    pool, psc, table = paged(*room, page, B, C + per * page, seed=9)
    src, dst = table[:, :C // page].contiguous(), table[:, C // page:].contiguous()
    kept = torch.zeros((B, HKV, keep), dtype=torch.int32, device=DEV)
    if in_place:
        new_lens, new_w = lens.clone(), w.clone()
        gq.evict_kv_paged(pool, src, new_lens, new_w, keep, recent, first, kept=kept, kv_scales=psc)
        dst = src
    else:
        new_lens, new_w = torch.zeros_like(lens), torch.full((B, HKV, keep), 2.0, device=DEV)
        gq.evict_kv_paged(pool, src, lens, w, keep, recent, first, out_table=dst, out_lengths=new_lens,
                          out_weights=new_w, kept=kept, kv_scales=psc)

    def flat(x):
        return None if x is None else x[dst.long()].movedim(1, 3).flatten(3, 4)
    check_evicted(fmt, kv, sc, w, lens, keep, recent, first, flat(pool), flat(psc), new_w, new_lens, kept,
                  clean_w=not in_place)


def test_evict_special_weights(library):
    kv, sc, w = evict_inputs("f16", 1, 500, seed=3)
    w[0, 0, ::3] = float("nan")
    w[0, 1] = 0.0
    w[0, 1, ::2] = -0.0
    w[0, 2, 10:400] = float("inf")
    w[0, 3] = -w[0, 3]
    w[0, 4, ::5] = -float("inf")
    w[0, 5] = float("nan")
    w[0, 6] = torch.arange(500, device=DEV) * 1e-45
    lens = torch.tensor([500], dtype=torch.int32, device=DEV)
    out, ol = torch.zeros((1, 2, HKV, 250, D), dtype=torch.float16, device=DEV), torch.zeros_like(lens)
    kept = gq.evict_kv(kv, lens, w, 250, 10, 5, out=out, out_lengths=ol)
    for h in range(HKV):
        assert kept[0, h].tolist() == kept64(w[0, h].tolist(), 500, 250, 10, 5)


# ------------------------------------------- edges, and all of them together


def test_prefill_masked_values(library):
    """Infinities and NaN in slots that a query does not see never reach it; in slots
    that it sees they do, at every chunk size around the tiles' and units' edges."""
    for fmt, dtype in (("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e2m1", "f16")):
        n, L, C = 70, 300, 384
        kv, sc = new_cache(fmt, 1, C, 4)
        ks, vs = scale_of(fmt)
        bad = [L - n + 3, L - n + 40, L - 1]  # slots of the chunk itself
        for t in bad:
            if fmt in TD:
                kv[0, 1, :, t, 5] = float("nan") if t != L - 1 else float("inf")
            elif fmt == "e4m3":
                kv[0, 1, :, t, 5] = 0x7F
            else:
                sc[0, 1, :, t, 0] = 0x7F  # dims 0..15
        for plane in (0, 1):  # behind the length: anything
            if fmt in TD:
                kv[0, plane, :, L:] = float("nan")
            elif fmt == "e4m3":
                kv[0, plane, :, L:] = 0xFF
            else:
                sc[0, plane, :, L:] = 0x7F
        if fmt in TD:
            kv[0, 0, 2, L - 10] = float("nan")  # a key of one head
        q = torch.randn((n, HQ, D), generator=gen(5), device=DEV).to(TD[dtype])
        starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        lens = torch.tensor([L], dtype=torch.int32, device=DEV)
        out = gq.gqa_prefill(q, kv, starts, lens, k_scale=ks, v_scale=vs, kv_scales=sc)
        K, V = (values(kv[:, p], None if sc is None else sc[:, p], fmt, s)[0] for p, s in ((0, ks), (1, vs)))
        dims = range(16) if fmt == "e2m1" else (5,)
        for j in range(n):
            end = L - n + j + 1
            head_nan = fmt in TD and end > L - 10
            for d in dims:
                seen = [t for t in bad if t < end]
                col = out[j, :, d].float()
                want_nan = any(not (fmt in TD and t == L - 1) for t in seen)
                rows = [h for h in range(HQ) if not (head_nan and 8 <= h < 12)]
                if want_nan:
                    assert torch.isnan(col[rows]).all()
                elif seen:
                    assert torch.isposinf(col[rows]).all()
                else:
                    assert torch.isfinite(col[rows]).all()
            if head_nan:
                assert torch.isnan(out[j, 8:12].float()).all()
            clean = [d for d in range(D) if d not in dims]
            ref, a, e = attend64(q[j], torch.nan_to_num(K, nan=0.0, posinf=0.0), torch.nan_to_num(V, nan=0.0, posinf=0.0), end)
            rows = [h for h in range(HQ) if not (head_nan and 8 <= h < 12)]
            half = torch.finfo(TD[dtype]).eps / 2
            bound = half * ref.abs() + (half + 2 * e + 2 ** -18) * a + 2 ** -24
            err = (out[j].double() - ref).abs()
            assert (err[rows][:, clean] <= bound[rows][:, clean]).all()


@pytest.mark.parametrize("fmt,dtype", FORMATS)
def test_prefill_small_caches(library, fmt, dtype):
    # caches of fewer rows than a tile has, odd capacities
    prefill_case(fmt, dtype, [(1, 1)], 1, seed=11)
    prefill_case(fmt, dtype, [(2, 3), (3, 3), (0, 0)], 3, seed=12)
    prefill_case(fmt, dtype, [(40, 77)], 77, seed=13, q_scale=0.37)
    prefill_case(fmt, dtype, [(5, 16)], 16, page=16, seed=14, q_scale=0.0)


def test_prefill_many_rows(library):
    # more rows than a block has threads, most of them short, some without tokens
    rows = [((7 * b) % 3, 1 + (5 * b) % 40) for b in range(1000)]
    rows = [(min(n, L), L) for n, L in rows]
    prefill_case("bf16", "bf16", rows, 41, seed=15, sample=1)
    prefill_case("e4m3", "bf16", [(90, 100), (0, 100)] * 150, 100, seed=16, sample=1)


@pytest.mark.parametrize("fmt,dtype", [("f16", "f16"), ("bf16", "bf16"), ("i8", "bf16"), ("e4m3", "bf16")])
@pytest.mark.parametrize("mag", [1e-6, 30.0])
def test_prefill_magnitudes(library, fmt, dtype, mag):
    if dtype == "f16":
        mag = min(max(mag, 1e-3), 30.0)
    prefill_case(fmt, dtype, [(40, 300), (130, 130)], 300, seed=6, mag=mag, sample=20)


def test_prefill_scales_apart(library):
    """int8 rows whose V scales differ by powers of two over a tile, zero among them."""
    def edit(kv, sc):
        e = torch.randint(-30, 6, sc.shape[2:], generator=gen(1), device=DEV).float()
        sc[:, 1] = torch.exp2(e).to(torch.bfloat16)
        sc[:, 1, :, ::17] = 0
    prefill_case("i8", "bf16", [(60, 500)], 512, seed=7, sample=30, edit=edit)
    prefill_case("i8", "f16", [(60, 500)], 512, seed=7, sample=30, edit=lambda kv, sc: sc[:, 1].fill_(2.0 ** -20))


def test_prefill_out_of_contract(library):
    """Lengths and starts out of order are clamped and told; nothing outside is touched."""
    kv, _ = new_cache("bf16", 3, 256, 8)
    q = torch.randn((50, HQ, D), generator=gen(9), device=DEV).to(torch.bfloat16)
    ws = torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    out = torch.full_like(q, 3.0)
    starts = torch.tensor([-5, 20, 40, 60], dtype=torch.int32, device=DEV)
    lens = torch.tensor([10, 1000, -3], dtype=torch.int32, device=DEV)  # below its chunk, above the capacity, negative
    gq.gqa_prefill(q, kv, starts, lens, out=out, workspace=ws)
    assert gq.get_status(ws) == gq.api.FLAG_LENGTH_CLAMPED
    assert not out[:10].any() and not out[40:].any()  # queries without a slot: zero rows
    want = gq.gqa_prefill(q[10:40].contiguous(), kv, torch.tensor([0, 10, 30, 30], dtype=torch.int32, device=DEV),
                          torch.tensor([10, 256, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(out[10:40], want)
    pool, _, table = paged(kv, None, 64, 3, 256)
    table[1, 2] = 10 ** 6
    gq.gqa_prefill_paged(q, pool, table, torch.tensor([0, 0, 50, 50], dtype=torch.int32, device=DEV),
                         torch.full((3,), 256, dtype=torch.int32, device=DEV), out=out, workspace=ws)
    assert gq.get_status(ws) == gq.api.FLAG_PAGE_CLAMPED


def test_prefill_many_launches(library):
    """Launches back to back give the same bits each time and no wait runs out."""
    rows = [(0, 100), (513, 4000), (64, 64), (1, 4096), (300, 2000), (1024, 1024)]
    kv, _ = new_cache("bf16", len(rows), 4096, 10)
    n = torch.tensor([r[0] for r in rows])
    starts = torch.cat((torch.zeros(1, dtype=torch.int64), n.cumsum(0))).to(torch.int32).to(DEV)
    lens = torch.tensor([r[1] for r in rows], dtype=torch.int32, device=DEV)
    q = torch.randn((int(n.sum()), HQ, D), generator=gen(11), device=DEV).to(torch.bfloat16)
    ws = torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    first = gq.gqa_prefill(q, kv, starts, lens, workspace=ws)
    outs = [torch.empty_like(q) for _ in range(4)]
    for o in outs:
        o.copy_(first)
    for k in range(400):
        gq.gqa_prefill(q, kv, starts, lens, out=outs[k % 4], workspace=ws)
    assert gq.get_status(ws) == 0
    for o in outs:
        assert torch.equal(o, first)


def test_prefill_equals_decode(library):
    """One token a row: within the decode's own rounding of the decode call."""
    B, C = 5, 700
    kv, _ = new_cache("f16", B, C, 12)
    lens = torch.tensor([1, 700, 128, 129, 333], dtype=torch.int32, device=DEV)
    q = torch.randn((B, HQ, D), generator=gen(13), device=DEV).to(torch.float16)
    a = gq.gqa_prefill(q, kv, torch.arange(B + 1, dtype=torch.int32, device=DEV), lens)
    b = gq.gqa_decode(q, kv, lens)
    assert ((a.float() - b.float()).abs() <= 2 ** -9 * (1 + b.float().abs())).all()


def test_long_offsets(library):
    """Element offsets past 32 bits: the last rows of a large cache."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 40 GB")
    B, C = 9, 131072
    kv = torch.zeros((B, 2, HKV, C, D), dtype=torch.bfloat16, device=DEV)  # 4.8 GB, 2.4e9 elements
    kv[B - 1] = torch.randn((2, HKV, C, D), generator=gen(14), device=DEV).to(torch.bfloat16)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    lens[B - 1] = C
    starts = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    starts[B] = 33
    q = torch.randn((33, HQ, D), generator=gen(15), device=DEV).to(torch.bfloat16)
    out = gq.gqa_prefill(q, kv, starts, lens)
    K, V = kv[B - 1, 0].double(), kv[B - 1, 1].double()
    half = torch.finfo(torch.bfloat16).eps / 2
    for j in (0, 32):
        ref, a, e = attend64(q[j], K, V, C - 33 + j + 1)
        assert ((out[j].double() - ref).abs() <= half * ref.abs() + (half + 2 * e + 2 ** -18) * a + 2 ** -126).all()
    w = torch.zeros((B, HKV, C), device=DEV)
    gq.accumulate_weights(q[:B].contiguous(), kv, lens, w)
    ref, e = weights64(q[B - 1][None], K, C, 1)
    assert ((w[B - 1].double() - ref).abs() <= e + 2 ** -126).all()
    out_lens = lens.clone()
    small = torch.zeros((B, 2, HKV, 600, D), dtype=torch.bfloat16, device=DEV)
    kept = gq.evict_kv(kv, lens, w, 600, 8, 4, out=small, out_lengths=out_lens)
    for h in (0, 7):
        at = torch.tensor(kept64(w[B - 1, h].tolist(), C, 600, 8, 4), device=DEV)
        assert torch.equal(kept[B - 1, h].long(), at)
        assert torch.equal(small[B - 1, :, h], kv[B - 1, :, h][:, at])


def serving_state(fmt="bf16", dtype="bf16", B=4, C=512, seed=20):
    kv, sc = new_cache(fmt, B, C, seed)
    g = gen(seed + 1)
    n = 40
    return dict(kv=kv, sc=sc, B=B, C=C, q=torch.randn((B * n, HQ, D), generator=g, device=DEV).to(TD[dtype]),
                starts=torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV),
                lens=torch.tensor([512, 40, 300, 401][:B], dtype=torch.int32, device=DEV))


def run_together(s, ws):
    """A chunk attended, a window's weights summed, its drafts judged, the cache cut."""
    B, C = s["B"], s["C"]
    ks, vs = scale_of("e2m1") if s["sc"] is not None else (1.0, 1.0)
    out = gq.gqa_prefill(s["q"], s["kv"], s["starts"], s["lens"], k_scale=ks, v_scale=vs, kv_scales=s["sc"], out=ws["out"],
                         workspace=ws["prefill"])
    w = gq.accumulate_weights(s["q"].view(B, -1, HQ, D)[:, :2].contiguous(), s["kv"], s["lens"], ws["w"], k_scale=ks,
                              kv_scales=s["sc"], add=False, workspace=ws["weights"])
    tokens, accepted = gq.verify_drafts(ws["p"], ws["d"], ws["u"], draft_probs=ws["dq"], sequence_lengths=s["lens"],
                                        out_lengths=ws["len1"], tokens=ws["tokens"], accepted=ws["accepted"])
    kept = gq.evict_kv(s["kv"], ws["len1"], w, 100, 16, 4, out=ws["kv"], out_scales=ws["sc"], out_lengths=ws["len2"],
                       out_weights=ws["w2"], kept=ws["kept"], kv_scales=s["sc"], workspace=ws["evict"])
    return [out, w, tokens, accepted, ws["len1"], kept, ws["kv"], ws["len2"], ws["w2"]]


def together_buffers(s, seed=30):
    B, C = s["B"], s["C"]
    fmt = "e2m1" if s["sc"] is not None else "bf16"
    p, d, u, q, _ = draft_inputs(B, 3, 997, "f32", seed=seed)
    kv, sc = new_cache(fmt, B, 100, 40)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(out=torch.zeros_like(s["q"]), w=torch.zeros((B, HKV, C), device=DEV), p=p, d=d, u=u, dq=q,
                tokens=torch.zeros((B, 3), **i32), accepted=torch.zeros(B, **i32), len1=torch.zeros(B, **i32),
                len2=torch.zeros(B, **i32), kv=kv, sc=sc, w2=torch.zeros((B, HKV, 100), device=DEV),
                kept=torch.zeros((B, HKV, 100), **i32),
                prefill=torch.zeros(gq.prefill_workspace_size(), dtype=torch.uint8, device=DEV),
                weights=torch.zeros(gq.weights_workspace_size(B, C, 2), dtype=torch.uint8, device=DEV),
                evict=torch.zeros(gq.evict_workspace_size(B, 100), dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
def test_together_graphs_and_streams(library, fmt):
    s = serving_state(fmt)
    ws = together_buffers(s)
    want = [x.clone() for x in run_together(s, ws)]
    # the same through a captured graph, replayed after its inputs changed and back
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run_together(s, ws)
    q = s["q"].clone()
    s["q"].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got[0], want[0])
    s["q"].copy_(q)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # two streams at once, a set of buffers each, and the side streams' tensors made there
    other = [(torch.cuda.Stream(), together_buffers(s)) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, w in other:
            with torch.cuda.stream(st):
                run_together(s, w)
    torch.cuda.synchronize()
    for _, w in other:
        with torch.cuda.stream(torch.cuda.Stream()):
            again = run_together(s, w)
        torch.cuda.synchronize()
        for a, b in zip(again, want):
            assert torch.equal(a, b)


def test_chain(library):
    """A prompt written in two chunks and attended, a step's drafts judged and the lengths
    shortened, the weights summed over steps, the cache cut in place and decoded."""
    B, C, dt = 2, 640, torch.bfloat16
    g = gen(50)
    kv = torch.zeros((B, 2, HKV, C, D), dtype=dt, device=DEV)
    w_norm = torch.ones(D, dtype=dt, device=DEV)
    done = torch.zeros(B, dtype=torch.int32, device=DEV)
    for n in ([100, 33], [300, 200]):
        rows = torch.repeat_interleave(torch.arange(B), torch.tensor(n)).to(torch.int32).to(DEV)
        slots = torch.cat([torch.arange(k) for k in n]).to(torch.int32).to(DEV) + done[rows.long()]
        x = torch.randn((sum(n), HQ + 2 * HKV, D), generator=g, device=DEV).to(dt)
        q = gq.write_kv(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], w_norm, w_norm, slots, rows, slots, kv)
        done = done + torch.tensor(n, dtype=torch.int32, device=DEV)
        starts = torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device=DEV)
        out = gq.gqa_prefill(q, kv, starts, done)
        half = torch.finfo(dt).eps / 2
        for b in range(B):
            for j in (0, n[b] - 1):
                i = int(starts[b]) + j
                ref, a, e = attend64(q[i], kv[b, 0].double(), kv[b, 1].double(), int(done[b]) - n[b] + j + 1)
                assert ((out[i].double() - ref).abs() <= half * ref.abs() + (half + 2 * e + 2 ** -18) * a + 2 ** -126).all()
    weights = torch.zeros((B, HKV, C), device=DEV)
    total = torch.zeros((B, HKV, C), dtype=torch.float64, device=DEV)
    bound = total.clone()
    for step in range(3):
        qs = torch.randn((B, 1, HQ, D), generator=g, device=DEV).to(dt)
        gq.accumulate_weights(qs, kv, done, weights)
        for b in range(B):
            L = int(done[b])
            x, e = weights64(qs[b], kv[b, 0].double(), L, 1)
            total[b, :, :L] += x
            bound[b, :, :L] += e + 2 ** -23 * total[b, :, :L]
    assert ((weights.double() - total).abs() <= bound + 2 ** -126).all()
    before, old, lens0 = kv.clone(), weights.clone(), done.clone()
    kept = gq.evict_kv(kv, done, weights, 128, recent=32, first=4)
    check_evicted("bf16", before, None, old, lens0, 128, 32, 4, kv, None, weights, done, kept, clean_w=False)
    q1 = torch.randn((B, HQ, D), generator=g, device=DEV).to(dt)
    o = gq.gqa_decode(q1, kv, done)
    for b in range(B):
        k, v = (torch.stack([before[b, p, h][kept[b, h].long()] for h in range(HKV)]).double() for p in (0, 1))
        ref, _, _ = attend64(q1[b], k, v, 128)
        assert ((o[b].double() - ref).abs() <= 3e-2 * (1 + ref.abs())).all()


def test_refusals(library):
    kv, _ = new_cache("bf16", 2, 64, 60)
    q = torch.zeros((10, HQ, D), dtype=torch.bfloat16, device=DEV)
    starts = torch.tensor([0, 5, 10], dtype=torch.int32, device=DEV)
    lens = torch.tensor([64, 64], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        gq.gqa_prefill(q, kv, starts[:2], lens)
    with pytest.raises(ValueError):
        gq.gqa_prefill(q.view(10, HQ // 2, 2 * D), kv, starts, lens)
    with pytest.raises(gq.GqaError, match="dtype of q"):
        gq.gqa_prefill(q.half(), kv, starts, lens)
    with pytest.raises(gq.GqaError, match="WORKSPACE"):
        gq.gqa_prefill(q, kv, starts, lens, workspace=torch.zeros(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(gq.GqaError, match="overlaps"):
        gq.gqa_prefill(q, kv, starts, lens, out=q)
    with pytest.raises(gq.GqaError, match="q_scale"):
        gq.gqa_prefill(q, kv, starts, lens, q_scale=float("nan"))
    assert gq.gqa_prefill(q[:0], kv, torch.zeros_like(starts), lens).shape == (0, HQ, D)
    p, d, u, dq, n = draft_inputs(2, 3, 50, "f32")
    for bad in (dict(drafts=d[:, :1].contiguous()), dict(uniforms=u.double()), dict(draft_probs=dq.half()),
                dict(out_lengths=n), dict(probs=p.transpose(1, 2))):
        with pytest.raises(ValueError):
            gq.verify_drafts(**{**dict(probs=p, drafts=d, uniforms=u), **bad})
    with pytest.raises(gq.GqaError, match="strides"):
        gq.verify_drafts(p[:1].expand(2, 3, 50), d, u)
    w = torch.zeros((2, HKV, 64), device=DEV)
    with pytest.raises(ValueError):
        gq.accumulate_weights(q[:2], kv, lens, w[:, :, :32])
    with pytest.raises(ValueError):
        gq.accumulate_weights(q.view(2, 5, HQ, D), kv, lens, w)
    with pytest.raises(gq.GqaError, match="first and recent"):
        gq.evict_kv(kv, lens, w, 10, recent=8, first=4)
    with pytest.raises(ValueError):
        gq.evict_kv(kv, lens, w, 10, out_lengths=lens)
    with pytest.raises(ValueError):
        gq.evict_kv(kv, lens, w, 10, out=torch.zeros_like(kv))
    with pytest.raises(gq.GqaError, match="slots a row"):
        gq.evict_kv(kv, lens, w, 10, out=torch.zeros_like(kv[:, :, :, :8]).contiguous(), out_lengths=lens.clone())
    with pytest.raises(gq.GqaError, match="overlaps"):
        gq.evict_kv(kv, lens, w, 10, out=kv, out_lengths=lens.clone())
    with pytest.raises(gq.GqaError, match="overlaps"):
        gq.evict_kv(kv, lens, w, 10, out=torch.zeros_like(kv), out_lengths=lens)


def test_weights_nan_key(library):
    """A NaN key makes every weight of the rows that see it NaN, and hidden slots' none."""
    for C in (300, 40000):  # on chip and in two launches
        kv, _ = new_cache("f16", 1, C, 61)
        kv[0, 0, 3, C - 2] = float("nan")
        q = torch.randn((1, 2, HQ, D), generator=gen(62), device=DEV).half()
        q[0, :, 12] *= 40  # (weights that underflow beside the largest)
        lens = torch.tensor([C - 1], dtype=torch.int32, device=DEV)  # the last slot is behind the length
        w = gq.accumulate_weights(q, kv, lens, torch.zeros((1, HKV, C), device=DEV))
        assert torch.isfinite(w[0, [0, 1, 2, 4, 5, 6, 7]]).all() and w[0, 3, C - 1] == 0
        assert torch.isnan(w[0, 3, :C - 1]).all()  # token 1 sees the NaN key
        lens.fill_(C - 2)  # now no token sees it
        w = gq.accumulate_weights(q, kv, lens, torch.zeros((1, HKV, C), device=DEV))
        assert torch.isfinite(w).all()

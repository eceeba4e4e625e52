"""What the prompt attention, the draft verification and the cache eviction are measured on.

Four kinds of pass, over 32 query heads, 8 KV heads and head_dim 128:

  prefill  attention of chunks of new tokens over a cache of any format,
           contiguous or paged; the chunks of the rows lie one behind another
           in q, and a chunk's tokens are the last slots of its row
  drafts   drafted tokens accepted or refused against the target's
           probabilities, and the next token drawn, from given random numbers
  weights  the softmax weight that every slot of a cache gets from a step's
           queries, summed for each KV head
  evict    the slots of a cache with the largest such sums moved together
           into a smaller cache, the newest and the first ones always among
           them (from a 4-bit cache: read back to 16 bits after that)

A 4-bit row is 64 bytes: byte j holds dims 2j (low nibble) and 2j + 1 (high
nibble) as e2m1 codes; kv_scales holds 8 e4m3 scales a row.
"""
import math

import torch

own = False

HQ, HKV, D, GROUP = 32, 8, 128, 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# the scales of all keys and of all values that a program has from its calibration
SCALES = {"fp4": (10 / 1024, 9 / 1024), "e4m3": (1 / 32, 1 / 32)}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # a short question put to a short context: latency
        {"name": "prefill 17 of 1024", "kind": "prefill", "dtype": "f16", "fmt": "f16", "batch": 1, "capacity": 1024,
         "n_lo": 17, "n_hi": 17, "len_lo": 1024, "len_hi": 1024, "page": 0},
        # a whole prompt into an empty cache
        {"name": "prefill 8192 of 8192", "kind": "prefill", "dtype": "bf16", "fmt": "bf16", "batch": 1,
         "capacity": 8192, "n_lo": 8192, "n_hi": 8192, "len_lo": 8192, "len_hi": 8192, "page": 0},
        # a serving step of ragged chunks, one row without new tokens
        {"name": "prefill 16 ragged of 8192", "kind": "prefill", "dtype": "f16", "fmt": "f16", "batch": 16,
         "capacity": 8192, "n_lo": 0, "n_hi": 1023, "len_lo": 1023, "len_hi": 8191, "page": 0},
        # one chunk of a long prompt over its long prefix in pages
        {"name": "prefill 512 of 131072 paged", "kind": "prefill", "dtype": "bf16", "fmt": "bf16", "batch": 1,
         "capacity": 131072, "n_lo": 512, "n_hi": 512, "len_lo": 131072, "len_hi": 131072, "page": 256},
        # chunks of four prompts over a paged 4-bit cache
        {"name": "prefill fp4 4x1024 of 16384 paged", "kind": "prefill", "dtype": "bf16", "fmt": "fp4", "batch": 4,
         "capacity": 16384, "n_lo": 1024, "n_hi": 1024, "len_lo": 8192, "len_hi": 16384, "page": 64},
        # one request's drafts, drawn greedily: latency
        {"name": "drafts 1x3 of 32000", "kind": "drafts", "dtype": "f32", "batch": 1, "window": 4, "vocab": 32000,
         "greedy": True},
        # a serving batch's drafts with the probabilities that they were drawn from
        {"name": "drafts 64x3 of 131072", "kind": "drafts", "dtype": "f32", "batch": 64, "window": 4, "vocab": 131072,
         "greedy": False},
        # a short context's step: latency
        {"name": "weights 1x1024", "kind": "weights", "dtype": "f16", "fmt": "f16", "batch": 1, "capacity": 1024,
         "len_lo": 1024, "len_hi": 1024, "q_len": 1, "page": 0},
        # a full serving batch over a paged 8-bit cache
        {"name": "weights e4m3 64x32768 paged", "kind": "weights", "dtype": "bf16", "fmt": "e4m3", "batch": 64,
         "capacity": 32768, "len_lo": 16384, "len_hi": 32768, "q_len": 1, "page": 256},
        # a short context cut to half: latency
        {"name": "evict 1x1024 to 512", "kind": "evict", "dtype": "f16", "fmt": "f16", "batch": 1, "capacity": 1024,
         "len_lo": 1024, "len_hi": 1024, "keep": 512, "recent": 32, "first": 4, "page": 0},
        # long prompts cut to a quarter
        {"name": "evict 8x32768 to 8192", "kind": "evict", "dtype": "bf16", "fmt": "bf16", "batch": 8,
         "capacity": 32768, "len_lo": 16385, "len_hi": 32767, "keep": 8192, "recent": 256, "first": 4, "page": 0},
        # a serving batch over a paged 4-bit cache, rows that are shorter than what is kept among them
        {"name": "evict fp4 32x8192 to 1001 paged", "kind": "evict", "dtype": "bf16", "fmt": "fp4", "batch": 32,
         "capacity": 8192, "len_lo": 0, "len_hi": 8192, "keep": 1001, "recent": 64, "first": 0, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "prefill", "drafts", "weights", "evict"])
    dtype = rng.choice(["f16", "bf16"])
    if kind == "drafts":
        vocab = _log(rng, 1000, 200000)
        return {"kind": kind, "dtype": rng.choice(["f32", "f32", dtype]), "batch": _log(rng, 1, min(128, (1 << 23) // vocab)),
                "window": rng.choice([1, 2, 3, 4, 8]), "vocab": vocab, "greedy": rng.random() < 0.4}
    page = rng.choice([0, 16, 64, 256])
    batch = _log(rng, 1, 32)
    fmt = rng.choice([dtype, dtype, "fp4", "i8", "e4m3"])
    capacity = _log(rng, 64, max(64, min(131072, (1 << 19) // batch)))
    capacity = -(-capacity // (page or 2)) * (page or 2)
    hi = rng.randint(1, capacity)
    case = {"kind": kind, "dtype": dtype, "fmt": fmt, "batch": batch, "capacity": capacity, "len_hi": hi,
            "len_lo": rng.choice([hi, hi // 2, 0]), "page": page}
    if kind == "prefill":
        n = min(hi, _log(rng, 1, max(1, min(4096, (1 << 24) // (batch * hi)))))
        case.update(n_lo=rng.choice([n, 0]), n_hi=n)
    elif kind == "weights":
        case["q_len"] = rng.choice([1, 1, 2, 3, 4])
    else:
        keep = _log(rng, 1, capacity)
        case.update(keep=keep, recent=rng.randint(0, keep // 2), first=rng.choice([0, min(4, keep // 2)]))
    return case


def _between(lo, hi, n, seed):
    return torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed))


def _sizes(case, seed):
    """(lengths, chunk sizes) of the rows of a case over a cache, on the host."""
    B = case["batch"]
    lens = _between(case["len_lo"], case["len_hi"], B, seed)
    if case["len_lo"] == 0 and B > 1:
        lens[B // 2] = 0
    if case["kind"] != "prefill":
        return lens, None
    n = torch.minimum(_between(case["n_lo"], case["n_hi"], B, seed + 1), lens)
    if case["n_lo"] == 0 and B > 1:
        n[B // 3] = 0
    return lens, n


def _row_bytes(fmt):
    return {"f16": 256, "bf16": 256, "e4m3": 128, "i8": 130, "fp4": 72}[fmt]


def work(case):
    kind, B = case["kind"], case["batch"]
    if kind == "drafts":
        width = {"f32": 4, "f16": 2, "bf16": 2}[case["dtype"]]
        return {"bytes": B * case["vocab"] * width * (1 if case["greedy"] else 2), "flops": 3 * B * case["vocab"]}
    mean = (case["len_lo"] + case["len_hi"]) / 2
    if kind == "prefill":
        n = min(mean, (case["n_lo"] + case["n_hi"]) / 2)
        seen = n * (mean - n) + n * (n + 1) / 2  # slots that a row's queries attend
        return {"bytes": B * (mean * 16 * _row_bytes(case["fmt"]) + 2 * n * HQ * D * 2),
                "flops": 4 * B * seen * HQ * D}
    if kind == "weights":
        return {"bytes": B * mean * HKV * (_row_bytes(case["fmt"]) + 4) + B * case["q_len"] * HQ * D * 2,
                "flops": 2 * B * mean * case["q_len"] * HQ * D}
    kept = min(mean, case["keep"])
    moved = 2 * B * kept * 16 * _row_bytes(case["fmt"]) + B * HKV * (4 * mean + 12 * kept)
    if case["fmt"] in SCALES or case["fmt"] == "i8":
        moved += B * kept * 16 * (_row_bytes(case["fmt"]) + 256)
    return {"bytes": moved, "flops": B * HKV * mean}


# ------------------------------------------------------------------ inputs


def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(seed * 1009 + k)


def _randn(shape, seed, k, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed, k), device="cuda", dtype=dtype)


def _quantise(x, fmt, scale):
    """(codes, scales) of rows x [..., 128]; `scale` is the one of all of them."""
    if fmt == "fp4":
        g = (x / scale).unflatten(-1, (D // GROUP, GROUP))
        s = (g.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
        wide = s.to(x.dtype).unsqueeze(-1)
        t = torch.where(wide > 0, g / wide, torch.zeros_like(g))
        m = t.abs().clamp(max=6)
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).to(x.dtype)
        m = (m / step).round() * step
        c = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
        c = (c | ((t < 0).to(torch.uint8) << 3)).flatten(-2)
        return c[..., 0::2] | (c[..., 1::2] << 4), s.view(torch.uint8)
    if fmt == "i8":
        s = (x.abs().amax(-1) / 127).to(torch.bfloat16)
        return (x / s.to(x.dtype).unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8), s
    if fmt == "e4m3":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), None
    return x.to(TYPES[fmt]), None


def _values(codes, scales, fmt, scale):
    """The rows that codes and scales stand for, in 32 bits."""
    if fmt == "fp4":
        n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        m = (n & 7).to(torch.float32)
        m = torch.where(m < 4, 0.5 * m, torch.where(m < 6, m - 2, 2 * m - 8))
        x = torch.where(n > 7, -m, m).unflatten(-1, (D // GROUP, GROUP))
        return (x * (scales.view(torch.float8_e4m3fn).to(torch.float32) * scale).unsqueeze(-1)).flatten(-2)
    if fmt == "i8":
        return codes.to(torch.float32) * scales.to(torch.float32).unsqueeze(-1)
    if fmt == "e4m3":
        return codes.view(torch.float8_e4m3fn).to(torch.float32) * scale
    return codes.to(torch.float32)


def _empty_cache(fmt, units, rows):
    width = 64 if fmt == "fp4" else D
    kind = {"fp4": torch.uint8, "i8": torch.int8, "e4m3": torch.uint8}.get(fmt) or TYPES[fmt]
    codes = torch.zeros((units, 2, HKV, rows, width), dtype=kind, device="cuda")
    scales = None
    if fmt == "fp4":
        scales = torch.zeros((units, 2, HKV, rows, D // GROUP), dtype=torch.uint8, device="cuda")
    elif fmt == "i8":
        scales = torch.zeros((units, 2, HKV, rows), dtype=torch.bfloat16, device="cuda")
    return codes, scales


def _cache(case, fmt, seed, spare=0):
    """A filled cache: keys whose channels differ in size, as they do after the key's norm weights, and values.
    Contiguous [B,2,8,C,...], or a pool of shuffled pages with its block table and `spare` more pages a row."""
    B, C, page = case["batch"], case["capacity"], case["page"]
    units, rows = (B * (C // page + spare), page) if page else (B, C)
    codes, scales = _empty_cache(fmt, units, rows)
    gain = torch.ones((2, HKV, 1, D), device="cuda")
    gain[0] = torch.exp(0.4 * _randn((HKV, 1, D), seed, 3))
    step = max(1, (1 << 27) // (2 * HKV * rows * D))
    for k in range(0, units, step):
        n = min(step, units - k)
        x = _randn((n, 2, HKV, rows, D), seed, 100 + k) * gain
        for plane in (0, 1):
            c, s = _quantise(x[:, plane], fmt, SCALES.get(fmt, (1, 1))[plane])
            codes[k:k + n, plane] = c
            if scales is not None:
                scales[k:k + n, plane] = s
    table = more = None
    if page:
        order = torch.randperm(units, generator=_gen(seed, 4), device="cuda").to(torch.int32)
        table = order[:B * (C // page)].view(B, C // page).contiguous()
        more = order[B * (C // page):].view(B, spare).contiguous()
    return codes, scales, table, more


def _gq():
    import gqa_decode_attention_sm_gb300 as gq
    return gq


def prepare(case, seed):
    kind, B = case["kind"], case["batch"]
    s = {"kind": kind, "case": case, "dtype": TYPES[case["dtype"]]}
    if kind == "drafts":
        _prepare_drafts(s, case, seed)
        return s
    fmt, C, page = case["fmt"], case["capacity"], case["page"]
    s["scale"] = SCALES.get(fmt, (1.0, 1.0))
    s["lens_host"], n = _sizes(case, seed)
    s["lens"] = s["lens_host"].to(torch.int32).cuda()
    spare = -(-case["keep"] // page) if kind == "evict" and page else 0
    s["kv"], s["scales"], s["table"], s["out_table"] = _cache(case, fmt, seed, spare)
    if kind == "prefill":
        s["starts_host"] = torch.cat((torch.zeros(1, dtype=torch.int64), n.cumsum(0)))
        s["starts"] = s["starts_host"].to(torch.int32).cuda()
        # room for the most tokens; what lies behind the last chunk is padding
        s["q"] = _randn((B * case["n_hi"], HQ, D), seed, 1).to(s["dtype"])
        s["out"] = torch.zeros_like(s["q"])
        if own:
            s["workspace"] = torch.zeros(_gq().prefill_workspace_size(), dtype=torch.uint8, device="cuda")
    if kind == "weights":
        s["q"] = _randn((B, case["q_len"], HQ, D), seed, 1).to(s["dtype"])
        s["acc"] = torch.zeros((B, HKV, C), device="cuda")
        if own:
            s["workspace"] = torch.zeros(_gq().weights_workspace_size(B, C, case["q_len"]), dtype=torch.uint8, device="cuda")
    if kind == "evict":
        # sums of softmax weights: a few large, many small, and none at all on slots that were just written
        w = torch.exp(2 * _randn((B, HKV, C), seed, 7))
        s["acc"] = torch.where(torch.rand((B, HKV, C), generator=_gen(seed, 8), device="cuda") < 0.1, 0.0, w / C)
        if page:
            s["out_kv"], s["out_scales"] = s["kv"], s["scales"]
        else:
            s["out_kv"], s["out_scales"] = _empty_cache(fmt, B, case["keep"] + case["keep"] % 2)
        s["out_acc"] = torch.zeros((B, HKV, case["keep"]), device="cuda")
        s["out_lens"] = torch.zeros_like(s["lens"])
        s["kept"] = torch.zeros((B, HKV, case["keep"]), dtype=torch.int32, device="cuda")
        rows = -(-case["keep"] // page) * page if page else s["out_kv"].shape[3]
        s["back"] = torch.zeros((B, 2, HKV, rows, D), dtype=s["dtype"], device="cuda")
        if own:
            s["workspace"] = torch.zeros(_gq().evict_workspace_size(B, case["keep"]), dtype=torch.uint8, device="cuda")
    return s


def _prepare_drafts(s, case, seed):
    B, T, V = case["batch"], case["window"], case["vocab"]
    # the target's probabilities, and the draft model's, which are near them; drafts drawn from the latter
    x = 2.5 * _randn((B, T, V), seed, 1)
    s["probs"] = torch.softmax(x, -1).to(s["dtype"])
    y = torch.softmax(x[:, :T - 1] + 0.7 * _randn((B, T - 1, V), seed, 2), -1)
    if case["greedy"]:
        s["draft_probs"] = None
        s["drafts"] = y.argmax(-1).to(torch.int32)
    else:
        s["draft_probs"] = y.to(s["dtype"])
        e = -torch.log1p(-torch.rand((B, T - 1, V), generator=_gen(seed, 3), device="cuda"))
        s["drafts"] = (y / e.clamp(min=1e-30)).argmax(-1).to(torch.int32) if T > 1 else \
            torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    if T > 2 and B > 2:
        s["drafts"][B // 2, 1:] = -1  # a request with a single draft
    s["u"] = torch.rand((B, T), generator=_gen(seed, 4), device="cuda")
    s["lens"] = torch.randint(T, 32768, (B,), generator=_gen(seed, 5), device="cuda", dtype=torch.int32)
    s["tokens"] = torch.zeros((B, T), dtype=torch.int32, device="cuda")
    s["accepted"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
    s["out_lens"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
    if own:
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------- the plain forms


def run(s):
    if own:
        return _run_own(s)
    return {"prefill": _plain_prefill, "drafts": _plain_drafts, "weights": _plain_weights,
            "evict": _plain_evict}[s["kind"]](s)


def _rows_of(pool, table):
    """A cache in pages as a contiguous one."""
    if pool is None or table is None:
        return pool
    x = pool[table.long()]  # [B, pages, 2, 8, page, ...]
    return x.movedim(1, 3).flatten(3, 4)


def _plane(s, plane, b, n):
    """Slots [0, n) of row b of the keys (0) or values (1), [8, n, 128] in 32 bits."""
    case = s["case"]
    if s["table"] is None:
        kv, sc = s["kv"][b:b + 1, plane], None if s["scales"] is None else s["scales"][b:b + 1, plane]
    else:
        pages = s["table"][b, :-(-n // case["page"])].long()
        kv, sc = s["kv"][pages, plane], None if s["scales"] is None else s["scales"][pages, plane]
    x = _values(kv, sc, case["fmt"], s["scale"][plane])
    return x.movedim(0, 1).flatten(1, 2)[:, :n]


def _plain_prefill(s):
    out = s["out"]
    for b in range(s["case"]["batch"]):
        at, end = int(s["starts_host"][b]), int(s["starts_host"][b + 1])
        n, L = end - at, int(s["lens_host"][b])
        if not n:
            continue
        k, v = _plane(s, 0, b, L), _plane(s, 1, b, L)
        q = s["q"][at:end].to(torch.float32).view(n, HKV, 4, D).permute(1, 2, 0, 3)  # [8, 4, n, 128]
        hidden = torch.arange(L, device="cuda").view(1, L) > torch.arange(L - n, L, device="cuda").view(n, 1)
        for h in range(HKV):
            x = torch.matmul(q[h], k[h].t()) / math.sqrt(D)
            x = x.masked_fill(hidden, -math.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(x, v[h]) / x.sum(-1, keepdim=True)
            out[at:end, 4 * h:4 * h + 4] = o.transpose(0, 1).to(s["dtype"])
    return {"out": out}


def _plain_drafts(s):
    case = s["case"]
    B, T, V = case["batch"], case["window"], case["vocab"]
    p, d, u = s["probs"], s["drafts"].long(), s["u"]
    given = torch.cumprod(((d >= 0) & (d < V)).long(), 1)  # a row's drafts end at its first -1
    at = d.clamp(0, V - 1).unsqueeze(-1)
    pd = torch.gather(p[:, :T - 1], 2, at).squeeze(-1).double()
    qd = torch.ones_like(pd) if case["greedy"] else torch.gather(s["draft_probs"], 2, at).squeeze(-1).double()
    taken = (u[:, :T - 1].double() * qd < pd) & (given == 1)
    n = torch.cumprod(taken.long(), 1).sum(1)
    refused = n < given.sum(1)  # a draft stands where the row's acceptance ended
    row = torch.arange(B, device="cuda")
    left = p[row, n].to(torch.float32)
    if T > 1:
        j = n.clamp(max=T - 2)
        if case["greedy"]:
            q = torch.zeros_like(left).scatter_(1, at[row, j], 1.0)
        else:
            q = s["draft_probs"][row, j].to(torch.float32)
        minus = (left - q) if not case["greedy"] else torch.where(q > 0, 0.0, left)
        left = torch.where(refused.view(B, 1), minus, left)
    # weights in whole units of 2^-38, so that their sums do not depend on the order
    w = (left.clamp(0, 1).double() * 2.0 ** 38).round().long()
    total = w.sum(1)
    target = (total * (u[:, T - 1].double() * 2 ** 24).floor().long()) >> 24
    pick = (torch.cumsum(w, 1) <= target.view(B, 1)).sum(1)
    tokens = torch.where(torch.arange(T - 1, device="cuda") < n.view(B, 1), d, -1)
    tokens = torch.cat((tokens, torch.full((B, 1), -1, device="cuda")), 1)
    tokens[row, n] = pick
    s["tokens"].copy_(tokens)
    s["accepted"].copy_(n)
    s["out_lens"].copy_((s["lens"] - (T - 1) + n).clamp(min=0))
    return {"tokens": s["tokens"], "accepted": s["accepted"], "lengths": s["out_lens"]}


def _plain_weights(s):
    case = s["case"]
    T, C, B = case["q_len"], case["capacity"], case["batch"]
    acc = s["acc"]
    for b in range(B):
        L = int(s["lens_host"][b])
        if not L:
            continue
        k = _plane(s, 0, b, L)
        q = s["q"][b].to(torch.float32).view(T, HKV, 4, D).permute(1, 2, 0, 3).reshape(HKV, 4 * T, D)
        x = (torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)).view(HKV, 4, T, L)
        end = L - T + torch.arange(T, device="cuda").view(T, 1)
        hidden = torch.arange(L, device="cuda").view(1, L) > end
        x = x.masked_fill(hidden, -math.inf)
        top = x.amax(-1, keepdim=True)
        x = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        total = x.sum(-1, keepdim=True)
        acc[b, :, :L] = torch.where(total > 0, x / total, 0.0).sum((1, 2))
    return {"weights": acc}


def _plain_evict(s):
    case = s["case"]
    C, B, keep, page = case["capacity"], case["batch"], case["keep"], case["page"]
    lens = s["lens"].long().view(B, 1, 1)
    t = torch.arange(C, device="cuda").view(1, 1, C)
    n = lens.clamp(max=keep)
    sure = (t < case["first"]) | (t >= lens - case["recent"])
    rank = torch.where(t < lens, torch.where(sure, math.inf, s["acc"]), -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices  # equal sums: the lowest slot first
    chosen = torch.zeros((B, HKV, C), dtype=torch.bool, device="cuda")
    chosen.scatter_(2, order[..., :keep], True)
    chosen &= t < lens
    kept = torch.sort(torch.where(chosen, t, C + 1), dim=-1).values[..., :keep]
    if kept.shape[-1] < keep:
        kept = torch.cat((kept, kept.new_full((B, HKV, keep - kept.shape[-1]), C + 1)), -1)
    live = torch.arange(keep, device="cuda").view(1, 1, keep) < n
    at = torch.where(live, kept, 0)
    s["kept"].copy_(torch.where(live, kept, -1))
    s["out_lens"].copy_(n.view(B))
    s["out_acc"].copy_(torch.where(live, torch.gather(s["acc"], 2, at), 0.0))
    rows = torch.arange(B, device="cuda").view(B, 1, 1).expand(B, HKV, keep)
    heads = torch.arange(HKV, device="cuda").view(1, HKV, 1).expand(B, HKV, keep)
    b, h, src = rows[live.expand_as(rows)], heads[live.expand_as(rows)], kept[live.expand_as(rows)]
    dst = torch.arange(keep, device="cuda").view(1, 1, keep).expand(B, HKV, keep)[live.expand_as(rows)]
    for out, kv in ((s["out_kv"], s["kv"]), (s["out_scales"], s["scales"])):
        if kv is None:
            continue
        for plane in (0, 1):
            if page:
                out[s["out_table"][b, dst // page].long(), plane, h, dst % page] = \
                    kv[s["table"][b, src // page].long(), plane, h, src % page]
            else:
                out[b, plane, h, dst] = kv[b, plane, h, src]
    return _evicted(s, None)


def _evicted(s, back):
    """What an eviction gives; a cache in pages or of few bits as the 16-bit values of its rows."""
    case = s["case"]
    if back is None and (case["page"] or s["scales"] is not None or case["fmt"] == "e4m3"):
        kv, sc = _rows_of(s["out_kv"], s["out_table"]), _rows_of(s["out_scales"], s["out_table"])
        x = torch.stack([_values(kv[:, p], None if sc is None else sc[:, p], case["fmt"], s["scale"][p])
                         for p in (0, 1)], 1)
        rows = s["back"].shape[3]
        live = torch.arange(rows, device="cuda") < s["out_lens"].view(-1, 1)
        back = torch.where(live.view(-1, 1, 1, rows, 1), x.to(s["dtype"]), s["back"])
    return {"kv": s["out_kv"] if back is None else back, "weights": s["out_acc"], "lengths": s["out_lens"],
            "kept": s["kept"]}


# --------------------------------------------------- the framework's kernels


def _run_own(s):
    gq = _gq()
    case, kind = s["case"], s["kind"]
    if kind == "drafts":
        gq.verify_drafts(s["probs"], s["drafts"], s["u"], draft_probs=s["draft_probs"], sequence_lengths=s["lens"],
                         out_lengths=s["out_lens"], tokens=s["tokens"], accepted=s["accepted"],
                         workspace=s["workspace"])
        return {"tokens": s["tokens"], "accepted": s["accepted"], "lengths": s["out_lens"]}
    ks, vs = s["scale"]
    paged = s["table"] is not None
    if kind == "prefill":
        how = dict(k_scale=ks, v_scale=vs, kv_scales=s["scales"], out=s["out"], workspace=s["workspace"])
        if paged:
            return {"out": gq.gqa_prefill_paged(s["q"], s["kv"], s["table"], s["starts"], s["lens"], **how)}
        return {"out": gq.gqa_prefill(s["q"], s["kv"], s["starts"], s["lens"], **how)}
    if kind == "weights":
        how = dict(k_scale=ks, kv_scales=s["scales"], add=False, workspace=s["workspace"])
        if paged:
            gq.accumulate_weights_paged(s["q"], s["kv"], s["table"], s["lens"], s["acc"], **how)
        else:
            gq.accumulate_weights(s["q"], s["kv"], s["lens"], s["acc"], **how)
        return {"weights": s["acc"]}
    how = dict(recent=case["recent"], first=case["first"], out_lengths=s["out_lens"], out_weights=s["out_acc"],
               kept=s["kept"], kv_scales=s["scales"], workspace=s["workspace"])
    if paged:
        gq.evict_kv_paged(s["kv"], s["table"], s["lens"], s["acc"], case["keep"], out_table=s["out_table"], **how)
        back = gq.read_kv_paged(s["kv"], s["out_table"], s["out_lens"], out=s["back"], k_scale=ks, v_scale=vs,
                                kv_scales=s["scales"])
        return _evicted(s, back)
    gq.evict_kv(s["kv"], s["lens"], s["acc"], case["keep"], out=s["out_kv"], out_scales=s["out_scales"], **how)
    if s["scales"] is None and case["fmt"] != "e4m3":
        return _evicted(s, None)
    return _evicted(s, gq.read_kv(s["out_kv"], s["out_lens"], out=s["back"], k_scale=ks, v_scale=vs,
                                  kv_scales=s["out_scales"]))


# ------------------------------------------------------- in 64 bits, by rows


def _row64(s, b, plane, h, L):
    """Slots [0, L) of KV head h of batch row b of one plane in 64 bits, from the format's definition."""
    case, fmt = s["case"], s["case"]["fmt"]
    if s["table"] is not None:
        pages = s["table"][b].long()[: -(-L // case["page"])]
        codes = s["kv"][pages, plane, h].flatten(0, 1)[:L]
        scales = None if s["scales"] is None else s["scales"][pages, plane, h].flatten(0, 1)[:L]
    else:
        codes = s["kv"][b, plane, h, :L]
        scales = None if s["scales"] is None else s["scales"][b, plane, h, :L]
    if fmt == "fp4":
        level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        level = torch.cat((level, -level))
        x = torch.empty((L, D), dtype=torch.float64, device="cuda")
        x[:, 0::2] = level[codes.long() % 16]
        x[:, 1::2] = level[codes.long() // 16]
        step = scales.contiguous().view(torch.float8_e4m3fn).double() * s["scale"][plane]
        return x * step.repeat_interleave(GROUP, 1)
    if fmt == "i8":
        return codes.double() * scales.double()[:, None]
    if fmt == "e4m3":
        return codes.contiguous().view(torch.float8_e4m3fn).double() * s["scale"][plane]
    return codes.double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, B = case["kind"], case["batch"]
    if kind == "drafts":
        return _exact_drafts(s, case)
    if kind == "prefill":
        if work(case)["flops"] > 6e12:
            return None
        out = s["out"].double()
        for b in range(B):
            at, end = int(s["starts_host"][b]), int(s["starts_host"][b + 1])
            L = int(s["lens_host"][b])
            for h in range(HKV if end > at else 0):
                K, V = _row64(s, b, 0, h, L), _row64(s, b, 1, h, L)
                for first in range(at, end, 512):  # the queries in blocks, each over the slots that its last one sees
                    last = min(end, first + 512)
                    top = L - (end - last)
                    see = torch.ones((last - first, top), dtype=torch.bool, device="cuda").tril(top - (last - first))
                    for g in range(4 * h, 4 * h + 4):
                        x = s["q"][first:last, g].double() @ K[:top].t() / math.sqrt(128.0)
                        out[first:last, g] = torch.softmax(torch.where(see, x, -math.inf), -1) @ V[:top]
        return {"out": out}
    if kind == "weights":
        T = case["q_len"]
        acc = torch.zeros((B, HKV, case["capacity"]), dtype=torch.float64, device="cuda")
        for b in range(B):
            L = int(s["lens_host"][b])
            for h in range(HKV if L else 0):
                K = _row64(s, b, 0, h, L)
                for j in range(T):
                    n = L - T + 1 + j
                    if n > 0:
                        x = s["q"][b, j, 4 * h:4 * h + 4].double() @ K[:n].t() / math.sqrt(128.0)
                        acc[b, h, :n] += torch.softmax(x, -1).sum(0)
        return {"weights": acc}
    keep = case["keep"]
    read_back = bool(case["page"]) or s["scales"] is not None or case["fmt"] == "e4m3"
    kv = (s["back"] if read_back else s["out_kv"]).double()
    weights = torch.zeros((B, HKV, keep), dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(s["lens_host"][b])
        sums = s["acc"][b, :, :L].tolist()
        for h in range(HKV if L else 0):
            lo, hi = min(case["first"], L), max(min(case["first"], L), L - case["recent"])
            slots = list(range(L))
            if L > keep:
                rest = sorted(range(lo, hi), key=lambda t: (-sums[h][t], t))[:keep - lo - (L - hi)]
                slots = sorted(list(range(lo)) + rest + list(range(hi, L)))
            at = torch.tensor(slots, device="cuda")
            weights[b, h, :len(slots)] = s["acc"][b, h, at].double()
            for plane in (0, 1):
                kv[b, plane, h, :len(slots)] = _row64(s, b, plane, h, L)[at]
    return {"kv": kv, "weights": weights, "lengths": None, "kept": None}


def _exact_drafts(s, case):
    """A row at a time, with whole numbers of the interpreter."""
    T, V = case["window"], case["vocab"]
    tokens, accepted = [], []
    for b in range(case["batch"]):
        taken, q = [], None
        u = s["u"][b].tolist()
        for j in range(T - 1):
            d = int(s["drafts"][b, j])
            if not 0 <= d < V:
                break
            q = torch.zeros(V, device="cuda") if case["greedy"] else s["draft_probs"][b, j].float()
            if case["greedy"]:
                q[d] = 1.0
            if u[j] * float(q[d]) < float(s["probs"][b, j, d]):
                taken.append(d)
                q = None
            else:
                break
        p = s["probs"][b, len(taken)].float()
        w = p if q is None else (p - q).clamp(min=0)
        whole = (w.double() * 2 ** 38).round().long().cpu()
        upto = whole.cumsum(0)
        target = (int(upto[-1]) * int(u[-1] * 2 ** 24)) // 2 ** 24
        pick = int(torch.searchsorted(upto, torch.tensor([target]), right=True)[0])
        tokens.append(taken + [pick] + [-1] * (T - 1 - len(taken)))
        accepted.append(len(taken))
    i32 = dict(dtype=torch.int32, device="cuda")
    n = torch.tensor(accepted, **i32)
    return {"tokens": torch.tensor(tokens, **i32), "accepted": n, "lengths": (s["lens"] - (T - 1) + n).clamp(min=0)}

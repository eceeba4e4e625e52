"""What the 4-bit cache operators are measured on.

Four kinds of pass, over 32 query heads, 8 KV heads and head_dim 128:

  decode  attention of 1 to 4 query tokens a request over a cache held in 4
          bits (e2m1 codes, an e4m3 scale for every 16 dims of a row and an
          fp32 scale for all keys and one for all values), contiguous or paged
  write   norm, rotary embedding (one position axis, or time, height and
          width) and the cache write of many tokens at once, 16-bit cache
  store   the same write into an fp4, int8 or e4m3 cache, then the rows read
          back to 16 bits, as a prompt taken in chunks does
  read    the rows of a cache of any format read back to a dense 16-bit cache

A 4-bit row is 64 bytes: byte j holds dims 2j (low nibble) and 2j + 1 (high
nibble) as e2m1 codes; kv_scales holds 8 e4m3 scales a row.
"""
import math

import torch

own = False

HQ, HKV, D, GROUP = 32, 8, 128, 16
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# the scales of all keys and of all values that a program has from its calibration
SCALES = {"fp4": (10 / 1024, 9 / 1024), "e4m3": (1 / 32, 1 / 32)}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # one request's decode step at a short context: latency
        {"name": "decode 1x1024", "kind": "decode", "dtype": "f16", "batch": 1, "capacity": 1024, "len_lo": 1024,
         "len_hi": 1024, "q_len": 1, "page": 0},
        # a serving batch of ragged lengths, one row of it empty (a finished request's place)
        {"name": "decode 32x8192 ragged", "kind": "decode", "dtype": "f16", "batch": 32, "capacity": 8192, "len_lo": 0,
         "len_hi": 8192, "q_len": 1, "page": 0},
        # long contexts: the cache's bytes are all that counts
        {"name": "decode 8x131072", "kind": "decode", "dtype": "bf16", "batch": 8, "capacity": 131072,
         "len_lo": 131072, "len_hi": 131072, "q_len": 1, "page": 0},
        # a full serving batch over a paged pool
        {"name": "decode 64x32768 paged", "kind": "decode", "dtype": "bf16", "batch": 64, "capacity": 32768,
         "len_lo": 16384, "len_hi": 32768, "q_len": 1, "page": 256},
        # a verify window of three tokens (speculative decoding), odd lengths
        {"name": "verify 3 8x32768", "kind": "decode", "dtype": "bf16", "batch": 8, "capacity": 32768, "len_lo": 16385,
         "len_hi": 32767, "q_len": 3, "page": 0},
        # the tokens of 64 verify windows of 4 written into a paged cache: latency
        {"name": "write 64x4 paged", "kind": "write", "dtype": "bf16", "fmt": "bf16", "tokens": 256, "batch": 64,
         "capacity": 256, "page": 16, "axes": 1, "interleaved": False, "fused": False, "norm": True},
        # a prompt with image tokens, taken from a fused projection
        {"name": "write 8192 image", "kind": "write", "dtype": "f16", "fmt": "f16", "tokens": 8192, "batch": 4,
         "capacity": 2112, "page": 0, "axes": 3, "interleaved": True, "fused": True, "norm": True},
        # a chunk of a prompt into a paged 4-bit cache, then the whole prefix back for the chunk's attention
        {"name": "store fp4 4096", "kind": "store", "dtype": "bf16", "fmt": "fp4", "tokens": 4096, "batch": 4,
         "capacity": 4096, "page": 64, "axes": 3, "interleaved": True, "fused": True, "norm": True},
        # the same of an int8 cache with odd sizes, positions in blocks of the axes, no norm
        {"name": "store int8 1531", "kind": "store", "dtype": "f16", "fmt": "i8", "tokens": 1531, "batch": 3,
         "capacity": 1000, "page": 0, "axes": 3, "interleaved": False, "fused": False, "norm": False},
        # the prefixes of long contexts read back from a 4-bit pool
        {"name": "read fp4 8x32768 paged", "kind": "read", "dtype": "bf16", "fmt": "fp4", "batch": 8,
         "capacity": 32768, "len_lo": 16384, "len_hi": 32768, "page": 256, "starts": False},
        # one short request's e4m3 cache: latency
        {"name": "read e4m3 1x1024", "kind": "read", "dtype": "f16", "fmt": "e4m3", "batch": 1, "capacity": 1024,
         "len_lo": 1023, "len_hi": 1023, "page": 0, "starts": False},
        # the last slots of ragged rows of a 16-bit pool made contiguous
        {"name": "read bf16 32x8192 paged", "kind": "read", "dtype": "bf16", "fmt": "bf16", "batch": 32,
         "capacity": 8192, "len_lo": 1, "len_hi": 8192, "page": 64, "starts": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "write", "store", "read"])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([0, 16, 64, 256])
    if kind == "decode":
        batch = _log(rng, 1, 64)
        capacity = _log(rng, 64, max(64, min(131072, (1 << 20) // batch)))
        q_len = rng.choice([1, 1, 2, 3, 4])
        capacity = -(-capacity // (page or 2)) * (page or 2)
        hi = rng.randint(q_len, capacity)
        return {"kind": kind, "dtype": dtype, "batch": batch, "capacity": capacity,
                "len_lo": rng.choice([hi, max(q_len, hi // 2), min(q_len, hi)]), "len_hi": hi, "q_len": q_len,
                "page": page}
    if kind in ("write", "store"):
        tokens = _log(rng, 1, 8192)
        batch = min(tokens, _log(rng, 1, 64))
        per = -(-tokens // batch)
        capacity = -(-(per + rng.randint(0, max(1, per // 2))) // (page or 8)) * (page or 8)
        axes = rng.choice([1, 3])
        return {"kind": kind, "dtype": dtype, "fmt": dtype if kind == "write" else rng.choice(["fp4", "fp4", "i8", "e4m3"]),
                "tokens": tokens, "batch": batch, "capacity": capacity, "page": page, "axes": axes,
                "interleaved": axes == 3 and rng.random() < 0.5, "fused": rng.random() < 0.5,
                "norm": rng.random() < 0.8}
    batch = _log(rng, 1, 32)
    capacity = _log(rng, 16, max(16, (1 << 17) // batch))
    capacity = -(-capacity // (page or 8)) * (page or 8)
    hi = rng.randint(1, capacity)
    fmt = rng.choice(["fp4", "fp4", "i8", "e4m3", dtype])
    return {"kind": kind, "dtype": dtype, "fmt": fmt, "batch": batch, "capacity": capacity,
            "len_lo": rng.choice([hi, 0]), "len_hi": hi, "page": page, "starts": rng.random() < 0.5}


def _lengths(case, seed):
    """A decode's or a read's lengths, on the host."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(case["len_lo"], case["len_hi"] + 1, (case["batch"],), generator=g)
    if case["len_lo"] == 0 and case["batch"] > 1:
        n[case["batch"] // 2] = 0
    return n


def _share(case):
    """Tokens of each batch row in a write (all but the last rows hold one more or the same)."""
    n, b = case["tokens"], case["batch"]
    return [n // b + (i < n % b) for i in range(b)]


def _row_bytes(fmt):
    return {"f16": 256, "bf16": 256, "e4m3": 128, "i8": 130, "fp4": 72}[fmt]


def work(case):
    kind, B = case["kind"], case["batch"]
    if kind in ("decode", "read"):  # the lengths' mean
        tokens = B * (case["len_lo"] + case["len_hi"]) / 2
    if kind == "decode":
        T = case["q_len"]
        return {"bytes": tokens * 16 * _row_bytes("fp4") + 2 * B * T * HQ * D * 2 + 4 * B,
                "flops": 4 * tokens * T * HQ * D}
    if kind == "read":
        if case["starts"]:
            tokens /= 2
        return {"bytes": tokens * 16 * (_row_bytes(case["fmt"]) + 256), "flops": 2 * tokens * 16 * D}
    n = case["tokens"]
    moved = n * ((HQ + 2 * HKV) * D * 2 + HQ * D * 2 + 16 * _row_bytes(case["fmt"]))
    flops = n * (HQ + HKV) * D * 8
    if kind == "store":
        kept = n + B * _prefix(case)
        moved += kept * 16 * (_row_bytes(case["fmt"]) + 256)
        flops += 2 * kept * 16 * D
    return {"bytes": moved, "flops": flops}


def _prefix(case):
    """Slots of each row that a store finds filled (the chunks before)."""
    return case["capacity"] - max(_share(case))


# ------------------------------------------------------------------ inputs


def _gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(seed * 1009 + k)


def _randn(shape, seed, k, dtype=torch.float32):
    return torch.randn(shape, generator=_gen(seed, k), device="cuda", dtype=dtype)


def _quantise(x, fmt, scale):
    """(codes, scales) of rows x [..., 128] in 32 or 64 bits; `scale` is the one of all of them."""
    if fmt == "fp4":
        g = (x / scale).unflatten(-1, (D // GROUP, GROUP))
        s = (g.abs().amax(-1) / 6).clamp(max=448).to(torch.float32).to(torch.float8_e4m3fn)
        wide = s.to(x.dtype).unsqueeze(-1)
        t = torch.where(wide > 0, g / wide, torch.zeros_like(g))
        m = t.abs().clamp(max=6)
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).to(x.dtype)
        m = (m / step).round() * step  # 0, 0.5, 1, 1.5, 2, 3, 4, 6: to the nearest, ties to the even code
        c = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
        c = (c | ((t < 0).to(torch.uint8) << 3)).flatten(-2)
        return c[..., 0::2] | (c[..., 1::2] << 4), s.view(torch.uint8)
    if fmt == "i8":
        s = (x.abs().amax(-1) / 127).to(torch.bfloat16)
        s = torch.where(s == 0, torch.ones_like(s), s)
        return (x / s.to(x.dtype).unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8), s
    if fmt == "e4m3":
        return (x / scale).clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8), None
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


def _cache(case, fmt, seed):
    """A filled cache: keys whose channels differ in size, as they do after the key's norm weights, and values.
    Contiguous [B,2,8,C,...], or a pool of shuffled pages with its block table."""
    B, C, page = case["batch"], case["capacity"], case["page"]
    units, rows = (B * C // page, page) if page else (B, C)
    width = 64 if fmt == "fp4" else D
    kind = {"fp4": torch.uint8, "i8": torch.int8, "e4m3": torch.uint8}.get(fmt) or TYPES[fmt]
    codes = torch.empty((units, 2, HKV, rows, width), dtype=kind, device="cuda")
    scales = None
    if fmt == "fp4":
        scales = torch.empty((units, 2, HKV, rows, D // GROUP), dtype=torch.uint8, device="cuda")
    elif fmt == "i8":
        scales = torch.empty((units, 2, HKV, rows), dtype=torch.bfloat16, device="cuda")
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
    table = None
    if page:
        order = torch.randperm(units, generator=_gen(seed, 4), device="cuda")
        table = order.to(torch.int32).view(B, C // page).contiguous()
    return codes, scales, table


def prepare(case, seed):
    kind, B = case["kind"], case["batch"]
    dtype = TYPES[case["dtype"]]
    fmt = "fp4" if kind == "decode" else case["fmt"]
    s = {"kind": kind, "case": case, "dtype": dtype, "scale": SCALES.get(fmt, (1.0, 1.0))}
    if kind in ("decode", "read"):
        s["lens_host"] = _lengths(case, seed)
        s["lens"] = s["lens_host"].to(torch.int32).cuda()
        s["kv"], s["scales"], s["table"] = _cache(case, fmt, seed)
    if kind == "decode":
        shape = (B, HQ, D) if case["q_len"] == 1 else (B, case["q_len"], HQ, D)
        s["q"] = _randn(shape, seed, 1).to(dtype)
        s["out"] = torch.empty_like(s["q"])
    if kind == "read":
        s["starts"] = (s["lens"] // 2) if case["starts"] else None
        s["out"] = torch.zeros((B, 2, HKV, case["capacity"], D), dtype=dtype, device="cuda")
    if kind in ("write", "store"):
        _prepare_tokens(s, case, seed)
    if own:
        # what a serving program keeps: the split count and its workspace, planned once for the cache's size
        import gqa_decode_attention_sm_gb300 as gq
        if kind == "decode" and case["q_len"] == 1 and not case["page"]:
            s["plan"] = gq.prepare({"Q": s["q"], "KV": s["kv"], "KV_SCALES": s["scales"], "O": s["out"],
                                    "sequence_lengths": s["lens"]}, k_scale=s["scale"][0], v_scale=s["scale"][1])
        elif kind == "decode":
            s["splits"] = gq.plan(B, case["capacity"], 4)
            s["workspace"] = torch.zeros(gq.workspace_size(B * case["q_len"], case["capacity"], s["splits"]),
                                         dtype=torch.uint8, device="cuda")
    return s


def _prepare_tokens(s, case, seed):
    n, B, dtype = case["tokens"], case["batch"], s["dtype"]
    share = _share(case)
    at = 0 if case["kind"] == "write" else _prefix(case)
    rows = torch.repeat_interleave(torch.arange(B), torch.tensor(share))
    slots = torch.cat([torch.arange(k) + at for k in share])
    # positions: text counts up on every axis; the middle half of a row is an image, a grid on two axes
    t = slots.clone() + 1000 * rows
    pos = torch.stack((t, t, t))
    if case["axes"] == 3:
        width = max(1, int(math.sqrt(max(share) / 2)))
        k = torch.cat([torch.arange(m) for m in share])
        m = torch.repeat_interleave(torch.tensor(share), torch.tensor(share))
        image = (k >= m // 4) & (k < m // 4 + m // 2)
        j = k - m // 4
        base = t - j
        pos = torch.where(image, torch.stack((base, base + j // width, base + j % width)), pos)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(seed))  # tokens come in any order
    s["rows"], s["slots"] = rows[perm].to(torch.int32).cuda(), slots[perm].to(torch.int32).cuda()
    pos = pos[:, perm].to(torch.int32).cuda()
    s["pos"] = pos[0].contiguous() if case["axes"] == 1 else pos.contiguous()
    s["section"] = None if case["axes"] == 1 else ((24, 20, 20) if case["interleaved"] else (16, 24, 24))
    wide = torch.exp(0.7 * _randn((1, HQ + 2 * HKV, 1), seed, 5))
    x = (_randn((n, HQ + 2 * HKV, D), seed, 6) * wide).to(dtype)
    parts = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    s["q"], s["k"], s["v"] = parts if case["fused"] else [p.contiguous() for p in parts]
    s["qw"] = s["kw"] = None
    if case["norm"]:
        s["qw"] = torch.exp(0.3 * _randn((D,), seed, 7)).to(dtype)
        s["kw"] = torch.exp(0.4 * _randn((D,), seed, 8)).to(dtype)
    s["q_out"] = torch.empty((n, HQ, D), dtype=dtype, device="cuda")
    s["kv"], s["scales"], s["table"] = _cache(case, case["fmt"], seed)
    if case["kind"] == "store":
        s["lens_host"] = torch.tensor(share) + at
        s["lens"] = s["lens_host"].to(torch.int32).cuda()
        s["starts"] = None
        s["out"] = torch.zeros((B, 2, HKV, case["capacity"], D), dtype=dtype, device="cuda")


# ---------------------------------------------------------- the plain forms


def run(s):
    if own:
        return _run_own(s)
    if s["kind"] == "decode":
        return {"out": _plain_decode(s)}
    if s["kind"] == "read":
        return {"kv": _plain_read(s)}
    q_out = _plain_write(s)
    if s["kind"] == "write":
        return {"q_out": q_out, "kv": s["kv"]}
    return {"q_out": q_out, "kv": _plain_read(s)}


def _rows_of(pool, table):
    """A cache in pages as a contiguous one."""
    if pool is None or table is None:
        return pool
    x = pool[table.long()]  # [B, pages, 2, 8, page, ...]
    return x.movedim(1, 3).flatten(3, 4)


def _plain_decode(s):
    case = s["case"]
    T, C, B = case["q_len"], case["capacity"], case["batch"]
    q = s["q"].to(torch.float32).view(B, T, HKV, HQ // HKV, D).permute(0, 2, 1, 3, 4).reshape(B, HKV, T * 4, D)
    kv, sc = _rows_of(s["kv"], s["table"]), _rows_of(s["scales"], s["table"])
    k = _values(kv[:, 0], sc[:, 0], "fp4", s["scale"][0])
    scores = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)  # [B, 8, T*4, C]
    last = s["lens"].view(B, 1) - T + 1 + torch.arange(T, device="cuda").view(1, T)  # slots below it are seen
    seen = torch.arange(C, device="cuda") < last.repeat_interleave(4, 1).view(B, 1, T * 4, 1)
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _values(kv[:, 1], sc[:, 1], "fp4", s["scale"][1]))
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.view(B, HKV, T, 4, D).permute(0, 2, 1, 3, 4).reshape(s["q"].shape).to(s["dtype"])


def _plain_read(s):
    case = s["case"]
    C = case["capacity"]
    kv, sc = _rows_of(s["kv"], s["table"]), _rows_of(s["scales"], s["table"])
    x = torch.stack([_values(kv[:, p], None if sc is None else sc[:, p], case["fmt"], s["scale"][p])
                     for p in (0, 1)], 1)
    first = s["starts"] if s["starts"] is not None else torch.zeros_like(s["lens"])
    at = (torch.arange(C, device="cuda") + first.view(-1, 1)).clamp(max=C - 1).long()  # [B, C]
    if s["starts"] is not None:
        x = torch.gather(x, 3, at.view(-1, 1, 1, C, 1).expand(-1, 2, HKV, -1, D))
    kept = torch.arange(C, device="cuda") < (s["lens"] - first).view(-1, 1)
    return torch.where(kept.view(-1, 1, 1, C, 1), x.to(s["dtype"]), s["out"])


def _angles(s):
    """Cosine and sine [N, 1, 64] of the rotary angles; the angles in 64 bits."""
    i = torch.arange(D // 2, device="cuda")
    pos = s["pos"]
    if pos.dim() == 1:
        at = pos.view(-1, 1).expand(-1, D // 2)
    else:
        t, h, w = s["section"]
        if s["case"]["interleaved"]:
            axis = torch.where((i % 3 == 1) & (i < 3 * h), 1, torch.where((i % 3 == 2) & (i < 3 * w), 2, 0))
        else:
            axis = (i >= t).long() + (i >= t + h).long()
        at = pos[axis].t()
    a = at.double() * torch.pow(torch.tensor(1e6, dtype=torch.float64, device="cuda"), -i.double() / (D // 2))
    return torch.cos(a).unsqueeze(1), torch.sin(a).unsqueeze(1)


def _rotated(x, w, cos, sin):
    """Norm and rotation of heads x [N, H, 128], in x's precision."""
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.to(x.dtype)
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_write(s):
    case = s["case"]
    cos, sin = _angles(s)
    q = _rotated(s["q"].float(), s["qw"], cos.float(), sin.float())
    # keys in 64 bits: a code next to a border of its rounding would turn on the 32-bit error
    k = _rotated(s["k"].double(), s["kw"], cos, sin)
    rows, slots = s["rows"].long(), s["slots"].long()
    if s["table"] is not None:
        rows, slots = s["table"][rows, slots // case["page"]].long(), slots % case["page"]
    for plane, x in ((0, k), (1, s["v"].double())):
        c, sc = _quantise(x, case["fmt"], s["scale"][plane])
        s["kv"][rows, plane, :, slots] = c
        if sc is not None:
            s["scales"][rows, plane, :, slots] = sc
    return q.to(s["dtype"])


# --------------------------------------------------- the framework's kernels


def _run_own(s):
    import gqa_decode_attention_sm_gb300 as gq
    case = s["case"]
    scale = dict(k_scale=s["scale"][0], v_scale=s["scale"][1])
    if s["kind"] == "decode":
        if "plan" in s:
            return {"out": gq.launch(s["plan"])}
        if s["table"] is not None:
            return {"out": gq.gqa_decode_paged(s["q"], s["kv"], s["table"], s["lens"], out=s["out"],
                                               num_splits=s["splits"], workspace=s["workspace"],
                                               kv_scales=s["scales"], **scale)}
        return {"out": gq.gqa_decode_verify(s["q"], s["kv"], s["lens"], kv_scales=s["scales"], out=s["out"],
                                            num_splits=s["splits"], workspace=s["workspace"], **scale)}
    if s["kind"] in ("write", "store"):
        how = dict(q_out=s["q_out"], mrope_section=s["section"], mrope_interleaved=case["interleaved"],
                   kv_scales=s["scales"], **scale)
        if s["table"] is not None:
            gq.write_kv_paged(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["pos"], s["rows"], s["slots"], s["kv"],
                              s["table"], **how)
        else:
            gq.write_kv(s["q"], s["k"], s["v"], s["qw"], s["kw"], s["pos"], s["rows"], s["slots"], s["kv"], **how)
        if s["kind"] == "write":
            return {"q_out": s["q_out"], "kv": s["kv"]}
    if s["table"] is not None:
        kv = gq.read_kv_paged(s["kv"], s["table"], s["lens"], starts=s["starts"], out=s["out"], kv_scales=s["scales"],
                              **scale)
    else:
        kv = gq.read_kv(s["kv"], s["lens"], starts=s["starts"], out=s["out"], kv_scales=s["scales"], **scale)
    return {"kv": kv} if s["kind"] == "read" else {"q_out": s["q_out"], "kv": kv}


# ------------------------------------------------------- in 64 bits, by rows


def _row64(s, b, plane, fmt, L):
    """Slots [0, L) of batch row b of one plane, [8, L, 128] in 64 bits, from the format's definition."""
    case = s["case"]
    if s["table"] is not None:
        pages = s["table"][b].long()
        codes = torch.cat([s["kv"][p, plane] for p in pages[: -(-L // case["page"])]], 1)[:, :L]
        scales = None if s["scales"] is None else torch.cat([s["scales"][p, plane] for p in
                                                             pages[: -(-L // case["page"])]], 1)[:, :L]
    else:
        codes = s["kv"][b, plane, :, :L]
        scales = None if s["scales"] is None else s["scales"][b, plane, :, :L]
    if fmt == "fp4":
        level = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        level = torch.cat((level, -level))
        x = torch.empty((HKV, L, D), dtype=torch.float64, device="cuda")
        x[..., 0::2] = level[codes.long() % 16]
        x[..., 1::2] = level[codes.long() // 16]
        step = scales.contiguous().view(torch.float8_e4m3fn).double() * s["scale"][plane]
        for g in range(D // GROUP):
            x[..., GROUP * g:GROUP * (g + 1)] *= step[..., g:g + 1]
        return x
    if fmt == "i8":
        return codes.double() * scales.double()[..., None]
    if fmt == "e4m3":
        return codes.contiguous().view(torch.float8_e4m3fn).double() * s["scale"][plane]
    return codes.double()


def exact(case, seed):
    s = prepare(case, seed)
    kind, B = case["kind"], case["batch"]
    if kind == "decode":
        T = case["q_len"]
        out = torch.zeros((B, T, HQ, D), dtype=torch.float64, device="cuda")
        q = s["q"].double().view(B, T, HQ, D)
        for b in range(B):
            L = int(s["lens_host"][b])
            if not L:
                continue
            K, V = (_row64(s, b, plane, "fp4", L) for plane in (0, 1))
            for j in range(T):
                n = L - T + 1 + j
                if n < 1:
                    continue
                for h in range(HKV):
                    w = torch.softmax(q[b, j, 4 * h:4 * h + 4] @ K[h, :n].t() / math.sqrt(128.0), -1)
                    out[b, j, 4 * h:4 * h + 4] = w @ V[h, :n]
        return {"out": out.view(s["q"].shape)}
    if kind != "read":
        # a rotation as a product of complex numbers
        i = torch.arange(64, dtype=torch.float64, device="cuda")
        p = s["pos"].double()
        if p.dim() == 1:
            p = p.expand(3, -1)
        angle = p[0].unsqueeze(1) * 1e6 ** (-i / 64)
        if case["axes"] == 3:
            t, h, w = s["section"]
            for axis, count in ((1, h), (2, w)):
                if case["interleaved"]:
                    at = torch.arange(axis, 3 * count, 3, device="cuda")
                else:
                    at = torch.arange(count, device="cuda") + (t if axis == 1 else t + h)
                angle[:, at] = p[axis].unsqueeze(1) * 1e6 ** (-i[at] / 64)
        turn = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)

        def head(x, w):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / 128 + 1e-6) * w.double()
            z = torch.complex(x[..., :64].contiguous(), x[..., 64:].contiguous()) * turn
            return torch.cat((z.real, z.imag), -1)

        q_out, k = head(s["q"], s["qw"]), head(s["k"], s["kw"])
        fmt = case["fmt"]
        kv = torch.stack((k, s["v"].double()), 1)  # [N, 2, 8, 128]
        k_scale, v_scale = s["scale"]
        all_of = torch.tensor([k_scale, v_scale], dtype=torch.float64, device="cuda").view(1, 2, 1, 1)
        if fmt == "fp4":  # rounded to what the codes stand for: the levels' midpoints go to the even code
            g = (kv / all_of).reshape(-1, 2, HKV, 8, 16)
            step = torch.clamp(g.abs().max(-1, keepdim=True).values / 6, max=448).float()
            step = step.to(torch.float8_e4m3fn).double()
            t = g / step.clamp(min=1e-30)
            m = t.abs()
            near = torch.zeros_like(m)
            for low, high, even in ((0, 0.5, 0), (0.5, 1, 1), (1, 1.5, 1), (1.5, 2, 2), (2, 3, 2), (3, 4, 4), (4, 6, 4)):
                mid = (low + high) / 2
                near = torch.where((m > mid) | ((m == mid) & (even == high)), float(high), near)
            kv = (torch.sign(t) * near * step).reshape(kv.shape) * all_of
        elif fmt == "i8":
            step = (kv.abs().max(-1, keepdim=True).values / 127).to(torch.bfloat16).double()
            step[step == 0] = 1
            kv = torch.clamp(torch.round(kv / step), -127, 127) * step
        elif fmt == "e4m3":
            kv = (kv / all_of).clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * all_of
        rows, slots = s["rows"].tolist(), s["slots"].tolist()
        if kind == "write":
            whole = s["kv"].double()
            for n, (r, t) in enumerate(zip(rows, slots)):
                if case["page"]:
                    r, t = int(s["table"][r, t // case["page"]]), t % case["page"]
                whole[r, :, :, t] = kv[n]
            return {"q_out": q_out, "kv": whole}
    # rows read back, what was just written in its place
    out = s["out"].double()
    starts = [0] * B if s["starts"] is None else s["starts"].tolist()
    for b in range(B):
        L = int(s["lens_host"][b])
        if L > starts[b]:
            for plane in (0, 1):
                out[b, plane, :, :L - starts[b]] = _row64(s, b, plane, case["fmt"], L)[:, starts[b]:]
    if kind == "read":
        return {"kv": out}
    for n, (r, t) in enumerate(zip(rows, slots)):
        out[r, :, :, t] = kv[n]
    return {"q_out": q_out, "kv": out}

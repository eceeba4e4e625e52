"""Cache writes of many tokens and the read-back against their definitions in
64 bits (GPU), on the product and on the range-checked library.

Bounds, each derived from the arithmetic and not from a run:
  q_out and 16-bit keys  half a step of the stored type and 2^-19 of the head's
                         largest |z| (the FP32 norm, rotation and angles)
  16-bit values          the input bits
  e4m3                   keys within half an e4m3 step (2^-4 of the value, or
                         2^-10 below 2^-6) and the same 2^-19; values bit by bit
  int8                   the scale within half a bf16 step (2^-8) of amax / 127,
                         the code within half a step, and the same 2^-19
  e2m1                   scales and codes of keys and values equal to the
                         definition's (both zeros are one value)
  read-back              bit by bit code * scale * tensor scale in FP32, rounded
"""
import math

import numpy as np
import pytest
import torch

import gqa_decode_attention_sm_gb300 as gq
from gqa_decode_attention_sm_gb300 import _lib, api, inputs

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
TD = {"f16": torch.float16, "bf16": torch.bfloat16}
HQ, HKV, D = 32, 8, 128


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
    """A cache of random bytes (so that a stray write shows), and its scales."""
    g = gen(seed + 17)
    kind = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}.get(fmt, torch.uint8)
    shape = (units, 2, HKV, rows, 64 if fmt == "e2m1" else D)
    if fmt in TD:
        kv = torch.randn(shape, generator=g, device=DEV).to(kind)
    else:
        kv = torch.randint(0, 120, shape, generator=g, device=DEV).to(kind)
    sc = None
    if fmt == "i8":
        sc = torch.rand(shape[:4], generator=g, device=DEV).to(torch.bfloat16)
    if fmt == "e2m1":
        sc = torch.randint(0, 120, (*shape[:4], 8), generator=g, device=DEV).to(torch.uint8)
    return kv, sc


def axis_of(i, section, interleaved):
    if section is None:
        return 0
    t, h, w = section
    if interleaved:
        return 1 if i % 3 == 1 and i < 3 * h else 2 if i % 3 == 2 and i < 3 * w else 0
    return 0 if i < t else 1 if i < t + h else 2


def rotated(x, w, pos, section=None, interleaved=False, eps=1e-6, theta=1e6):
    """The definition in float64: x [N, H, 128]."""
    x = x.double()
    if w is not None:
        eps = float(np.float32(eps))
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    p = pos.double() if pos.dim() == 2 else pos.double()[None]
    f = float(np.float32(theta))
    a = torch.stack([p[axis_of(i, section, interleaved)] * f ** (-i / 64) for i in range(64)], -1)[:, None]
    c, s = torch.cos(a), torch.sin(a)
    lo, hi = x[..., :64], x[..., 64:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)


def tokens(n, batch, capacity, dtype, seed=0, fused=False, mag=1.0, axes=1):
    g = gen(seed)
    x = (torch.randn((n, HQ + 2 * HKV, D), generator=g, device=DEV) * mag
         * torch.exp(0.7 * torch.randn((1, HQ + 2 * HKV, 1), generator=g, device=DEV))).to(dtype)
    q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    at = torch.randperm(batch * capacity, generator=g, device=DEV)[:n]
    pos = torch.randint(0, 200000, (3, n), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
    w = [torch.exp(0.4 * torch.randn((D,), generator=g, device=DEV)).to(dtype) for _ in range(2)]
    return dict(q=q, k=k, v=v, qw=w[0], kw=w[1], pos=pos[0].contiguous() if axes == 1 else pos,
                rows=(at // capacity).to(torch.int32), slots=(at % capacity).to(torch.int32))


def same_codes(a, b):
    """e2m1 bytes equal, -0 being 0."""
    def clean(x):
        lo, hi = x & 15, x >> 4
        return torch.where(lo == 8, 0, lo), torch.where(hi == 8, 0, hi)
    return all(torch.equal(x, y) for x, y in zip(clean(a), clean(b)))


def check_heads(got, z):
    err = (got.double() - z).abs()
    bound = z.abs() * (torch.finfo(got.dtype).eps / 2) + z.abs().amax(-1, keepdim=True) * 2 ** -19
    # below the normal range a step is absolute
    bound = torch.clamp(bound, min=torch.finfo(got.dtype).tiny * torch.finfo(got.dtype).eps / 2)
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3f} of the bound"


def check_written(fmt, dtype, kv, sc, z, v, ks, vs):
    """Rows kv [N, 2, 8, .] (and scales) against exact keys z and values v."""
    if fmt in TD:
        check_heads(kv[:, 0], z)
        assert torch.equal(kv[:, 1], v)
        return
    slack = z.abs().amax(-1, keepdim=True) * 2 ** -19
    if fmt == "e4m3":
        got = kv[:, 0].contiguous().view(torch.float8_e4m3fn).double() * ks
        lim = torch.clamp(z, -448 * ks, 448 * ks)
        assert ((got - lim).abs() <= torch.clamp(lim.abs() * 2 ** -4, min=2 ** -10 * ks) + slack).all()
        want = (v.float() * float(np.float32(1) / np.float32(vs))).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(kv[:, 1], want.view(torch.uint8))
    elif fmt == "i8":
        for x, plane, slk in ((z, 0, slack), (v.double(), 1, slack * 0)):
            s, amax = sc[:, plane].double(), x.abs().amax(-1) / 127
            amax = torch.where(amax == 0, 1.0, amax)  # an all-zero row keeps scale 1
            assert ((s - amax).abs() <= amax * 2 ** -8 + slk[..., 0]).all()
            err = (kv[:, plane].double() * s[..., None] - x).abs()
            assert (err <= s[..., None] * (0.5 + 2 ** -16) + slk).all()
    else:
        for x, plane, s in ((z, 0, ks), (v.double(), 1, vs)):
            codes, scales = inputs.quantise_e2m1(x, float(np.float32(s)))
            assert torch.equal(sc[:, plane], scales), f"plane {plane}: {int((sc[:, plane] != scales).sum())} scales"
            assert same_codes(kv[:, plane], codes), f"plane {plane}: {int((kv[:, plane] != codes).sum())} bytes"


def page_table(batch, capacity, page, seed=0):
    n = batch * capacity // page
    table = torch.randperm(n + 3, generator=gen(seed + 5), device=DEV)[:n].to(torch.int32).view(batch, capacity // page)
    return table.contiguous(), n + 3


def run_write(t, fmt, batch, capacity, page=0, section=None, interleaved=False, norm=True, ks=1.0, vs=1.0, seed=0, **kw):
    table = None
    if page:
        table, units = page_table(batch, capacity, page, seed)
        kv, sc = new_cache(fmt, units, page, seed)
    else:
        kv, sc = new_cache(fmt, batch, capacity, seed)
    before = kv.clone(), None if sc is None else sc.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    a = (t["q"], t["k"], t["v"], t["qw"] if norm else None, t["kw"] if norm else None, t["pos"], t["rows"], t["slots"])
    how = dict(mrope_section=section, mrope_interleaved=interleaved, k_scale=ks, v_scale=vs, kv_scales=sc, workspace=ws,
               **kw)
    q_out = gq.write_kv_paged(*a, kv, table, **how) if page else gq.write_kv(*a, kv, **how)
    flags = gq.get_status(ws)
    assert not flags & api.FLAG_BOUNDS
    return q_out, kv, sc, before, table, flags


def rows_at(kv, sc, table, page, rows, slots):
    r, s = rows.long(), slots.long()
    if table is not None:
        r, s = table[r, s // page].long(), s % page
    return kv[r, :, :, s], None if sc is None else sc[r, :, :, s], (r, s)


def check_write(t, dtype, fmt, batch, capacity, page=0, section=None, interleaved=False, norm=True, ks=1.0, vs=1.0,
                seed=0, **kw):
    q_out, kv, sc, before, table, flags = run_write(t, fmt, batch, capacity, page, section, interleaved, norm, ks, vs,
                                                    seed, **kw)
    assert flags == 0
    how = dict(section=section, interleaved=interleaved, **kw_of(kw))
    check_heads(q_out, rotated(t["q"], t["qw"] if norm else None, t["pos"], **how))
    z = rotated(t["k"], t["kw"] if norm else None, t["pos"], **how)
    got, gsc, (r, s) = rows_at(kv, sc, table, page, t["rows"], t["slots"])
    check_written(fmt, dtype, got, gsc, z, t["v"], ks, vs)
    # and nothing else has changed
    before[0][r, :, :, s] = got
    assert torch.equal(before[0].view(torch.uint8), kv.view(torch.uint8))
    if sc is not None:
        before[1][r, :, :, s] = gsc
        assert torch.equal(before[1], sc)
    return q_out, kv, sc, table


def kw_of(kw):
    return {("theta" if k == "rope_theta" else k): v for k, v in kw.items() if k in ("eps", "rope_theta")}


FORMATS = [("f16", "f16"), ("bf16", "bf16"), ("e4m3", "bf16"), ("e4m3", "f16"), ("i8", "f16"), ("i8", "bf16"),
           ("e2m1", "bf16"), ("e2m1", "f16")]
SCALES = {"e4m3": (0.04, 0.03125), "e2m1": (10 / 1024, 9 / 1024)}


@pytest.mark.parametrize("fmt,dtype", FORMATS)
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("n", [1, 7, 300, 1300])
def test_write_matches_the_definition(fmt, dtype, page, n):
    ks, vs = SCALES.get(fmt, (1.0, 1.0))
    t = tokens(n, 3, 512, TD[dtype], seed=n, fused=n % 2 == 1)
    check_write(t, TD[dtype], fmt, 3, 512, page, ks=ks, vs=vs)


@pytest.mark.parametrize("section,interleaved", [((24, 20, 20), True), ((16, 24, 24), False), ((22, 21, 21), True),
                                                 ((64, 0, 0), False), ((64, 0, 0), True), ((0, 0, 64), False),
                                                 ((1, 62, 1), False), ((43, 0, 21), True)])
@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("e2m1", "f16")])
def test_rotary_axes(section, interleaved, fmt, dtype):
    t = tokens(130, 2, 100, TD[dtype], seed=3, axes=3)
    ks, vs = SCALES.get(fmt, (1.0, 1.0))
    check_write(t, TD[dtype], fmt, 2, 100, 0, section, interleaved, ks=ks, vs=vs)


def test_three_equal_axes_are_one():
    t = tokens(40, 2, 64, torch.bfloat16, seed=4, axes=3)
    t["pos"][1:] = t["pos"][0]
    a = run_write(t, "bf16", 2, 64, section=(24, 20, 20), interleaved=True)
    t["pos"] = t["pos"][0].contiguous()
    b = run_write(t, "bf16", 2, 64)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("theta,eps", [(1e4, 1e-5), (1.0, 0.0), (5e5, 1.0)])
def test_theta_and_eps(theta, eps):
    t = tokens(33, 1, 64, torch.float16, seed=5)
    check_write(t, torch.float16, "f16", 1, 64, rope_theta=theta, eps=eps)


def test_positions_at_the_ends():
    # FP64 angles themselves are only good to 2^-53 of the angle: at 2^31 that is
    # 2^-22 rad, which joins the bound (of the pair's size) in 64 bits too
    t = tokens(16, 1, 16, torch.float16, seed=6)
    t["pos"] = torch.tensor([0, 1, -1, 2, 3, 1000003, 2 ** 20, 2 ** 24 + 1, -2 ** 20, 12345678, 7, 8, 9, 10, 11, 12],
                            dtype=torch.int32, device=DEV)
    check_write(t, torch.float16, "f16", 1, 16)
    check_write(t, torch.float16, "e2m1", 1, 16, ks=0.01, vs=0.01)
    t["pos"] = torch.tensor([2 ** 31 - 1 - i for i in range(8)] + [-2 ** 31 + i for i in range(8)], dtype=torch.int32,
                            device=DEV)
    q_out = run_write(t, "f16", 1, 16)[0]
    z = rotated(t["q"], t["qw"], t["pos"])
    assert ((q_out.double() - z).abs() <= z.abs() * 2 ** -11 + z.abs().amax(-1, keepdim=True) * 2 ** -18).all()


def test_no_norm_and_ties():
    # at position 0 the rotation is the identity and, without a norm, z = x: every
    # tie of the rounding is met exactly, by keys and by values
    for dtype in TD.values():
        n = 512
        t = tokens(n, 1, n, dtype, seed=7)
        t["pos"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        t["k"] = (torch.randint(-96, 97, (n, HKV, D), generator=gen(1), device=DEV) / 16).to(dtype)
        t["v"] = (torch.randint(-96, 97, (n, HKV, D), generator=gen(2), device=DEV) / 16).to(dtype)
        check_write(t, dtype, "e2m1", 1, n, norm=False)
        check_write(t, dtype, "e2m1", 1, n, norm=False, ks=0.75, vs=1.5)
        check_write(t, dtype, "i8", 1, n, norm=False)


@pytest.mark.parametrize("mag", [1e-4, 1e3])
@pytest.mark.parametrize("fmt", ["bf16", "e2m1", "i8", "e4m3"])
def test_magnitudes(mag, fmt):
    # values far from 1: e2m1 scales in the subnormal range, and saturated ones
    t = tokens(64, 1, 64, torch.bfloat16, seed=8, mag=mag)
    check_write(t, torch.bfloat16, fmt, 1, 64, norm=False, ks=0.01, vs=0.01)
    t = tokens(64, 1, 64, torch.bfloat16, seed=9, mag=mag)
    t["k"][3] = 0
    t["v"][5] = 0
    t["v"][6, :, 16:32] = 0
    check_write(t, torch.bfloat16, fmt, 1, 64, norm=True, ks=0.01, vs=0.01)


def test_infinite_values_saturate():
    t = tokens(8, 1, 8, torch.bfloat16, seed=32)
    t["v"][0, 0, 5], t["v"][1, 3, 100], t["v"][2, 7, 0] = math.inf, -math.inf, 3e38
    t["v"][2, 7, 1] = 1e4
    q_out, kv, sc, before, table, flags = run_write(t, "e2m1", 1, 8, ks=1.0, vs=1.0)
    got, gsc, _ = rows_at(kv, sc, table, 0, t["rows"], t["slots"])
    v = inputs.dequantise_e2m1(got[:, 1], gsc[:, 1], 1.0)
    assert v[0, 0, 5] == 2688 and v[1, 3, 100] == -2688 and v[2, 7, 0] == 2688 and v[2, 7, 1] == 2688
    finite = torch.isfinite(t["v"].double()).unflatten(-1, (8, 16)).all(-1) & (t["v"].abs().amax(-1) < 1e3)[..., None]
    want, wsc = inputs.quantise_e2m1(torch.nan_to_num(t["v"].double(), posinf=0, neginf=0), 1.0)
    assert torch.equal(gsc[:, 1][finite], wsc[finite])
    assert same_codes(got[:, 1].unflatten(-1, (8, 8))[finite], want.unflatten(-1, (8, 8))[finite])


def test_many_keys_are_rounded_as_the_exact_ones():
    # about a hundredth of the units meet a rounding that FP32 cannot decide
    t = tokens(6000, 1, 6000, torch.bfloat16, seed=10, axes=3)
    check_write(t, torch.bfloat16, "e2m1", 1, 6000, section=(24, 20, 20), interleaved=True, ks=10 / 1024, vs=9 / 1024)


def test_every_key_in_doubt():
    # position 0 without a norm: z = x, and every code is a tie.  More tokens than a
    # warp's list of units in doubt holds (32, for about 33 units a warp here)
    n = 40000
    t = tokens(n, 1, n, torch.bfloat16, seed=26)
    t["pos"] = torch.zeros(n, dtype=torch.int32, device=DEV)
    level = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], device=DEV)
    x = level[torch.randint(0, 8, (n, HKV, D), generator=gen(3), device=DEV)]
    x = x * torch.where(torch.rand((n, HKV, D), generator=gen(4), device=DEV) < 0.5, -1.0, 1.0)
    x[..., ::16] = 6.0
    t["k"] = x.to(torch.bfloat16)
    check_write(t, torch.bfloat16, "e2m1", 1, n, norm=False)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("n", [20, 2500])
def test_padding_and_bad_places_write_nothing(fmt, page, n):
    t = tokens(n, 2, 2048, torch.bfloat16, seed=11)
    t["slots"][0], t["slots"][3], t["rows"][5], t["rows"][6] = -1, 2048, -1, 2
    q_out, kv, sc, before, table, flags = run_write(t, fmt, 2, 2048, page, ks=0.01, vs=0.01)
    assert flags == api.FLAG_SLOT_CLAMPED
    check_heads(q_out, rotated(t["q"], t["qw"], t["pos"]))
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[[0, 3, 5, 6]] = False
    got, gsc, (r, s) = rows_at(kv, sc, table, page, t["rows"][keep], t["slots"][keep])
    check_written(fmt, torch.bfloat16, got, gsc, rotated(t["k"], t["kw"], t["pos"])[keep], t["v"][keep], 0.01, 0.01)
    before[0][r, :, :, s] = got
    assert torch.equal(before[0].view(torch.uint8), kv.view(torch.uint8))


def test_bad_page_writes_nothing():
    t = tokens(8, 1, 64, torch.bfloat16, seed=12)
    table, units = page_table(1, 64, 16)
    kv, sc = new_cache("e2m1", units, 16)
    t["slots"] = torch.arange(8, dtype=torch.int32, device=DEV) * 8
    t["rows"].zero_()
    for bad in (units, -1, 2 ** 31 - 1):
        table[0, 1] = bad
        before = kv.clone()
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        gq.write_kv_paged(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv, table,
                          kv_scales=sc, workspace=ws)
        assert gq.get_status(ws) == api.FLAG_PAGE_CLAMPED
        changed = (kv != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert set(changed) <= {int(table[0, j]) for j in (0, 2, 3)}


def test_append_takes_the_4_bit_cache():
    for page in (0, 32):
        t = tokens(5, 5, 64, torch.bfloat16, seed=13)
        t["rows"] = torch.arange(5, dtype=torch.int32, device=DEV)
        a = run_write(t, "e2m1", 5, 64, page, ks=0.01, vs=0.02)
        table, units = page_table(5, 64, page or 64)
        kv, sc = new_cache("e2m1", units if page else 5, page or 64)
        args = (t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["slots"], kv)
        how = dict(k_scale=0.01, v_scale=0.02, kv_scales=sc)
        q_out = gq.append_kv_paged(*args, table, **how) if page else gq.append_kv(*args, **how)
        assert torch.equal(q_out, a[0]) and torch.equal(kv, a[1]) and torch.equal(sc, a[2])


@pytest.mark.parametrize("fmt", ["f16", "e4m3", "i8"])
def test_one_token_a_row_is_the_append_step(fmt):
    # both hold z to FP32 accuracy: the stored 16-bit values are neighbours at most
    t = tokens(9, 9, 32, torch.float16, seed=14)
    t["rows"] = torch.arange(9, dtype=torch.int32, device=DEV)
    a = run_write(t, fmt, 9, 32, ks=0.05, vs=0.05)
    kv, sc = new_cache(fmt, 9, 32)
    q_out = gq.append_kv(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["slots"], kv, k_scale=0.05, v_scale=0.05,
                         kv_scales=sc)
    top = q_out.double().abs().amax(-1, keepdim=True)
    assert ((q_out.double() - a[0].double()).abs() <= q_out.double().abs() * 2 ** -10 + top * 2 ** -19).all()
    assert torch.equal(kv[:, 1], a[1][:, 1])


# ------------------------------------------------------------------ read-back


def values32(kv, sc, fmt, ks, vs):
    """code * scale * tensor scale in FP32, [units, 2, 8, rows, 128]."""
    if fmt in TD:
        return kv.float()
    if fmt == "e2m1":
        x = torch.stack([inputs.dequantise_e2m1(kv[:, p], sc[:, p], 1.0) for p in (0, 1)], 1).float()
    elif fmt == "i8":
        x = kv.float() * sc.float()[..., None]
    else:
        x = kv.view(torch.float8_e4m3fn).float()
    both = torch.tensor([ks, vs], dtype=torch.float32, device=DEV).view(1, 2, 1, 1, 1)
    return x * both


def contiguous(x, table):
    return x if table is None else x[table.long()].movedim(1, 3).flatten(3, 4)


@pytest.mark.parametrize("fmt", ["f16", "bf16", "e4m3", "i8", "e2m1"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("out_capacity", [None, 100, 3])
def test_read_matches_the_definition(fmt, dtype, page, out_capacity):
    B, C = 5, 320
    table, units = (None, B) if not page else page_table(B, C, page)
    kv, sc = new_cache(fmt, units, page or C, seed=1)
    lens = torch.tensor([0, 1, 319, 320, 130], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 0, 5, 319, 130], dtype=torch.int32, device=DEV)
    want = contiguous(values32(kv, sc, fmt, 0.7, 1.3), table).to(TD[dtype])
    for st in (None, starts):
        out = torch.full((B, 2, HKV, out_capacity or C, D), -7.0, dtype=TD[dtype], device=DEV)
        ref = out.clone()
        for b in range(B):
            s = 0 if st is None else int(st[b])
            n = max(0, min(int(lens[b]) - s, out.shape[3]))
            ref[b, :, :, :n] = want[b, :, :, s:s + n]
        ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
        how = dict(starts=st, out=out, k_scale=0.7, v_scale=1.3, kv_scales=sc, workspace=ws)
        got = gq.read_kv_paged(kv, table, lens, **how) if page else gq.read_kv(kv, lens, **how)
        assert got is out and torch.equal(out, ref)
        assert gq.get_status(ws) == 0


def test_read_defaults_clamps_and_flags():
    kv, sc = new_cache("e2m1", 3, 64)
    lens = torch.tensor([70, -3, 20], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 0, 30], dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = torch.full((3, 2, HKV, 64, D), 5.0, dtype=torch.bfloat16, device=DEV)
    gq.read_kv(kv, lens, starts=starts, out=out, kv_scales=sc, workspace=ws)
    assert gq.get_status(ws) == api.FLAG_LENGTH_CLAMPED
    assert (out[1:] == 5).all()
    assert torch.equal(out[0], values32(kv, sc, "e2m1", 1, 1)[0].bfloat16())
    assert gq.read_kv(kv, lens, kv_scales=sc).dtype == torch.bfloat16
    assert gq.read_kv(kv, lens, kv_scales=sc, dtype=torch.float16).dtype == torch.float16
    half = new_cache("f16", 2, 32)[0]
    got = gq.read_kv(half, torch.tensor([32, 32], dtype=torch.int32, device=DEV))
    assert torch.equal(got, half)


def test_read_bad_pages_are_clamped_and_flagged():
    table, units = page_table(1, 64, 16)
    kv, sc = new_cache("e2m1", units, 16)
    table[0, 2] = units + 5
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    lens = torch.tensor([64], dtype=torch.int32, device=DEV)
    gq.read_kv_paged(kv, table, lens, kv_scales=sc, workspace=ws)
    assert gq.get_status(ws) == api.FLAG_PAGE_CLAMPED
    lens[0] = 32  # an entry that no slot uses is not looked at
    gq.read_kv_paged(kv, table, lens, kv_scales=sc, workspace=ws)
    assert gq.get_status(ws) == 0


# -------------------------------------------------------------------- together


def test_chunks_windows_decode_and_read_back_together():
    """A prompt with image tokens written in chunks into a paged 4-bit cache, a
    window of draft tokens written and verified, then one decode step; each
    attention against the definition on the cache's own values, and the
    read-back through the 16-bit decode."""
    B, C, page, dtype = 3, 512, 64, torch.bfloat16
    ks, vs = 10 / 1024, 9 / 1024
    table, units = page_table(B, C, page)
    kv, sc = new_cache("e2m1", units, page)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    sc_kw = dict(k_scale=ks, v_scale=vs, kv_scales=sc)

    def write(chunks, seed):
        t = tokens(sum(chunks), B, C, dtype, seed=seed, fused=True, axes=3)
        t["rows"] = torch.repeat_interleave(torch.arange(B), torch.tensor(chunks)).to(torch.int32).to(DEV)
        t["slots"] = torch.cat([torch.arange(n, device=DEV) + lens[b] for b, n in enumerate(chunks)]).to(torch.int32)
        q = gq.write_kv_paged(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv, table,
                              mrope_section=(24, 20, 20), mrope_interleaved=True, **sc_kw)
        lens.add_(torch.tensor(chunks, dtype=torch.int32, device=DEV))
        return q

    def definition(q, T):
        x = contiguous(torch.stack([inputs.dequantise_e2m1(kv[:, p], sc[:, p], s) for p, s in ((0, ks), (1, vs))], 1),
                       table)
        out = torch.zeros((B, T, HQ, D), dtype=torch.float64, device=DEV)
        for b in range(B):
            for j in range(T):
                n = int(lens[b]) - T + 1 + j
                s = torch.einsum("ghd,gtd->ght", q[b, j].double().view(8, 4, D), x[b, 0, :, :n]) / math.sqrt(D)
                out[b, j] = torch.einsum("ght,gtd->ghd", torch.softmax(s, -1), x[b, 1, :, :n]).reshape(HQ, D)
        return out, float(x[:, 1].abs().max())

    write([100, 37, 256], 1)
    write([64, 101, 3], 2)
    q3 = write([3, 3, 3], 3).view(B, 3, HQ, D)
    out = gq.gqa_decode_paged(q3, kv, table, lens, **sc_kw)
    ref, vmax = definition(q3, 3)
    assert ((out.double() - ref).abs() <= ref.abs() * 2 ** -8 + vmax * 2 ** -10).all()
    q1 = write([1, 1, 1], 4)
    out = gq.gqa_decode_paged(q1, kv, table, lens, **sc_kw)
    ref, vmax = definition(q1[:, None], 1)
    assert ((out.double()[:, None] - ref).abs() <= ref.abs() * 2 ** -8 + vmax * 2 ** -10).all()
    # the read-back rounds K and V to bf16 (2^-8 of each): the scores move by at
    # most 2^-8 of sum |q k| / sqrt(128), the weights by e^(twice that)
    back = gq.read_kv_paged(kv, table, lens, out=torch.zeros((B, 2, HKV, C, D), dtype=dtype, device=DEV), **sc_kw)
    again = gq.gqa_decode(q1, back, lens)
    x = back.double()
    move = float((q1.double().view(B, 8, 4, D).abs() @ x[:, 0].abs().transpose(-1, -2)).max()) / math.sqrt(D) * 2 ** -8
    bound = ref.abs() * 2 ** -7 + vmax * (math.expm1(2 * move) + 2 ** -8 + 2 ** -10)
    assert ((again.double()[:, None] - ref).abs() <= bound).all()


def test_streams_graphs_and_repeats_are_alike():
    t = tokens(70, 2, 64, torch.bfloat16, seed=20)
    kv, sc = new_cache("e2m1", 2, 64)
    lens = torch.tensor([64, 33], dtype=torch.int32, device=DEV)
    q_out = torch.empty_like(t["q"])
    back = torch.zeros((2, 2, HKV, 64, D), dtype=torch.bfloat16, device=DEV)

    def step():
        gq.write_kv(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv, q_out=q_out,
                    k_scale=0.01, v_scale=0.01, kv_scales=sc)
        gq.read_kv(kv, lens, out=back, k_scale=0.01, v_scale=0.01, kv_scales=sc)

    step()
    first = [x.clone() for x in (q_out, kv, sc, back)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(first, (q_out, kv, sc, back)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (q_out, kv, sc, back):
        x.zero_()
    graph.replay()
    written = torch.zeros((2, 64), dtype=torch.bool, device=DEV)
    written[t["rows"].long(), t["slots"].long()] = True
    assert torch.equal(q_out, first[0])
    assert torch.equal(kv.movedim(3, 1)[written], first[1].movedim(3, 1)[written])
    # new inputs in the same buffers: the graph reads them
    u = tokens(70, 2, 64, torch.bfloat16, seed=21)
    for k in ("q", "k", "v", "pos"):
        t[k].copy_(u[k])
    graph.replay()
    check_heads(q_out, rotated(t["q"], t["qw"], t["pos"]))


def test_offsets_past_32_bits():
    # the last slot of a 4.3 GB plane pair, and projections 2^31 elements apart
    C = 1 << 22
    kv = torch.zeros((1, 2, HKV, C, 64), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((1, 2, HKV, C, 8), dtype=torch.uint8, device=DEV)
    far = (1 << 31) + 8
    big = torch.zeros(far + HQ * D, dtype=torch.bfloat16, device=DEV)
    q = big.as_strided((2, HQ, D), (far, D, 1))
    t = tokens(2, 1, 2, torch.bfloat16, seed=22)
    q.copy_(t["q"])
    slots = torch.tensor([C - 1, C - 2], dtype=torch.int32, device=DEV)
    rows = torch.zeros(2, dtype=torch.int32, device=DEV)
    q_out = gq.write_kv(q, t["k"], t["v"], t["qw"], t["kw"], t["pos"], rows, slots, kv, k_scale=0.01, v_scale=0.01,
                        kv_scales=sc)
    check_heads(q_out, rotated(t["q"], t["qw"], t["pos"]))
    z = rotated(t["k"], t["kw"], t["pos"])
    check_written("e2m1", torch.bfloat16, kv[0, :, :, slots.long()].movedim(2, 0), sc[0, :, :, slots.long()].movedim(2, 0),
                  z, t["v"], 0.01, 0.01)
    out = torch.zeros((1, 2, HKV, 4, D), dtype=torch.float16, device=DEV)
    gq.read_kv(kv, torch.tensor([C], dtype=torch.int32, device=DEV), out=out, k_scale=0.01, v_scale=0.01, kv_scales=sc,
               starts=torch.tensor([C - 2], dtype=torch.int32, device=DEV))
    want = values32(kv[:, :, :, -2:], sc[:, :, :, -2:], "e2m1", 0.01, 0.01).half()
    assert torch.equal(out[:, :, :, :2], want) and not out[:, :, :, 2:].any()


def test_no_tokens_and_refusals():
    t = tokens(4, 2, 64, torch.bfloat16, seed=23)
    kv, sc = new_cache("bf16", 2, 64)
    good = dict(q_proj=t["q"], k_proj=t["k"], v_proj=t["v"], q_norm_w=t["qw"], k_norm_w=t["kw"], positions=t["pos"],
                rows=t["rows"], slots=t["slots"], kv=kv)
    none = {k: v[:0] for k, v in good.items() if k not in ("kv", "q_norm_w", "k_norm_w")}
    before = kv.clone()
    assert gq.write_kv(**{**good, **none}).shape == (0, HQ, D) and torch.equal(kv, before)

    def refused(kind, **kw):
        with pytest.raises(kind):
            gq.write_kv(**{**good, **kw})

    refused(TypeError, q_proj=None)
    refused(TypeError, rows=None)
    refused(ValueError, q_proj=t["q"].float())
    refused(ValueError, q_proj=t["q"].cpu())
    refused(ValueError, k_proj=t["k"][:2])
    refused(ValueError, k_proj=t["k"].half())
    refused(ValueError, v_proj=t["v"].transpose(1, 2).contiguous().transpose(1, 2))
    refused(ValueError, q_norm_w=None)
    refused(ValueError, positions=t["pos"].long())
    refused(ValueError, positions=t["pos"][None].repeat(3, 1))
    refused(ValueError, mrope_section=(24, 20, 20))
    refused(ValueError, mrope_section=(32, 32), positions=t["pos"][None].repeat(3, 1))
    refused(ValueError, kv=kv[..., :64])
    refused(ValueError, q_out=torch.empty_like(t["q"].half()))
    pos3 = t["pos"][None].repeat(3, 1)
    refused(gq.GqaError, mrope_section=(24, 20, 21), positions=pos3)
    refused(gq.GqaError, mrope_section=(-1, 33, 32), positions=pos3)
    refused(gq.GqaError, mrope_section=(20, 22, 22), positions=pos3, mrope_interleaved=True)
    refused(gq.GqaError, rope_theta=0.5)
    refused(gq.GqaError, eps=-1.0)
    refused(gq.GqaError, k_scale=0.0)
    refused(gq.GqaError, q_out=t["q"])
    refused(gq.GqaError, kv=new_cache("f16", 2, 64)[0])
    codes, scales = new_cache("e2m1", 2, 64)
    refused(TypeError, kv=codes)
    refused(ValueError, kv=codes, kv_scales=scales[..., :4].contiguous())
    refused(gq.GqaError, kv=codes, kv_scales=scales, k_scale=1e-35)
    odd = torch.zeros(4 * HQ * D + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, HQ, D)
    refused(gq.GqaError, q_proj=odd)
    lens = torch.tensor([1, 2], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        gq.read_kv(kv, lens, dtype=torch.float32)
    with pytest.raises(ValueError):
        gq.read_kv(kv, lens.long())
    with pytest.raises(ValueError):
        gq.read_kv(kv, lens, out=torch.empty((2, 2, HKV, 64, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        gq.read_kv(codes, lens)
    with pytest.raises(gq.GqaError, match="overlaps"):
        gq.read_kv(kv, lens, out=kv)
    with pytest.raises(TypeError):
        gq.read_kv_paged(kv, None, lens)


def test_the_native_binding_and_the_interpreted_one_are_alike(monkeypatch):
    assert api._native is not None, "the native binding is not built"
    t = tokens(37, 2, 64, torch.bfloat16, seed=30, fused=True, axes=3)
    table, units = page_table(2, 64, 16)
    lens = torch.tensor([64, 33], dtype=torch.int32, device=DEV)
    calls = []
    real = api._native

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(real, name)(*a)
                calls.append((name, r is not None))
                return r
            return call

    got = []
    for native in (Spy(), None):
        monkeypatch.setattr(api, "_native", native)
        for paged in (False, True):
            kv, sc = new_cache("e2m1", units if paged else 2, 16 if paged else 64)
            how = dict(mrope_section=(24, 20, 20), mrope_interleaved=True, k_scale=0.01, v_scale=0.02, kv_scales=sc)
            a = (t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"])
            out = torch.zeros((2, 2, HKV, 64, D), dtype=torch.float16, device=DEV)
            rd = dict(out=out, k_scale=0.01, v_scale=0.02, kv_scales=sc)
            if paged:
                q_out = gq.write_kv_paged(*a, kv, table, **how)
                gq.read_kv_paged(kv, table, lens, **rd)
            else:
                q_out = gq.write_kv(*a, kv, **how)
                gq.read_kv(kv, lens, **rd)
            got.append((q_out, kv, sc, out))
        # a refused call gives the same error either way
        with pytest.raises(gq.GqaError, match="sum to 64"):
            gq.write_kv(t["q"], t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"],
                        new_cache("bf16", 2, 64)[0], mrope_section=(1, 2, 3))
    assert calls == [("write", True), ("read", True)] * 2 + [("write", True)]
    for x, y in zip(got[:2], got[2:]):
        assert all(torch.equal(u, v) for u, v in zip(x, y))


def test_a_stream_of_its_own_and_tensors_made_elsewhere():
    # the call runs on the current stream, whichever stream made its tensors
    t = tokens(500, 1, 500, torch.bfloat16, seed=31)
    ref = run_write(t, "bf16", 1, 500)
    kv = new_cache("bf16", 1, 500)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms: a call on another stream would pass it
        q = t["q"] * 1
        q_out = gq.write_kv(q, t["k"], t["v"], t["qw"], t["kw"], t["pos"], t["rows"], t["slots"], kv)
    side.synchronize()
    assert torch.equal(q_out, ref[0]) and torch.equal(kv, ref[1])


def random_call(seed):
    """One random write, read back and (e2m1) decoded, each against its definition."""
    rng = np.random.default_rng(seed)
    fmt, dtype = FORMATS[rng.integers(len(FORMATS))] if rng.random() < 0.5 else ("e2m1", "bf16")
    page = int(rng.choice([0, 16, 32, 128]))
    B = int(rng.integers(1, 6))
    C = int(np.exp(rng.uniform(np.log(16), np.log(1500))))
    C = -(-C // (page or 8)) * (page or 8)
    n = int(min(B * C, np.exp(rng.uniform(0, np.log(4000)))))
    axes = int(rng.choice([1, 3]))
    interleaved = bool(rng.random() < 0.5)
    section = None
    if axes == 3:
        h, w = (int(x) for x in rng.integers(0, 22 if interleaved else 33, 2))
        section = (64 - h - w, h, w)
    ks, vs = (float(np.float32(x)) for x in np.exp(rng.uniform(-6, -2, 2))) if fmt in SCALES else (1.0, 1.0)
    t = tokens(n, B, C, TD[dtype], seed=seed, fused=bool(rng.random() < 0.5), axes=axes, mag=float(np.exp(rng.uniform(-3, 3))))
    t["pos"] = torch.randint(0, 1 << int(rng.integers(1, 23)), t["pos"].shape, generator=gen(seed + 1), device=DEV,
                             dtype=torch.int64).to(torch.int32)
    q_out, kv, sc, table = check_write(t, TD[dtype], fmt, B, C, page, section, interleaved, norm=bool(rng.random() < 0.8),
                                       ks=ks, vs=vs, seed=seed)
    if fmt == "e2m1":
        sc.clamp_(max=0x7E)
    lens = torch.tensor(rng.integers(0, C + 1, B), dtype=torch.int32, device=DEV)
    starts = torch.tensor([int(rng.integers(0, int(x) + 1)) for x in lens], dtype=torch.int32, device=DEV)
    want = contiguous(values32(kv, sc, fmt, ks, vs), table)
    out = torch.full((B, 2, HKV, int(rng.integers(1, C + 9)), D), 3.0, dtype=TD[dtype], device=DEV)
    ref = out.clone()
    for b in range(B):
        s, m = int(starts[b]), min(int(lens[b]) - int(starts[b]), out.shape[3])
        ref[b, :, :, :m] = want[b, :, :, s:s + m].to(TD[dtype])
    how = dict(starts=starts, out=out, k_scale=ks, v_scale=vs, kv_scales=sc)
    got = gq.read_kv_paged(kv, table, lens, **how) if page else gq.read_kv(kv, lens, **how)
    assert torch.equal(got, ref)
    if fmt != "e2m1":
        return
    T = int(rng.integers(1, 5))
    q = torch.randn((B, T, HQ, D) if T > 1 else (B, HQ, D), generator=gen(seed + 2), device=DEV).to(TD[dtype])
    S = int(rng.integers(1, 20))
    q_scale = float(np.float32(1.0 / max(1.0, float(want[:, 0].square().mean().sqrt()))))  # scores of the order of one
    sc_kw = dict(k_scale=ks, v_scale=vs, kv_scales=sc, q_scale=q_scale, num_splits=S)
    if page:
        o = gq.gqa_decode_paged(q, kv, table, lens, **sc_kw)
    else:
        o = gq.gqa_decode_verify(q if T > 1 else q[:, None].contiguous(), kv, lens, **sc_kw).view(q.shape)
    x = want.double()
    ref = torch.zeros((B, T, HQ, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        for j in range(T):
            m = int(lens[b]) - T + 1 + j
            if m > 0:
                s = torch.einsum("ghd,gtd->ght", q.view(B, T, HQ, D)[b, j].double().view(8, 4, D), x[b, 0, :, :m])
                ref[b, j] = torch.einsum("ght,gtd->ghd", torch.softmax(s * q_scale / math.sqrt(D), -1),
                                         x[b, 1, :, :m]).reshape(HQ, D)
    # half a step of the output; the weights' rounding to fp16 (2^-11 and 2^-25 a
    # token) and the scores' (2^-13), each of the largest value
    top = float(x[:, 1].abs().max())
    bound = ref.abs() * (torch.finfo(o.dtype).eps / 2) + top * (2 ** -11 + C * 2 ** -25 + 2 ** -13) + 2 ** -25
    assert ((o.view(ref.shape).double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    random_call(seed)

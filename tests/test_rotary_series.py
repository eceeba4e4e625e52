"""The sine and cosine that the many-token write forms from a 64-bit fraction of a turn, emulated operation by
operation on the CPU: how far they are from the exact ones (the write's bounds rest on it)."""
import numpy as np

F = np.float32


def fma(a, b, c):
    """FP32 a * b + c with one rounding: the product is exact in FP64, the sum there good to 2^-53."""
    return (a.astype(np.float64) * np.float64(b) + np.float64(c)).astype(F)


def sincos_turn(h):
    """write_kv.cuh's sincos_turn for the high words h (uint32) of a turn."""
    quad = (h + np.uint32(0x20000000)) >> np.uint32(30)
    r = (h - (quad << np.uint32(30))).astype(np.int32)
    unit = F(1.46291807926715968e-9)
    rf = r.astype(F)
    x = rf * unit
    rest = fma((r - rf.astype(np.int64)).astype(F), unit, fma(rf, unit, -x) + rf * F(-4.0709404e-17))
    x2 = x * x
    sp = fma(x2, F(2.75573192e-6), F(-1.98412698e-4))
    sp = fma(x2, sp, F(8.33333333e-3))
    sp = fma(x2, sp, F(-1.66666667e-1))
    sx = fma(x * x2, sp, x)
    cp = fma(x2, F(-2.75573192e-7), F(2.48015873e-5))
    cp = fma(x2, cp, F(-1.38888889e-3))
    cp = fma(x2, cp, F(4.16666667e-2))
    cp = fma(x2, cp, F(-0.5))
    cx = fma(x2, cp, F(1))
    sx, cx = fma(cx, rest, sx), fma(-sx, rest, cx)
    s, c = np.where(quad & 1, cx, sx), np.where(quad & 1, sx, cx)
    return np.where(quad & 2, -s, s), np.where((quad + 1) & 2, -c, c)


def test_sine_and_cosine_are_within_three_halves_of_2_to_the_minus_24():
    rng = np.random.default_rng(0)
    h = np.concatenate([rng.integers(0, 1 << 32, 1 << 21, dtype=np.uint64),
                        np.arange(0, 1 << 32, 4099, dtype=np.uint64),
                        # the quadrants' borders, where the reduced angle is largest or 0
                        (np.arange(8)[:, None] * (1 << 29) + np.arange(-2048, 2048)).ravel().astype(np.uint64)
                        & np.uint64(0xFFFFFFFF)]).astype(np.uint32)
    s, c = sincos_turn(h)
    # a turn's fraction h / 2^32 as an angle of at most pi / 4 and its quadrant, in FP64
    quad = np.floor(h.astype(np.float64) / 2 ** 30 + 0.5)
    a = (h.astype(np.float64) - quad * 2 ** 30) * (2 * np.pi / 2 ** 32)
    q = quad.astype(np.int64) % 4
    es = np.choose(q, [np.sin(a), np.cos(a), -np.sin(a), -np.cos(a)])
    ec = np.choose(q, [np.cos(a), -np.sin(a), -np.cos(a), np.sin(a)])
    # In units of 2^-24, half an ulp of a number in [1/2, 1) is 1/2: the series' last FMA and the correction's make
    # 1.  The rest of the series, at most x^2 / 2 = 0.31 for a cosine and x^3 / 6 = 0.081 for a sine, brings two
    # roundings of itself (one unit each) and its coefficients' (1/2): below 0.4 more.
    assert np.abs(s - es).max() <= 1.5 * 2 ** -24
    assert np.abs(c - ec).max() <= 1.5 * 2 ** -24

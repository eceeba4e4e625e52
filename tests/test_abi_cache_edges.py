"""Refusals at the edges of the cache write and read-back calls (no GPU: validation answers before any CUDA call)."""
from test_abi_fp4 import EINVAL, P, _write, lib  # noqa: F401

E4M3 = 2


def test_e4m3_scales_without_a_normal_reciprocal(lib):  # noqa: F811
    for kw in (dict(k_=2.0 ** -127), dict(v_=1e-40), dict(k_=2.0 ** 127), dict(v_=3e38)):
        assert _write(lib, fmt=E4M3, **kw) == EINVAL, kw
        assert _write(lib, True, fmt=E4M3, **kw) == EINVAL, kw

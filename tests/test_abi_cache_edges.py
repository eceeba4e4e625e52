"""Refusals at the edges of the cache write and read-back calls (no GPU: validation answers before any CUDA call)."""
import subprocess
import sys

import pytest
import torch

from gqa_decode_attention_sm_gb300 import _lib, api, build
from test_abi_fp4 import EALIAS, EINVAL, P, _write, lib  # noqa: F401

E4M3 = 2


def test_e4m3_scales_without_a_normal_reciprocal(lib):  # noqa: F811
    for kw in (dict(k_=2.0 ** -127), dict(v_=1e-40), dict(k_=2.0 ** 127), dict(v_=3e38)):
        assert _write(lib, fmt=E4M3, **kw) == EINVAL, kw
        assert _write(lib, True, fmt=E4M3, **kw) == EINVAL, kw


def test_the_binding_is_for_the_librarys_own_interface(lib, monkeypatch):  # noqa: F811
    build.build_native()
    assert api._native is not None and api._native.interface == build.interface() == lib.gqa_interface().decode()
    assert _lib.address("gqa_write_kv") != 0
    # a library of another interface is not called by address, and the native call says "not judged"
    monkeypatch.setattr(_lib, "binding_interface", "h0")
    assert _lib.address("gqa_write_kv") == 0
    assert api._native.write(_lib.address("gqa_write_kv"), *[None] * 20) is None


def test_a_binding_for_another_torch_python_or_header_is_built_again(tmp_path, monkeypatch):
    path = build.build_native()
    assert build.native_is_current(path)
    copy = tmp_path / "_native.so"
    with open(path, "rb") as f:
        data = f.read()
    mark = build.native_built_for().encode()
    assert mark in data
    copy.write_bytes(data.replace(mark, b"x" * len(mark)))
    assert not build.native_is_current(str(copy))
    assert not build.native_is_current(str(tmp_path / "absent.so"))
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert not build.native_is_current(path)


def test_importing_the_package_loads_no_binary():
    code = ("import gqa_decode_attention_sm_gb300 as gq\n"
            "maps = lambda: [x for x in open('/proc/self/maps').read().split() if 'gqa_decode_attention_sm_gb300' in x]\n"
            "assert not maps(), maps()\n"
            "from gqa_decode_attention_sm_gb300 import api\n"
            "assert api._binding() is not None and any(x.endswith('_native.so') for x in maps())\n")
    build.build_native()
    subprocess.run([sys.executable, "-c", code], check=True, cwd=build.ROOT)


def test_a_read_backs_workspace_overlaps_no_input(lib):  # noqa: F811
    # (a flag set in it would change the cache or the lengths)
    def call(ws, paged=False):
        kv, sc, lens, starts, out, table = P[:6]
        if paged:
            return lib.gqa_read_kv_paged(kv, 4, sc, table, 4, 16, 64, lens, starts, out, 1, 2, 64, 1.0, 1.0, ws, 256, None)
        return lib.gqa_read_kv(kv, 4, sc, lens, starts, out, 1, 2, 64, 64, 1.0, 1.0, ws, 256, None)

    for ws in (P[0] + 64, P[1], P[2] - 252, P[3], P[4] - 128):
        assert call(ws) == EALIAS and call(ws, True) == EALIAS
    assert call(P[5], True) == EALIAS


@pytest.mark.parametrize("which", ["build", "build_checked", "build_native"])
def test_a_build_that_fails_is_told_even_beside_an_older_binary(which, monkeypatch):
    import __graft_entry__ as entry

    def broken(**kw):
        raise subprocess.CalledProcessError(1, "nvcc")

    for name in ("build", "build_checked", "build_native"):
        monkeypatch.setattr(build, name, broken if name == which else lambda **kw: None)
    with pytest.raises(subprocess.CalledProcessError):
        entry.build()

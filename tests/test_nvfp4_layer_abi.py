"""Refusals of the NVFP4 layer's entry points, on a host without a GPU: every
invalid call returns its documented status before the device is touched.  No
pointer passed here is dereferenced."""
import ctypes

import pytest

A = 0x100000          # a 256-byte aligned address; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    from adaptive_block_scaled_b200 import build
    L = ctypes.CDLL(build.build())
    vp, i64, i, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.nvfp4_linear.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, sz, vp, i, vp, vp]
    L.nvfp4_linear_workspace_bytes.argtypes = [i64, i64, i64]
    L.nvfp4_linear_workspace_bytes.restype = sz
    return L


BIG = 1 << 40


def linear(lib, **kw):
    d = dict(ac=A, asc=A, at=A, bc=A, bs=A, bt=A, M=4, N=64, K=64, ws=A, n=BIG, c=A, dt=1, err=A)
    d.update(kw)
    return lib.nvfp4_linear(d["ac"], d["asc"], d["at"], d["bc"], d["bs"], d["bt"], d["M"], d["N"],
                            d["K"], d["ws"], d["n"], d["c"], d["dt"], d["err"], None)


def test_linear_refusals(lib):
    for k in ("ac", "asc", "at", "bc", "bs", "bt", "c", "err"):
        assert linear(lib, **{k: None}) == 1, k
    for kw in (dict(K=0), dict(K=16), dict(K=48), dict(K=-32), dict(M=-1), dict(N=-1),
               dict(M=(1 << 22) + 1), dict(N=(1 << 22) + 1), dict(K=(1 << 20) + 32)):
        assert linear(lib, **kw) == 2, kw
    assert linear(lib, dt=3) == 3 and linear(lib, dt=-1) == 3
    for kw in (dict(ac=A + 8), dict(bc=A + 8), dict(asc=A + 2), dict(bs=A + 2), dict(at=A + 2),
               dict(bt=A + 1), dict(c=A + 1), dict(c=A + 2, dt=0), dict(err=A + 2),
               dict(M=256, N=256, ws=A + 128)):
        assert linear(lib, **kw) == 4, kw
    need = lib.nvfp4_linear_workspace_bytes(256, 256, 64)
    assert need > 0
    assert linear(lib, M=256, N=256, ws=None) == 6
    assert linear(lib, M=256, N=256, n=need - 1) == 6


def test_linear_empty_is_ok(lib):
    assert linear(lib, M=0, c=None, ac=None) == 0
    assert linear(lib, N=0, c=None, bc=None) == 0


def test_linear_workspace(lib):
    f = lib.nvfp4_linear_workspace_bytes
    assert f(1, 4096, 4096) == 0 and f(4096, 16, 64) == 0     # few rows, few columns
    assert f(256, 512, 256) == (2 + 4) * 2048                 # 128 rows x 16 scales
    assert f(257, 512, 288) == (3 + 4) * 2 * 2048             # rows and K rounded up
    for bad in ((0, 4, 64), (4, 0, 64), (4, 4, 16), (4, 4, 40), (1 << 23, 4, 64)):
        assert f(*bad) == 0

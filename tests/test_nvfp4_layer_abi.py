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
    for n in ("if4", "nvfp4"):
        getattr(L, n + "_quantize_t").argtypes = [vp, i, i64, i64, i64, vp, vp, vp, vp, vp, i, vp, vp]
        getattr(L, n + "_rms_norm_quantize").argtypes = [
            vp, i64, vp, i64, vp, i, i, i64, i64, ctypes.c_float, vp, i64, vp, vp, vp, vp, vp, vp, vp]
    L.if4_rms_norm_backward_workspace_bytes.argtypes = [i64, i64]
    L.if4_rms_norm_backward_workspace_bytes.restype = sz
    L.if4_rms_norm_backward.argtypes = [vp, i64, vp, i64, vp, i, vp, vp, i64, i, i64, i64, vp, i64,
                                        vp, vp, sz, vp]
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
    for kw in (dict(ac=A + 8), dict(bc=A + 8), dict(asc=A + 1), dict(bs=A + 1), dict(at=A + 2),
               dict(bt=A + 1), dict(c=A + 1), dict(c=A + 2, dt=0), dict(err=A + 2),
               dict(M=1024, N=1280, ws=A + 128)):
        assert linear(lib, **kw) == 4, kw
    need = lib.nvfp4_linear_workspace_bytes(1024, 1280, 64)
    assert need > 0
    assert linear(lib, M=1024, N=1280, ws=None) == 6
    assert linear(lib, M=1024, N=1280, n=need - 1) == 6


def test_linear_empty_is_ok(lib):
    assert linear(lib, M=0, c=None, ac=None) == 0
    assert linear(lib, N=0, c=None, bc=None) == 0


def test_linear_workspace(lib):
    f = lib.nvfp4_linear_workspace_bytes
    assert f(1, 4096, 4096) == 0 and f(64, 1 << 20, 64) == 0 and f(256, 256, 64) == 0
    # blocks of 128 rows x 16 scales: two per 256 rows of A, two per 240 of B
    assert f(1024, 1440, 256) == (8 + 12) * 2048
    assert f(1025, 1441, 288) == (10 + 14) * 2 * 2048         # rows and K rounded up
    for bad in ((0, 4, 64), (4, 0, 64), (4, 4, 16), (4, 4, 40), (1 << 23, 4, 64)):
        assert f(*bad) == 0


@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
def test_quantize_t_refusals(lib, mode):
    f = getattr(lib, mode + "_quantize_t")

    def call(x=A, dt=1, r=32, c=32, ld=32, co=A, s=A, ct=A, st=A, ts=A, m=0, err=None):
        return f(x, dt, r, c, ld, co, s, ct, st, ts, m, err, None)

    for k in ("x", "ct", "st", "ts", "co", "s"):      # codes and scales go together
        assert call(**{k: None}) == 1, k
    for kw in (dict(r=24), dict(c=24, ld=24), dict(r=-16), dict(ld=16), dict(r=1 << 31)):
        assert call(**kw) == 2, kw
    assert call(dt=5) == 3 and call(m=2) == 5
    for kw in (dict(x=A + 8), dict(ld=36), dict(co=A + 8), dict(ct=A + 8), dict(ts=A + 2),
               dict(err=A + 1)):
        assert call(**kw) == 4, kw


@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
def test_rms_norm_quantize_refusals(lib, mode):
    f = getattr(lib, mode + "_rms_norm_quantize")

    def call(x=A, ldx=64, res=A, ldr=64, w=A, wdt=1, dt=1, r=4, c=64, eps=1e-6, h=A, ldh=64,
             rstd=A, co=A, s=A, ts=A, amax=A, err=A):
        return f(x, ldx, res, ldr, w, wdt, dt, r, c, eps, h, ldh, rstd, co, s, ts, amax, err, None)

    for k in ("x", "w", "co", "s", "ts"):
        assert call(**{k: None}) == 1, k
    wide = (1 << 22) + 16
    for kw in (dict(c=40), dict(r=-1), dict(ldx=32), dict(ldr=32), dict(ldh=32),
               dict(c=wide, ldx=wide, ldr=wide, ldh=wide)):
        assert call(**kw) == 2, kw
    for kw in (dict(dt=4), dict(wdt=2), dict(wdt=7), dict(dt=0, wdt=1)):
        assert call(**kw) == 3, kw
    for kw in (dict(x=A + 8), dict(res=A + 8), dict(h=A + 8), dict(w=A + 8), dict(ldx=68),
               dict(ldr=68), dict(ldh=68), dict(co=A + 8), dict(rstd=A + 2), dict(ts=A + 2),
               dict(amax=A + 2), dict(err=A + 2)):
        assert call(**kw) == 4, kw
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == 5, eps


def test_rms_norm_backward_refusals(lib):
    def call(dy=A, ldy=64, h=A, ldh=64, w=A, wdt=1, rstd=A, dres=A, ldr=64, dt=1, r=4, c=64, dx=A,
             ldx=64, dw=A, ws=A, n=BIG):
        return lib.if4_rms_norm_backward(dy, ldy, h, ldh, w, wdt, rstd, dres, ldr, dt, r, c, dx, ldx,
                                         dw, ws, n, None)

    for k in ("dy", "h", "w", "rstd", "dx", "dw"):
        assert call(**{k: None}) == 1, k
    for kw in (dict(c=40), dict(r=-1), dict(ldy=32), dict(ldh=32), dict(ldr=32), dict(ldx=32)):
        assert call(**kw) == 2, kw
    for kw in (dict(dt=4), dict(wdt=2)):
        assert call(**kw) == 3, kw
    for kw in (dict(dy=A + 8), dict(h=A + 8), dict(w=A + 8), dict(dres=A + 8), dict(dx=A + 8),
               dict(ldy=68), dict(rstd=A + 2), dict(dw=A + 2), dict(ws=A + 64)):
        assert call(**kw) == 4, kw
    need = lib.if4_rms_norm_backward_workspace_bytes(4, 64)
    assert need == 4 * 64 * 4
    assert call(ws=None) == 6 and call(n=need - 1) == 6
    assert lib.if4_rms_norm_backward_workspace_bytes(1 << 20, 64) == 296 * 64 * 4
    for bad in ((0, 64), (4, 0), (4, 40), (1 << 31, 64), (1, (1 << 22) + 16)):
        assert lib.if4_rms_norm_backward_workspace_bytes(*bad) == 0


def test_python_refusals():
    """Errors of the binding that need no device: shapes, types, overlapping rows."""
    import torch

    from adaptive_block_scaled_b200 import binding as b
    x = torch.zeros((32, 32))
    with pytest.raises(ValueError, match="CUDA"):
        b.quantize_t(x)
    with pytest.raises(ValueError, match="mode"):
        b.quantize_t(x, "int8")
    with pytest.raises(ValueError, match="overlap"):
        b.quantize_t(torch.zeros((1, 32)).expand(32, 32))
    with pytest.raises(ValueError, match="contiguous rows"):
        b.quantize_t(torch.zeros((32, 48)).T)
    with pytest.raises(ValueError, match="mode"):
        b.rms_norm_quantize(x, torch.ones(32), torch.ones(1), mode="bf16")
    with pytest.raises(ValueError, match="CUDA"):
        b.rms_norm_quantize(x, torch.ones(32), torch.ones(1))
    with pytest.raises(ValueError, match="CUDA"):
        b.rms_norm_backward(x, x, torch.ones(32), torch.ones(32))
    u = torch.zeros((32, 16), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        b.linear_nvfp4((u, u, torch.ones(1)), (u, u, torch.ones(1)))

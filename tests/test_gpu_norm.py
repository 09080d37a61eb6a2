"""GPU tests of the RMS norm with a quantized output and of its gradient.

Forward: h, rstd, codes and scale bytes must be those of the stated
arithmetic (binary64 statistics, binary32 products, the oracle's quantizer),
bit for bit.  Gradient: against the formula in binary64 and against
differences.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

MODES = {"if4": oracle.MODE_IF4, "nvfp4": oracle.MODE_NVFP4}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
U = 2.0 ** -24


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def data(rows, cols, dtype, seed, wdtype=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    x[:, torch.rand((cols,), generator=g) < 0.02] *= 20.0
    r = torch.randn((rows, cols), generator=g)
    w = 1.0 + 0.1 * torch.randn((cols,), generator=g)
    return x.to(dtype), r.to(dtype), w.to(wdtype or dtype)


def reference(x, r, w, eps):
    """h (x's type), rstd and y as float32 arrays, in the stated arithmetic."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h64 = h.double().numpy()
    rstd = (1.0 / np.sqrt((h64 * h64).sum(1) / x.shape[1] + float(np.float32(eps)))).astype(np.float32)
    y = (h.float().numpy() * rstd[:, None]) * w.float().numpy()[None, :]
    return h, rstd, y


def check(x, r, w, mode="if4", ts=0.012, eps=1e-6, inplace=None):
    """x, r, w on the host, strides kept on the device by the caller."""
    bb = B()
    xd, rd, wd = x.cuda(), None if r is None else r.cuda(), w.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    amax = torch.zeros(1, device="cuda")
    t = torch.tensor([ts], device="cuda")
    codes, scales, h, rstd = bb.rms_norm_quantize(xd, wd, t, residual=rd, eps=eps, mode=mode,
                                                  amax=amax, err_flag=err)
    torch.cuda.synchronize()
    h0, rstd0, y0 = reference(x, r, w, eps)
    assert int(err) == 0
    assert torch.equal(h.cpu(), h0)
    assert np.array_equal(rstd.cpu().numpy(), rstd0)
    assert np.float32(amax.item()) == np.abs(y0).max()
    q = oracle.quantize(y0, np.float32(ts), mode=MODES[mode])
    assert np.array_equal(scales.cpu().numpy(), q["scales"])
    assert np.array_equal(codes.cpu().numpy(), q["codes"])


SIZES = [(1, 16), (3, 48), (1, 4096), (5, 416), (37, 5008), (300, 1024), (130, 4096), (64, 8192),
         (9, 16400), (4, 33024), (2, 70000), (2000, 256)]


@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(rows, cols, dtype, mode):
    x, r, w = data(rows, cols, dtype, rows * 3 + cols)
    check(x, r if (rows + cols) % 3 else None, w, mode)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(7, 1024), (33, 5008), (3, 33024)])
def test_forward_float32_weight(rows, cols, dtype):
    x, r, w = data(rows, cols, dtype, 5, torch.float32)
    check(x, r, w)


@pytest.mark.parametrize("dtype", DTYPES)
def test_zero_rows_and_large_and_small_values(dtype):
    x, _, w = data(9, 512, dtype, 8)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 1e-3
    x[3] = 0.0
    x[3, 7] = 100.0
    if dtype != torch.float16:
        x[4] *= 1e15                      # squares past binary32's range
        x[5] *= 1e-25
    check(x, None, w, eps=1e-12)
    check(x, None, w, eps=0.5, mode="nvfp4")


@pytest.mark.parametrize("ts", [1e-6, 1.0, 1e6])
def test_saturating_and_vanishing_block_scales(ts):
    x, r, w = data(17, 2048, torch.bfloat16, 3)
    check(x, r, w, ts=ts)
    check(x, r, w, ts=ts, mode="nvfp4")


@pytest.mark.parametrize("cols", [400, 4096, 33024])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_in_place(which, cols):
    bb = B()
    x, r, w = data(21, cols, torch.bfloat16, 4)
    xd, rd = x.cuda(), r.cuda()
    codes = torch.empty((21, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((21, cols // 16), dtype=torch.uint8, device="cuda")
    ts = torch.tensor([0.01], device="cuda")
    h = xd if which == "x" else rd
    bb.if4_rms_norm_quantize(xd, rd, w.cuda(), 1e-5, h, None, codes, scales, ts)
    h0, _, y0 = reference(x, r, w, 1e-5)
    assert torch.equal(h.cpu(), h0)
    q = oracle.quantize(y0, np.float32(0.01))
    assert np.array_equal(codes.cpu().numpy(), q["codes"])
    assert np.array_equal(scales.cpu().numpy(), q["scales"])


@pytest.mark.parametrize("cols", [400, 4096, 33024])
@pytest.mark.parametrize("dtype", DTYPES)
def test_strides_and_no_writes_outside(dtype, cols):
    bb = B()
    rows = 11
    unit = 4 if dtype == torch.float32 else 8          # 16 bytes
    x, r, w = data(rows, cols, dtype, 6)
    big = [torch.full((rows + 2, cols + 3 * unit), 7.0, dtype=dtype, device="cuda") for _ in range(3)]
    xd, rd, hd = (b[1:rows + 1, k * unit:k * unit + cols] for k, b in zip((1, 2, 0), big))
    xd.copy_(x), rd.copy_(r)
    cb = torch.full((16 + rows * cols // 2 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sb = torch.full((16 + rows * cols // 16 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    codes = cb[16:16 + rows * cols // 2].view(rows, cols // 2)
    scales = sb[16:16 + rows * cols // 16].view(rows, cols // 16)
    rstd = torch.full((rows + 2,), 7.0, device="cuda")
    bb.nvfp4_rms_norm_quantize(xd, rd, w.cuda(), 1e-6, hd, rstd[1:-1], codes, scales,
                               torch.tensor([0.01], device="cuda"))
    h0, rstd0, y0 = reference(x, r, w, 1e-6)
    q = oracle.quantize(y0, np.float32(0.01), mode=oracle.MODE_NVFP4)
    assert np.array_equal(codes.cpu().numpy(), q["codes"])
    assert np.array_equal(scales.cpu().numpy(), q["scales"])
    assert torch.equal(hd.cpu(), h0) and np.array_equal(rstd[1:-1].cpu().numpy(), rstd0)
    out = big[2].clone()
    out[1:rows + 1, :cols] = 7.0
    assert torch.all(out == 7.0) and float(rstd[0]) == 7.0 and float(rstd[-1]) == 7.0
    for f, n in ((cb, rows * cols // 2), (sb, rows * cols // 16)):
        assert torch.all(f[:16] == 0xA5) and torch.all(f[16 + n:] == 0xA5)


@pytest.mark.parametrize("cols", [400, 4096, 33024])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_nonfinite_is_reported_and_stays_in_its_row(bad, cols):
    bb = B()
    x, _, w = data(6, cols, torch.bfloat16, 2)
    xb = x.clone()
    xb[2, 77] = bad
    ts = torch.tensor([0.01], device="cuda")
    good = bb.rms_norm_quantize(x.cuda(), w.cuda(), ts)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = bb.rms_norm_quantize(xb.cuda(), w.cuda(), ts, err_flag=err)
    assert int(err) == bb.DEV_NONFINITE
    keep = torch.tensor([0, 1, 3, 4, 5], device="cuda")
    assert torch.equal(good[0][keep], got[0][keep]) and torch.equal(good[1][keep], got[1][keep])


def test_invalid_tensor_scale_is_reported():
    bb = B()
    x, _, w = data(2, 32, torch.bfloat16, 2)
    for ts in (0.0, -1.0, float("nan"), float("inf")):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        bb.rms_norm_quantize(x.cuda(), w.cuda(), torch.tensor([ts], device="cuda"), err_flag=err)
        assert int(err) & bb.DEV_BAD_SCALE


def test_amax_is_raised_not_overwritten_and_gives_the_next_scale():
    bb = B()
    x, _, w = data(40, 1024, torch.bfloat16, 12)
    ts = torch.tensor([0.01], device="cuda")
    amax = torch.tensor([1e4], device="cuda")
    bb.rms_norm_quantize(x.cuda(), w.cuda(), ts, amax=amax)
    assert float(amax) == 1e4
    amax.zero_()
    bb.rms_norm_quantize(x.cuda(), w.cuda(), ts, amax=amax)
    bb.if4_tensor_scale(amax, ts)
    y0 = reference(x, None, w, 1e-6)[2]
    assert np.float32(ts.item()) == oracle.tensor_scale(np.abs(y0).max())


def test_empty():
    bb = B()
    w = torch.ones(64, device="cuda")
    ts = torch.ones(1, device="cuda")
    codes, scales, h, rstd = bb.rms_norm_quantize(torch.empty((0, 64), device="cuda"), w, ts)
    assert codes.shape == (0, 32) and rstd.shape == (0,)
    dx, dw = bb.rms_norm_backward(torch.empty((0, 64), device="cuda"),
                                  torch.empty((0, 64), device="cuda"), w,
                                  torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros_like(dw))


# -------------------------------------------------------------- gradient ----

def formula(dy, h, w, rstd, dres):
    """dx, dw and the sums of magnitudes that bound their rounding, binary64."""
    dy, h, w = dy.double(), h.double(), w.double()
    rs = rstd.double().unsqueeze(1)
    n, g = h * rs, dy * w
    C = h.shape[1]
    dx = rs * (g - n * (g * n).mean(1, keepdim=True))
    mag = rs * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dres is not None:
        dx, mag = dx + dres.double(), mag + dres.double().abs()
    return dx, (dy * n).sum(0), mag, (dy * n).abs().sum(0), C


def check_backward(dy, h, w, dres, eps=1e-6):
    bb = B()
    rstd = (1.0 / (h.double().square().mean(1) + eps).sqrt()).float()
    dx, dw = bb.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(),
                                  dres=None if dres is None else dres.cuda())
    torch.cuda.synchronize()
    dx0, dw0, mag, magw, C = formula(dy, h, w, rstd, dres)
    # the row sum: a chain of at most 8 + C / 256 additions per thread, then at most
    # 16 levels; eight more roundings on the way to dx; half a step of its type
    steps = C / 256 + 32
    half = torch.finfo(h.dtype).eps / 2
    tol = half * dx0.abs() + mag * (steps * U * (1 + half)) + \
        (2.0 ** -25 if h.dtype == torch.float16 else 0.0)
    d = (dx.cpu().double() - dx0).abs()
    assert torch.all(d <= tol), float((d / tol.clamp(min=1e-300)).max())
    # dw: a chain over a block's rows, then over the blocks; three roundings a term
    rows = h.shape[0]
    tolw = magw * ((rows / 296 + 296 + 8) * U)
    dd = (dw.cpu().double() - dw0).abs()
    assert torch.all(dd <= tolw), float((dd / tolw.clamp(min=1e-300)).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_backward(rows, cols, dtype):
    x, r, w = data(rows, cols, dtype, rows + cols)
    g = torch.Generator().manual_seed(1)
    dy = (0.1 * torch.randn((rows, cols), generator=g)).to(dtype)
    check_backward(dy, x, w, r if (rows + cols) % 3 else None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(7, 1024), (303, 5008), (3, 33024)])
def test_backward_float32_weight(rows, cols, dtype):
    x, r, w = data(rows, cols, dtype, 5, torch.float32)
    check_backward(r.clone(), x, w, r)


def test_backward_many_rows():
    x, r, w = data(6000, 512, torch.bfloat16, 5)
    check_backward(r, x, w, r)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [400, 16384, 33024])
def test_backward_products_past_float32(cols, dtype):
    """dy * h leaves binary32's range, dy * n and the gradients do not."""
    x, r, w = data(19, cols, dtype, 12)
    h, dy = x.float(), r.float()
    h[::3] *= 1e30
    dy[::2] *= 1e12
    h[1] = 0.0
    check_backward(dy.to(dtype), h.to(dtype), w, None)


@pytest.mark.parametrize("cols", [400, 4096, 33024])
@pytest.mark.parametrize("which", ["dy", "dres"])
def test_backward_in_place(which, cols):
    bb = B()
    x, r, w = data(301, cols, torch.bfloat16, 9)
    dy, dres = r.cuda(), (0.5 * r).cuda()
    rstd = torch.rand(301, device="cuda") + 0.5
    want, dww = bb.rms_norm_backward(dy, x.cuda(), w.cuda(), rstd, dres=dres)
    need = bb.if4_rms_norm_backward_workspace_bytes(301, cols)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    dw = torch.empty(cols, device="cuda")
    out = dy if which == "dy" else dres
    bb.if4_rms_norm_backward(dy, x.cuda(), w.cuda(), rstd, dres, out, dw, ws)
    assert torch.equal(out, want) and torch.equal(dw, dww)


@pytest.mark.parametrize("cols", [400, 4096, 33024])
def test_backward_strides_and_no_writes_outside(cols):
    bb = B()
    rows, dtype = 13, torch.bfloat16
    x, r, w = data(rows, cols, dtype, 6)
    rstd = torch.rand(rows, device="cuda") + 0.5
    want, dww = bb.rms_norm_backward(r.cuda(), x.cuda(), w.cuda(), rstd, dres=x.cuda())
    big = [torch.full((rows + 2, cols + 24), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    dy, h, dres, dx = (b[1:rows + 1, 8 * k:8 * k + cols] for k, b in zip((1, 2, 0, 1), big))
    dy.copy_(r), h.copy_(x), dres.copy_(x)
    need = bb.if4_rms_norm_backward_workspace_bytes(rows, cols)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    dw = torch.full((cols + 2,), 7.0, device="cuda")
    bb.if4_rms_norm_backward(dy, h, w.cuda(), rstd, dres, dx, dw[1:-1], ws)
    assert torch.equal(dx, want) and torch.equal(dw[1:-1], dww)
    out = big[3].clone()
    out[1:rows + 1, 8:8 + cols] = 7.0
    assert torch.all(out == 7.0) and float(dw[0]) == 7.0 and float(dw[-1]) == 7.0
    assert torch.all(ws[need:] == 0xA5)


def test_backward_against_differences():
    """d/dt of sum(dy * norm(x + t u) * w) and of its weight, by central differences."""
    x, _, w = data(4, 64, torch.float32, 3)
    g = torch.Generator().manual_seed(8)
    dy = torch.randn((4, 64), generator=g)
    eps = 1e-3

    def f(xx, ww):
        xx, ww = xx.double(), ww.double()
        return (dy.double() * xx / (xx.square().mean(1, keepdim=True) + eps).sqrt() * ww).sum()

    rstd = (1.0 / (x.double().square().mean(1) + eps).sqrt()).float()
    dx, dw = B().rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd.cuda())
    step = 1e-4
    for k in range(12):
        u = torch.randn((4, 64), generator=g, dtype=torch.float64)
        num = (f(x.double() + step * u, w) - f(x.double() - step * u, w)) / (2 * step)
        got = (dx.cpu().double() * u).sum()
        assert abs(num - got) <= 1e-5 * (dx.cpu().double() * u).abs().sum()
        v = torch.randn((64,), generator=g, dtype=torch.float64)
        num = (f(x, w.double() + step * v) - f(x, w.double() - step * v)) / (2 * step)
        got = (dw.cpu().double() * v).sum()
        assert abs(num - got) <= 1e-5 * (dw.cpu().double() * v).abs().sum()


@pytest.mark.parametrize("rows,cols", [(900, 4096), (17, 33024)])
def test_backward_gives_the_same_bits_every_time(rows, cols):
    bb = B()
    x, r, w = data(rows, cols, torch.bfloat16, 2)
    a = [t.cuda() for t in (r, x, w)] + [torch.rand(rows, device="cuda")]
    first = bb.rms_norm_backward(*a)
    for _ in range(3):
        again = bb.rms_norm_backward(*a)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])

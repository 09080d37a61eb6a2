"""The norm and its gradient at widths between the powers of two and between
8192 and 16384 columns, where each block holds other numbers of threads and
units than at the widths of test_gpu_norm.py."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_norm import B, DTYPES, check, check_backward, data, reference

pytestmark = pytest.mark.gpu

# whole and partial last groups of threads; (rows, columns)
WIDTHS = [(7, 96), (150, 544), (31, 2064), (301, 5120), (9, 6144), (5, 8176), (304, 8208), (3, 9216),
          (40, 10240), (11, 12288), (300, 12304), (6, 14336), (310, 16384), (4, 16368)]


@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_forward(rows, cols, dtype, mode):
    rows = min(rows, 160)                  # (the oracle's time) still two rows per block
    x, r, w = data(rows, cols, dtype, rows + 2 * cols)
    check(x, r if rows % 2 else None, w, mode)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(5, 8208), (12, 10240), (3, 16384)])
def test_forward_float32_weight(rows, cols, dtype):
    x, r, w = data(rows, cols, dtype, 5, torch.float32)
    check(x, r, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [8208, 12304, 16384])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_forward_in_place(which, cols, dtype):
    bb = B()
    x, r, w = data(21, cols, dtype, 4)
    xd, rd = x.cuda(), r.cuda()
    codes = torch.empty((21, cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((21, cols // 16), dtype=torch.uint8, device="cuda")
    h = xd if which == "x" else rd
    bb.if4_rms_norm_quantize(xd, rd, w.cuda(), 1e-5, h, None, codes, scales,
                             torch.tensor([0.01], device="cuda"))
    h0, _, y0 = reference(x, r, w, 1e-5)
    q = oracle.quantize(y0, np.float32(0.01))
    assert torch.equal(h.cpu(), h0)
    assert np.array_equal(codes.cpu().numpy(), q["codes"])
    assert np.array_equal(scales.cpu().numpy(), q["scales"])


@pytest.mark.parametrize("dres", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", WIDTHS)
def test_backward(rows, cols, dtype, dres):
    x, r, w = data(rows, cols, dtype, rows + cols)
    g = torch.Generator().manual_seed(1)
    dy = (0.1 * torch.randn((rows, cols), generator=g)).to(dtype)
    check_backward(dy, x, w, r if dres else None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(303, 8208), (9, 12304), (150, 16384)])
def test_backward_float32_weight(rows, cols, dtype):
    x, r, w = data(rows, cols, dtype, 5, torch.float32)
    check_backward(r.clone(), x, w, r)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [96, 2064, 8208, 12304, 16384])
@pytest.mark.parametrize("which", ["dy", "dres"])
def test_backward_in_place(which, cols, dtype):
    bb = B()
    x, r, w = data(310, cols, dtype, 9)
    dy, dres = r.cuda(), (0.5 * r).cuda()
    rstd = torch.rand(310, device="cuda") + 0.5
    want, dww = bb.rms_norm_backward(dy, x.cuda(), w.cuda(), rstd, dres=dres)
    ws = torch.empty(bb.if4_rms_norm_backward_workspace_bytes(310, cols), dtype=torch.uint8,
                     device="cuda")
    dw = torch.empty(cols, device="cuda")
    out = dy if which == "dy" else dres
    bb.if4_rms_norm_backward(dy, x.cuda(), w.cuda(), rstd, dres, out, dw, ws)
    assert torch.equal(out, want) and torch.equal(dw, dww)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [96, 2064, 8208, 12304, 16384])
def test_backward_strides_and_no_writes_outside(cols, dtype):
    bb = B()
    rows, unit = 13, 4 if dtype == torch.float32 else 8          # 16 bytes
    x, r, w = data(rows, cols, dtype, 6)
    rstd = torch.rand(rows, device="cuda") + 0.5
    want, dww = bb.rms_norm_backward(r.cuda(), x.cuda(), w.cuda(), rstd, dres=x.cuda())
    big = [torch.full((rows + 2, cols + 3 * unit), 7.0, dtype=dtype, device="cuda") for _ in range(4)]
    dy, h, dres, dx = (b[1:rows + 1, k * unit:k * unit + cols] for k, b in zip((1, 2, 0, 1), big))
    dy.copy_(r), h.copy_(x), dres.copy_(x)
    need = bb.if4_rms_norm_backward_workspace_bytes(rows, cols)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    dw = torch.full((cols + 2,), 7.0, device="cuda")
    bb.if4_rms_norm_backward(dy, h, w.cuda(), rstd, dres, dx, dw[1:-1], ws)
    assert torch.equal(dx, want) and torch.equal(dw[1:-1], dww)
    out = big[3].clone()
    out[1:rows + 1, unit:unit + cols] = 7.0
    assert torch.all(out == 7.0) and float(dw[0]) == 7.0 and float(dw[-1]) == 7.0
    assert torch.all(ws[need:] == 0xA5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(900, 96), (900, 2064), (500, 8208), (400, 12304), (310, 16384)])
def test_backward_gives_the_same_bits_every_time(rows, cols, dtype):
    bb = B()
    x, r, w = data(rows, cols, dtype, 2)
    a = [t.cuda() for t in (r, x, w)] + [torch.rand(rows, device="cuda")]
    first = bb.rms_norm_backward(*a, dres=a[0])
    for _ in range(3):
        again = bb.rms_norm_backward(*a, dres=a[0])
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])

"""The norm's weight gradient: a sum over all rows of a batch.

Roundings, each at most U = 2^-24 of its value: n = h * rstd; at most one of a
term's own size in a block's sum, which is kept in twice binary32's precision;
a block's sum; the result.  So |dw - exact| <= U |dw| + 3 U sum |dy n|, and a
long sum of equal terms is as good as a short one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def exact(dy, h, rstd, step=2048):
    """dw, and the sum of the magnitudes, in binary64."""
    s = m = 0.0
    for i in range(0, h.shape[0], step):
        p = dy[i:i + step].double() * h[i:i + step].double() * rstd[i:i + step].double().unsqueeze(1)
        s, m = s + p.sum(0), m + p.abs().sum(0)
    return s, m


# (the last of each type is past the widths whose rows a block holds)
@pytest.mark.parametrize("dtype,rows,cols", [
    (torch.bfloat16, 300000, 400), (torch.bfloat16, 40000, 2064), (torch.bfloat16, 20000, 8192),
    (torch.bfloat16, 20000, 12304), (torch.bfloat16, 40000, 16400), (torch.float16, 40000, 2064),
    (torch.float32, 300000, 400), (torch.float32, 40000, 2064), (torch.float32, 40000, 8208)])
def test_many_equal_terms(dtype, rows, cols):
    """Every addition to a binary32 sum of 64 and more terms would round in the
    same direction: terms of 1 + 0.98 * 2^-18."""
    bb = B()
    one = torch.ones((rows, cols), dtype=dtype, device="cuda")
    w = torch.ones(cols, dtype=dtype, device="cuda")
    rstd = torch.full((rows,), 1.0 + 0.98 * 2.0 ** -18, device="cuda")
    dx, dw = bb.rms_norm_backward(one, one, w, rstd)
    want = rows * float(rstd[0].double())
    err = float((dw.double() - want).abs().max()) / want
    assert err <= 4 * U, err / U
    for sign in (-1.0, 1.0):                   # the same, cancelled by a large term
        dy = one.clone()
        dy[::7] = sign * 6.0
        s, m = exact(dy[:, :16], one[:, :16], rstd)
        d = (bb.rms_norm_backward(dy, one, w, rstd)[1][:16].double() - s).abs()
        assert torch.all(d <= U * s.abs() + 3 * U * m * (1 + 2.0 ** -10)), float((d / m).max()) / U


@pytest.mark.parametrize("dtype,rows,cols", [
    (torch.bfloat16, 16384, 4096), (torch.bfloat16, 30001, 1024), (torch.float16, 9000, 5120),
    (torch.bfloat16, 6000, 12304), (torch.bfloat16, 3000, 16400), (torch.float32, 16384, 2048),
    (torch.float32, 4000, 8208)])
def test_no_worse_than_binary64_sums_of_binary32_products(dtype, rows, cols):
    """That form rounds n and dy * n of every row and the sum; the kernel rounds n
    and 296 (or fewer) partial sums instead of the products, which in a sum of
    independent terms is as much.  Over 1024 and more columns the two root mean
    squares differ by a few per cent; a quarter is allowed."""
    bb = B()
    g = torch.Generator(device="cuda").manual_seed(rows)

    def randn(scale=1.0):
        return (scale * torch.randn((rows, cols), generator=g, device="cuda")).to(dtype)

    h, dy = randn(), randn(0.01)
    w = torch.ones(cols, dtype=dtype, device="cuda")
    rstd = (1.0 / h.double().square().mean(1).sqrt()).float()
    dw = bb.rms_norm_backward(dy, h, w, rstd)[1]
    s, m = exact(dy, h, rstd)
    plain = sum((dy[i:i + 2048].float() * (h[i:i + 2048].float() * rstd[i:i + 2048].unsqueeze(1)))
                .double().sum(0) for i in range(0, rows, 2048)).float()
    d = (dw.double() - s).abs()
    assert torch.all(d <= U * s.abs() + 3 * U * m * (1 + 2.0 ** -10))
    ours, theirs = float(d.square().mean().sqrt()), float((plain.double() - s).square().mean().sqrt())
    assert ours <= 1.25 * theirs, ours / theirs


@pytest.mark.parametrize("cols", [64, 400, 4096, 12304, 16400])
def test_overflow_and_nan_stay_in_their_columns(cols):
    """Inf, NaN and sums past binary32's range: what the plain sum gives."""
    bb = B()
    rows = 700
    h = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    dy = h.clone()
    dy[300, 1] = float("inf")
    dy[301, 2] = float("nan")
    dy[:, 3] = 3e38
    dy[302, 4], dy[690, 4] = float("inf"), float("-inf")
    dy[:, 5] = -3e38
    rstd = torch.ones(rows, device="cuda")
    dw = bb.rms_norm_backward(dy, h, torch.ones(cols, device="cuda"), rstd)[1].cpu()
    assert dw[1] == float("inf") and torch.isnan(dw[2]) and dw[3] == float("inf")
    assert torch.isnan(dw[4]) and dw[5] == float("-inf")
    rest = torch.ones(cols, dtype=torch.bool)
    rest[1:6] = False
    assert torch.all(dw[rest] == rows)

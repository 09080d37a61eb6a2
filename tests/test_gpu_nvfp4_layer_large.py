"""The NVFP4 layer's operators on tensors whose byte and element offsets pass
32 bits: samples against the same operator on a small copy of the sampled part
(which the other tests hold to the oracle)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def rows_of(n, total, seed):
    g = torch.Generator().manual_seed(seed)
    r = torch.randint(0, total, (n,), generator=g)
    r[0], r[-1] = 0, total - 1
    return r.cuda()


def fill(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def test_quantize_t():
    bb = B()
    rows, cols = 65536, 36864                     # 2.4e9 elements, 4.8 GB
    x = fill((rows, cols), torch.bfloat16, 1)
    ts = torch.tensor([0.002], device="cuda")
    codes, scales, codes_t, scales_t, _ = bb.quantize_t(x, "nvfp4", ts=ts, with_rows=True)
    c = rows_of(32, cols, 2)
    want = bb.quantize(x[:, c].T.contiguous(), "nvfp4", ts=ts)
    assert torch.equal(codes_t[c], want[0]) and torch.equal(scales_t[c], want[1])
    r = rows_of(32, rows, 3)
    want = bb.quantize(x[r], "nvfp4", ts=ts)
    assert torch.equal(codes[r], want[0]) and torch.equal(scales[r], want[1])
    # the computed scale sees the last element
    x[-1, -1] = 2688.0
    del codes, scales, codes_t, scales_t
    assert float(bb.quantize_t(x, "nvfp4")[2]) == 1.0


@pytest.mark.parametrize("cols", [4096, 36864])
def test_norm_and_gradient(cols):
    bb = B()
    rows = 2_400_000_000 // cols
    x = fill((rows, cols), torch.bfloat16, 1)
    w = fill((cols,), torch.bfloat16, 2)
    ts = torch.tensor([0.002], device="cuda")
    codes, scales, h, rstd = bb.rms_norm_quantize(x, w, ts, residual=x, mode="nvfp4")
    r = rows_of(64, rows, 3)
    want = bb.rms_norm_quantize(x[r], w, ts, residual=x[r], mode="nvfp4")
    for got, k in zip((codes, scales, h, rstd), want):
        assert torch.equal(got[r], k)
    del codes, scales
    dx, dw = bb.rms_norm_backward(x, h, w, rstd, dres=x)
    want, _ = bb.rms_norm_backward(x[r], h[r], w, rstd[r], dres=x[r])
    assert torch.equal(dx[r], want)
    del dx
    s = sum((x[i:i + 4096].double() * h[i:i + 4096].double() *
             rstd[i:i + 4096].double().unsqueeze(1)).sum(0) for i in range(0, rows, 4096))
    assert torch.all((dw.double() - s).abs() <= 1e-4 * s.abs().max())


@pytest.mark.parametrize("M,N,K", [(36000, 65600, 64), (70000, 24, 131072), (40, 70000, 131072)])
def test_linear(M, N, K):
    """A product of 2.4e9 elements; operands of 4.6e9 code bytes, A's and B's."""
    bb = B()
    g = torch.Generator(device="cuda").manual_seed(5)

    def operand(rows):
        codes = torch.randint(0, 256, (rows, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.randint(0x28, 0x48, (rows, K // 16), generator=g, device="cuda",
                               dtype=torch.uint8)
        return codes, scales, torch.full((1,), 2.0 ** -9, device="cuda")

    a, b = operand(M), operand(N)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = bb.linear_nvfp4(a, b, err_flag=err)
    assert int(err) == 0

    def values(t, rows):
        return bb.dequantize(t[0][rows], t[1][rows], t[2], torch.float32).double()

    rm, rn = rows_of(min(M, 24), M, 6), rows_of(min(N, 24), N, 7)
    A, W = values(a, rm), values(b, rn)
    ref, mag = A @ W.T, A.abs() @ W.abs().T
    got = c[rm][:, rn].double()
    assert torch.all((got - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 +
                     mag * (K / 64 + 80) * 2.0 ** -23)

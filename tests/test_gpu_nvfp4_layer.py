"""The NVFP4 layer's operators run together, as a W4A4 linear layer uses them:
a decode step (norm, product), a training step (norm, three products, norm
gradient), both captured, on two streams, and on another device."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def decoded(codes, scales, ts):
    return torch.from_numpy(oracle.dequantize(codes.cpu().numpy(), scales.cpu().numpy(),
                                              np.float32(ts.item()))).double()


def close(c, a, b, scale_steps=16):
    """c against a b^T of decoded operands: the decode rounds q * scale * ts
    twice (2^-24 each), which the product does once for the whole sum."""
    K = a.shape[1]
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    tol = torch.finfo(c.dtype).eps / 2 * ref.abs() * 1.01 + \
        mag * ((K / 64 + 64) * 2.0 ** -23 + scale_steps * 2.0 ** -24)
    d = (c.cpu().double() - ref).abs()
    assert torch.all(d <= tol), float((d / tol).max())


def layer_inputs(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g).bfloat16().cuda()
    r = torch.randn((M, K), generator=g).bfloat16().cuda()
    wn = (1 + 0.1 * torch.randn((K,), generator=g)).bfloat16().cuda()
    w = (0.02 * torch.randn((N, K), generator=g)).bfloat16().cuda()
    dy = (1e-2 * torch.randn((M, N), generator=g)).bfloat16().cuda()
    return x, r, wn, w, dy


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (20, 1000, 1056), (160, 320, 288), (700, 1000, 288)])
def test_decode_step(M, N, K):
    bb = B()
    x, r, wn, w, _ = layer_inputs(M, N, K, M)
    ts = torch.tensor([0.005], device="cuda")
    b = bb.quantize(w, "nvfp4")
    codes, scales, h, rstd = bb.rms_norm_quantize(x, wn, ts, residual=r, mode="nvfp4")
    c = bb.linear_nvfp4((codes, scales, ts), b)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    close(c, decoded(codes, scales, ts), decoded(*b))


@pytest.mark.parametrize("M,N,K", [(96, 160, 224), (256, 384, 512), (320, 288, 1024), (1024, 1280, 1024)])
def test_training_step(M, N, K):
    bb = B()
    x, r, wn, w, dy = layer_inputs(M, N, K, N)
    ts = torch.tensor([0.005], device="cuda")
    codes, scales, h, rstd = bb.rms_norm_quantize(x, wn, ts, residual=r, mode="nvfp4")
    # the forward operand's own values, both ways, and the weight's and the gradient's
    a = bb.dequantize(codes, scales, ts)
    ac, asc, act, ast, ta = bb.quantize_t(a, "nvfp4", with_rows=True)
    wc, ws, wct, wst, tw = bb.quantize_t(w, "nvfp4", with_rows=True)
    yc, ys, yct, yst, ty = bb.quantize_t(dy, "nvfp4", with_rows=True)
    y = bb.linear_nvfp4((ac, asc, ta), (wc, ws, tw))
    da = bb.linear_nvfp4((yc, ys, ty), (wct, wst, tw))
    dw = bb.linear_nvfp4((yct, yst, ty), (act, ast, ta), dtype=torch.float32)
    assert y.shape == (M, N) and da.shape == (M, K) and dw.shape == (N, K)
    close(y, decoded(ac, asc, ta), decoded(wc, ws, tw))
    close(da, decoded(yc, ys, ty), decoded(wct, wst, tw))
    close(dw, decoded(yct, yst, ty), decoded(act, ast, ta))
    dx, dwn = bb.rms_norm_backward(da, h, wn, rstd, dres=da)
    n = h.double() * rstd.double().unsqueeze(1)
    gw = da.double() * wn.double()
    ref = da.double() + rstd.double().unsqueeze(1) * (gw - n * (gw * n).mean(1, keepdim=True))
    assert torch.all((dx.double() - ref).abs() <= 2 ** -8 * ref.abs() + 1e-5 * ref.abs().max())


@pytest.mark.parametrize("M", [3, 200, 3300])
def test_captured_step_equals_the_eager_one(M):
    bb = B()
    N, K = 384, 512
    x, r, wn, w, dy = layer_inputs(M, N, K, 7)
    ts = torch.tensor([0.005], device="cuda")
    b = bb.quantize(w, "nvfp4")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        codes, scales, h, rstd = bb.rms_norm_quantize(x, wn, ts, residual=r, mode="nvfp4",
                                                      err_flag=err)
        c = bb.linear_nvfp4((codes, scales, ts), b, err_flag=err)
        dx, dwn = bb.rms_norm_backward(h, h, wn, rstd, dres=r)
        return h, c, dx, dwn

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for seed in (8, 9):
        x2, r2 = layer_inputs(M, N, K, seed)[:2]
        x.copy_(x2), r.copy_(r2)
        for g, _ in graphs:
            g.replay()
        want = step()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(p, q) for p, q in zip(out, want))
    assert int(err) == 0


def test_two_streams_at_once():
    bb = B()
    N, K = 512, 1024
    ts = torch.tensor([0.005], device="cuda")
    sets = [layer_inputs(M, N, K, M) for M in (5, 300, 2400)]
    bs = [bb.quantize(s[3], "nvfp4") for s in sets]

    def step(s, b):
        codes, scales, h, rstd = bb.rms_norm_quantize(s[0], s[2], ts, residual=s[1], mode="nvfp4")
        c = bb.linear_nvfp4((codes, scales, ts), b)
        return (c, *bb.rms_norm_backward(h, h, s[2], rstd))

    want = [step(s, b) for s, b in zip(sets, bs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(4):
        for st, s, b, o in zip(streams, sets, bs, got):
            with torch.cuda.stream(st):
                o.append(step(s, b))
    torch.cuda.synchronize()
    for o, wnt in zip(got, want):
        assert all(torch.equal(p, q) for r in o for p, q in zip(r, wnt))


@pytest.mark.parametrize("M", [1, 40, 300, 2400])
def test_helpers_on_a_given_stream_share_no_memory_with_the_current_one(M):
    """Work on a side stream that is still waiting, while the current stream
    takes and fills every block that a helper could have returned to it."""
    bb = B()
    N, K = 512, 1024
    x, r, wn, w, dy = layer_inputs(max(M, 304), N, K, M)
    x, r = x[:M], r[:M]
    ts = torch.tensor([0.005], device="cuda")
    b = bb.quantize(w, "nvfp4")

    def step(st):
        codes, scales, h, rstd = bb.rms_norm_quantize(x, wn, ts, residual=r, mode="nvfp4", stream=st)
        c = bb.linear_nvfp4((codes, scales, ts), b, stream=st)
        dx, dwn = bb.rms_norm_backward(h, h, wn, rstd, stream=st)
        return (codes, scales, h, rstd, c, dx, dwn, *bb.quantize_t(dy, "nvfp4", stream=st))

    want = step(None)
    torch.cuda.synchronize()
    sizes = [bb.lib.nvfp4_linear_workspace_bytes(M, N, K),
             bb.lib.if4_rms_norm_backward_workspace_bytes(M, K), 4, 4 * M]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    got = step(side)
    fill = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
            for n in sizes for _ in range(4) if n]
    torch.cuda.synchronize()
    assert all(bool(torch.all(f == 0xA5)) for f in fill)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
def test_tensors_on_another_device_than_the_current_one():
    bb = B()
    ins = [t.to("cuda:1") for t in layer_inputs(200, 256, 512, 3)]
    ts = torch.tensor([0.005], device="cuda:1")
    bc, bs, _, _, tw = bb.quantize_t(ins[3], "nvfp4", with_rows=True)
    codes, scales, h, rstd = bb.rms_norm_quantize(ins[0], ins[2], ts, residual=ins[1], mode="nvfp4")
    c = bb.linear_nvfp4((codes, scales, ts), (bc, bs, tw))
    dx, _ = bb.rms_norm_backward(h, h, ins[2], rstd)
    assert c.device == dx.device == torch.device("cuda:1")
    close(c, decoded(codes, scales, ts), decoded(bc, bs, tw))

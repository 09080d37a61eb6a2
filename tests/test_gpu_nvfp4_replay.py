"""Kernels that start early, run over the same buffers again and again: each
round rewrites the operands that the round before has read."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("M", [1, 2, 48, 300, 1300])      # (1300: CTA pairs in all but the first)
@pytest.mark.parametrize("N,K", [(256, 512), (2048, 2048), (1032, 1056)])
def test_norm_and_product_over_the_same_buffers(M, N, K, captured):
    bb = B()
    g = torch.Generator().manual_seed(M + N)
    rounds = 12
    xs = [torch.randn((M, K), generator=g).bfloat16().cuda() for _ in range(rounds)]
    ws = [(0.02 * torch.randn((N, K), generator=g)).bfloat16().cuda() for _ in range(rounds)]
    wn = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    ts = torch.tensor([0.004], device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    codes, scales = torch.empty((M, K // 2), **u8), torch.empty((M, K // 16), **u8)
    wc, wsc, wts = torch.empty((N, K // 2), **u8), torch.empty((N, K // 16), **u8), \
        torch.tensor([1e-4], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = bb.nvfp4_linear_workspace_bytes(M, N, K)
    work = torch.empty(need, **u8) if need else None
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(rounds)]

    def run():
        # one round: the activations' and the weight's codes rewritten, then read;
        # the next round's norm may start under this round's product
        for x, w, c in zip(xs, ws, outs):
            bb.nvfp4_quantize(w, wc, wsc, wts, bb.TS_GIVEN)
            bb.nvfp4_rms_norm_quantize(x, None, wn, 1e-6, None, None, codes, scales, ts)
            bb.nvfp4_linear(codes, scales, ts, wc, wsc, wts, work, c, err)
            bb.nvfp4_rms_norm_quantize(x[:1], None, wn, 1e-6, None, None, codes[:1], scales[:1], ts)

    want = []
    for x, w in zip(xs, ws):
        q = bb.quantize(w, "nvfp4", ts=wts)
        a = bb.rms_norm_quantize(x, wn, ts, mode="nvfp4")
        torch.cuda.synchronize()
        want.append(bb.linear_nvfp4((a[0], a[1], ts), q))
        torch.cuda.synchronize()
    run()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(4):
        for c in outs:
            c.zero_()
        if captured:
            graph.replay()
        else:
            run()
        torch.cuda.synchronize()
        assert int(err) == 0
        for c, k in zip(outs, want):
            assert torch.equal(c, k)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 256), (64, 512), (512, 2048)])
def test_quantizers_and_dequantizers_over_the_same_buffers(rows, cols, captured):
    """quantize -> dequantize (IF4, IF6, IF3) in place of the input, round after
    round: every kernel reads what the one before it wrote."""
    bb = B()
    g = torch.Generator().manual_seed(rows + cols)
    rounds = 12
    xs = [torch.randn((rows, cols), generator=g).bfloat16().cuda() for _ in range(rounds)]
    ts = torch.tensor([0.002], device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    codes = {b: torch.empty((rows, cols * b // 8), **u8) for b in (4, 6, 3)}
    scales = torch.empty((rows, cols // 16), **u8)
    buf = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda") for _ in range(rounds)]

    def run(sync=lambda: None):
        for x, out in zip(xs, outs):
            src = x
            for bits, dst in ((4, buf), (6, buf), (3, out)):
                if bits == 4:
                    bb.if4_quantize(src, codes[4], scales, ts, bb.TS_COMPUTE)
                    sync()
                    bb.if4_dequantize(codes[4], scales, ts, dst)
                else:
                    bb.ifw_quantize(src, bits, bb.W_ADAPTIVE, codes[bits], scales, ts, bb.TS_COMPUTE)
                    sync()
                    bb.ifw_dequantize(codes[bits], scales, ts, bits, dst)
                sync()
                src = buf

    run(torch.cuda.synchronize)
    want = [o.clone() for o in outs]
    run()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(4):
        for o in outs:
            o.zero_()
        if captured:
            graph.replay()
        else:
            run()
        torch.cuda.synchronize()
        for o, k in zip(outs, want):
            assert torch.equal(o, k)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 256), (16, 4096), (200, 2048), (40, 12288), (5, 33024)])
def test_norm_and_gradient_with_a_weight_just_written(rows, cols, captured):
    """Each round decodes another weight into the same buffer, then the norm and
    its gradient read it."""
    bb = B()
    g = torch.Generator().manual_seed(rows + cols)
    rounds = 8
    x = torch.randn((rows, cols), generator=g).bfloat16().cuda()
    dy = torch.randn((rows, cols), generator=g).bfloat16().cuda()
    ws = [bb.quantize((1 + 0.1 * torch.randn((1, cols), generator=g)).bfloat16().cuda())
          for _ in range(rounds)]
    ts = torch.tensor([0.01], device="cuda")
    w = torch.empty((1, cols), dtype=torch.bfloat16, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    outs = [(torch.empty((rows, cols // 2), **u8), torch.empty((rows, cols // 16), **u8),
             torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"),
             torch.empty(cols, device="cuda")) for _ in range(rounds)]
    rstd = torch.empty(rows, device="cuda")
    work = torch.empty(bb.if4_rms_norm_backward_workspace_bytes(rows, cols), **u8)

    def run(sync=lambda: None):
        for q, (codes, scales, dx, dw) in zip(ws, outs):
            bb.if4_dequantize(*q, w)
            sync()
            bb.if4_rms_norm_quantize(x, None, w[0], 1e-6, None, rstd, codes, scales, ts)
            sync()
            bb.if4_rms_norm_backward(dy, x, w[0], rstd, None, dx, dw, work)
            sync()

    run(torch.cuda.synchronize)
    want = [tuple(t.clone() for t in o) for o in outs]
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        for o, k in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o, k))

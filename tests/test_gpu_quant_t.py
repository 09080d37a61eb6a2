"""GPU tests of the quantizers along the rows: codes, scale bytes and tensor
scale byte-identical to the oracle's quantization of the transposed tensor
(and, for the row form, of the tensor itself)."""
import numpy as np
import pytest
import torch

import oracle
from adaptive_block_scaled_b200 import workloads

pytestmark = pytest.mark.gpu

MODES = {"if4": oracle.MODE_IF4, "nvfp4": oracle.MODE_NVFP4}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def same(codes, scales, ref):
    assert np.array_equal(scales.cpu().numpy(), ref["scales"])
    assert np.array_equal(codes.cpu().numpy(), ref["codes"])


def check(x, mode, with_rows, ts=None, x_host=None):
    bb = B()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bb.quantize_t(x, mode, ts=ts, with_rows=with_rows, err_flag=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    xf = x.float().cpu().numpy()
    t = oracle.tensor_scale(oracle.tensor_amax(xf)) if ts is None else np.float32(ts.item())
    assert np.float32(out[-1].item()) == t
    same(out[-3], out[-2], oracle.quantize(np.ascontiguousarray(xf.T), t, mode=MODES[mode]))
    if with_rows:
        same(out[0], out[1], oracle.quantize(xf, t, mode=MODES[mode]))


def values(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    x[:, torch.rand((cols,), generator=g) < 0.05] *= 20.0
    x[torch.rand((rows,), generator=g) < 0.05] *= 1e-3
    x[torch.rand((rows, cols), generator=g) < 0.1] = 0.0
    return x.to(dtype)


SIZES = [(16, 16), (16, 4096), (4096, 16), (32, 48), (48, 144), (128, 128), (144, 112),
         (256, 1024), (272, 400), (1008, 592), (2048, 1040)]


@pytest.mark.parametrize("with_rows", [False, True])
@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_against_oracle(rows, cols, dtype, mode, with_rows):
    check(values(rows, cols, dtype, rows * 5 + cols).cuda(), mode, with_rows)


@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
def test_full_workload(mode):
    check(workloads.llm_weight(3).cuda(), mode, True)


@pytest.mark.parametrize("mode", ["if4", "nvfp4"])
@pytest.mark.parametrize("ts", [1e-4, 3.0, 1e-9, 2.0 ** -117, 1e30])
def test_given_tensor_scale(mode, ts):
    """Block scales that saturate, are subnormal or underflow to zero."""
    x = values(160, 208, torch.float32, 11).cuda()
    check(x, mode, True, ts=torch.tensor([ts], device="cuda"))


def test_zero_tensor_and_signed_zeros():
    for x in (torch.zeros((64, 32)), -torch.zeros((64, 32))):
        check(x.cuda(), "if4", True)
    x = values(64, 64, torch.bfloat16, 2)
    x[:32] = -0.0
    check(x.cuda(), "nvfp4", True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (32, 16)])
def test_strided_and_16_byte_aligned(dtype, pad, offset):
    rows, cols = 96, 176
    if dtype == torch.float32:
        pad, offset = pad // 2, offset // 2
    big = values(rows, cols + pad + offset, dtype, 7).cuda()
    check(big[:, offset:offset + cols], "if4", True)


def test_equals_the_row_quantizer_of_a_transposed_copy():
    bb = B()
    x = values(512, 384, torch.bfloat16, 21).cuda()
    codes_t, scales_t, ts = bb.quantize_t(x, "if4")
    c, s, t = bb.quantize(x.T.contiguous(), "if4")
    assert torch.equal(c, codes_t) and torch.equal(s, scales_t) and torch.equal(ts, t)


def test_no_writes_outside():
    bb = B()
    rows, cols = 48, 144
    x = values(rows, cols, torch.bfloat16, 4).cuda()
    sizes = [(rows, cols // 2), (rows, cols // 16), (cols, rows // 2), (cols, rows // 16)]
    bufs = [torch.full((16 + a * b + 64,), 0xA5, dtype=torch.uint8, device="cuda") for a, b in sizes]
    views = [f[16:16 + a * b].view(a, b) for f, (a, b) in zip(bufs, sizes)]
    ts = torch.empty(1, device="cuda")
    bb.if4_quantize_t(x, *views, ts)
    for f, (a, b) in zip(bufs, sizes):
        assert torch.all(f[:16] == 0xA5) and torch.all(f[16 + a * b:] == 0xA5)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", DTYPES)
def test_nonfinite_input_is_reported(bad, dtype):
    bb = B()
    x = values(128, 144, dtype, 5)
    x[100, 131] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bb.quantize_t(x.cuda(), "nvfp4", ts=torch.ones(1, device="cuda"), err_flag=err)
    assert int(err) & bb.DEV_NONFINITE


@pytest.mark.parametrize("ts", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** -118, 2.0 ** 118])
def test_invalid_tensor_scale_is_reported(ts):
    bb = B()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bb.quantize_t(values(32, 32, torch.bfloat16, 1).cuda(), "nvfp4",
                  ts=torch.tensor([ts], device="cuda"), err_flag=err)
    assert int(err) & bb.DEV_BAD_SCALE


def test_empty():
    bb = B()
    for rows, cols in ((0, 32), (32, 0)):
        out = bb.quantize_t(torch.empty((rows, cols), device="cuda"), "if4", with_rows=True)
        assert out[2].shape == (cols, rows // 2) and float(out[4]) == 1.0


def test_graph_replayed_on_new_data():
    bb = B()
    x = values(256, 320, torch.bfloat16, 1).cuda()
    u8 = dict(dtype=torch.uint8, device="cuda")
    out = [torch.empty((256, 160), **u8), torch.empty((256, 20), **u8),
           torch.empty((320, 128), **u8), torch.empty((320, 16), **u8)]
    ts = torch.empty(1, device="cuda")
    bb.if4_quantize_t(x, *out, ts)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        bb.if4_quantize_t(x, *out, ts)
    for seed in (2, 3):
        x.copy_(values(256, 320, torch.bfloat16, seed) * seed)
        gr.replay()
        torch.cuda.synchronize()
        xf = x.float().cpu().numpy()
        t = oracle.tensor_scale(oracle.tensor_amax(xf))
        assert np.float32(ts.item()) == t
        same(out[2], out[3], oracle.quantize(np.ascontiguousarray(xf.T), t))
        same(out[0], out[1], oracle.quantize(xf, t))


def test_two_streams_at_once():
    bb = B()
    xs = [values(1024, 512, torch.bfloat16, s).cuda() for s in (1, 2)]
    want = [bb.quantize_t(x, "if4", with_rows=True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(4):
        for st, x, o in zip(streams, xs, got):
            with torch.cuda.stream(st):
                o.append(bb.quantize_t(x, "if4", with_rows=True))
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        for r in o:
            assert all(torch.equal(p, q) for p, q in zip(r, w))

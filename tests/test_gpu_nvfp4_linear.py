"""GPU tests of the NVFP4 x NVFP4 linear against its definition in binary64.

Tolerance: every product q q' s s' has at most 2 + 2 + 4 + 4 significant bits
and is exact in binary32.  The MMA adds 64 of them at a time to the
accumulator: at most K / 64 + 64 roundings of a sum bounded by the sum of the
magnitudes, each at most one step (2^-23, an addition that truncates), then
the product of the two tensor scales and the scaling (2^-24 each), up to eight
partial sums (8 * 2^-24) and half a step of C's type.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def operand(rows, K, g, lo=0x20, hi=0x58):
    codes = torch.randint(0, 256, (rows, K // 2), generator=g).to(torch.uint8)
    scales = torch.randint(lo, hi, (rows, K // 16), generator=g).to(torch.uint8)
    return codes, scales


def decode64(codes, scales):
    lut = torch.tensor(MAGS + tuple(-m for m in MAGS), dtype=torch.float64, device=codes.device)
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1, 16)
    s = scales.view(torch.float8_e4m3fn).double().unsqueeze(-1)
    return (lut[n.long()] * s).reshape(codes.shape[0], -1)


def check(c, a, b, ats, bts):
    K = a[0].shape[1] * 2
    A, W = decode64(*a), decode64(*b)
    ts = float(ats) * float(bts)
    ref, mag = (A @ W.T) * ts, (A.abs() @ W.abs().T) * abs(ts)
    half = torch.finfo(c.dtype).eps / 2
    tol = half * ref.abs() * (1 + 2 ** -8) + mag * ((K / 64 + 64) * 2.0 ** -23 + 10 * 2.0 ** -24)
    if c.dtype == torch.float16:
        tol = tol + 2.0 ** -25                      # half a step of its subnormals
    err = (c.double() - ref).abs()
    assert torch.all(err <= tol), (float((err / tol.clamp(min=1e-300)).max()), int((err > tol).sum()))


def run(a, b, ats, bts, dtype, c=None, ws=None, err=None):
    bb = B()
    M, N, K = a[0].shape[0], b[0].shape[0], a[0].shape[1] * 2
    c = torch.full((M, N), float("nan"), dtype=dtype, device="cuda") if c is None else c
    need = bb.nvfp4_linear_workspace_bytes(M, N, K)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if err is None else err
    bb.nvfp4_linear(*a, ats, *b, bts, ws, c, err)
    return c, err


def cuda(t):
    return tuple(x.cuda() for x in t)


SIZES = [(1, 1, 32), (1, 16, 32), (3, 7, 96), (1, 4096, 4096), (16, 128, 256), (17, 130, 288),
         (33, 300, 4128), (64, 129, 544), (65, 257, 1056), (128, 640, 2048), (5, 1000, 8192),
         (129, 129, 64), (256, 256, 512), (257, 513, 800), (1001, 1555, 4128), (2048, 2304, 1024),
         (300, 128, 512), (1300, 60, 320), (700, 20000, 96), (130, 264, 16384),
         # one and two tokens: whole and partial chunks of K, odd columns, and
         # sizes past the few-token kernel's
         (1, 37, 4128), (2, 129, 1056), (2, 4096, 4096), (1, 8193, 64), (2, 16, 8224),
         # one tile more and fewer than the pairs of SMs
         (256, 128 * 74, 64), (256, 128 * 75, 64), (512, 241, 544),
         # CTA pairs: both tile widths, few columns, last tiles of 1 to 16 columns
         (577, 2177, 64), (650, 1921, 800), (1500, 1700, 512), (4200, 241, 544), (1300, 1937, 256),
         (20000, 1, 64), (20000, 8, 320), (9990, 30, 1056), (10001, 128, 512), (300, 1936, 4128),
         # either side of the two kernels' limits
         (64, 19000, 64), (65, 148 * 128, 128), (128, 148 * 128 + 1, 128), (65, 74 * 128, 96),
         (65, 74 * 128 + 1, 96), (129, 49 * 128, 128), (129, 49 * 128 + 1, 128),
         (40, 8200, 4096), (48, 4100, 14432), (33, 14400, 2080)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_against_binary64(M, N, K, dtype):
    g = torch.Generator().manual_seed(M * 31 + N * 7 + K)
    a, b = cuda(operand(M, K, g)), cuda(operand(N, K, g))
    # keep the largest result inside half's range
    ats = torch.tensor([0.37 / K], device="cuda")
    bts = torch.tensor([0.0213], device="cuda")
    c, err = run(a, b, ats, bts, dtype)
    torch.cuda.synchronize()
    assert int(err) == 0
    check(c, a, b, ats, bts)


def test_full_workload():
    from adaptive_block_scaled_b200 import workloads
    bb = B()
    x, w = workloads.linear_operands(5)
    a, b = bb.quantize(x.cuda(), "nvfp4"), bb.quantize(w.cuda(), "nvfp4")
    c = bb.linear_nvfp4(a, b)
    rows = torch.randint(0, x.shape[0], (64,), generator=torch.Generator().manual_seed(1)).cuda()
    check(c[rows], (a[0][rows], a[1][rows]), b[:2], a[2], b[2])


@pytest.mark.parametrize("M,N", [(5, 200), (200, 384), (700, 1700)])
def test_operands_from_every_nvfp4_quantizer(M, N):
    bb = B()
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, 256), generator=g).bfloat16().cuda()
    w = torch.randn((N, 256), generator=g).bfloat16().cuda()
    for mode in ("nvfp4", "4over6"):
        a, b = bb.quantize(x, mode), bb.quantize(w, mode)
        check(bb.linear_nvfp4(a, b, torch.float32), a[:2], b[:2], a[2], b[2])


@pytest.mark.parametrize("M,N,K", [(2, 130, 512), (4, 130, 512), (140, 300, 768),
                                   (600, 2000, 768)])
def test_all_scales_and_signed_zeros(M, N, K):
    """Every finite E4M3 scale byte, zero included, and every code."""
    g = torch.Generator().manual_seed(K)
    a, b = cuda(operand(M, K, g, 0, 0x7F)), cuda(operand(N, K, g, 0, 0x7F))
    one = torch.ones(1, device="cuda")
    c, err = run(a, b, one, one, torch.float32)
    assert int(err) == 0
    check(c, a, b, one, one)


@pytest.mark.parametrize("M,N", [(2, 256), (8, 256), (256, 256), (640, 1930)])
def test_nan_scale_stays_in_its_row_and_column(M, N):
    g = torch.Generator().manual_seed(9)
    a, b = operand(M, 512, g), operand(N, 512, g)
    a[1][1, 7] = 0x7F
    b[1][11, 31] = 0x7F
    one = torch.ones(1, device="cuda")
    c, err = run(cuda(a), cuda(b), one, one, torch.float32)
    assert int(err) == 0
    want = torch.zeros((M, N), dtype=torch.bool)
    want[1], want[:, 11] = True, True
    assert torch.equal(c.isnan().cpu(), want)


@pytest.mark.parametrize("M,N,K", [(1, 256, 256), (2, 33, 288), (8, 256, 256), (8, 256, 288),
                                   (256, 256, 256), (256, 256, 288),
                                   (640, 1930, 256), (640, 1930, 288)])
@pytest.mark.parametrize("which", [0, 1])
def test_int4_groups_are_reported(M, N, K, which):
    g = torch.Generator().manual_seed(9)
    ops = [operand(M, K, g), operand(N, K, g)]
    ops[which][1][-1, -1] |= 0x80
    one = torch.ones(1, device="cuda")
    _, err = run(cuda(ops[0]), cuda(ops[1]), one, one, torch.bfloat16)
    assert int(err) == B().DEV_BAD_SCALE


@pytest.mark.parametrize("M,N,K", [(1, 201, 512), (3, 200, 512), (130, 200, 512), (130, 201, 512),
                                   (650, 1928, 512), (650, 1921, 512), (9500, 7, 512)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_alignment_and_no_writes_outside(M, N, K, dtype):
    """Scales on a 4-byte boundary only, codes on 16, C on its element's."""
    g = torch.Generator().manual_seed(M + N)
    a, b = operand(M, K, g), operand(N, K, g)

    def shifted(t, by):
        flat = torch.full((t.numel() + 64,), 0x7F, dtype=torch.uint8, device="cuda")
        v = flat[by:by + t.numel()].view(t.shape)
        v.copy_(t)
        return v

    a = (shifted(a[0], 16), shifted(a[1], 4))
    b = (shifted(b[0], 48), shifted(b[1], 12))
    flat = torch.full((M * N + 33,), 7.0, dtype=dtype, device="cuda")
    c = flat[1:1 + M * N].view(M, N)
    one = torch.full((1,), 2.0 ** -10, device="cuda")
    _, err = run(a, b, one, one, dtype, c=c)
    assert int(err) == 0
    check(c, a, b, one, one)
    assert float(flat[0]) == 7.0 and torch.all(flat[1 + M * N:] == 7.0)


@pytest.mark.parametrize("M,N,K", [(1, 100, 96), (2, 100, 512), (9, 100, 96), (9, 100, 512),
                                   (150, 200, 96), (150, 200, 512), (150, 200, 1056),
                                   (600, 2000, 96), (600, 2000, 512), (600, 2000, 1056)])
def test_rows_of_larger_operands(M, N, K):
    """Views that begin at an odd row: scales on a 2-byte boundary."""
    g = torch.Generator().manual_seed(K)
    a, b = cuda(operand(M + 3, K, g)), cuda(operand(N + 1, K, g))
    one = torch.full((1,), 2.0 ** -8, device="cuda")
    a, b = tuple(t[3:] for t in a), tuple(t[1:] for t in b)
    c, err = run(a, b, one, one, torch.float32)
    assert int(err) == 0
    check(c, a, b, one, one)


def test_empty():
    bb = B()
    z = torch.zeros(1, device="cuda")
    for M, N in ((0, 5), (5, 0), (0, 0)):
        g = torch.Generator().manual_seed(1)
        c = bb.linear_nvfp4((*cuda(operand(M, 64, g)), z), (*cuda(operand(N, 64, g)), z))
        assert c.shape == (M, N)


@pytest.mark.parametrize("M", [1, 300, 3300])
def test_two_graphs_replayed_in_turn(M):
    """Two captured calls that share the error word, each replayed on new data."""
    N, K = 272, 1056
    g = torch.Generator().manual_seed(M)
    one = torch.full((1,), 2.0 ** -12, device="cuda")
    sets = [(cuda(operand(M, K, g)), cuda(operand(N, K, g))) for _ in range(2)]
    need = max(1, B().nvfp4_linear_workspace_bytes(M, N, K))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs, graphs = [], []
    for a, b in sets:
        c, _ = run(a, b, one, one, torch.bfloat16, ws=ws, err=err)     # warm-up
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            run(a, b, one, one, torch.bfloat16, c=c, ws=ws, err=err)
        outs.append(c)
        graphs.append(gr)
    for _ in range(2):
        for a, b in sets:
            for t, n in zip((*a, *b), (*operand(M, K, g), *operand(N, K, g))):
                t.copy_(n)
        for c in outs:
            c.fill_(float("nan"))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for (a, b), c in zip(sets, outs):
            check(c, a, b, one, one)
    assert int(err) == 0


@pytest.mark.parametrize("M", [2, 512, 1300])
def test_two_streams_at_once_and_the_same_bits(M):
    N, K = 1024, 2048
    g = torch.Generator().manual_seed(M)
    one = torch.full((1,), 2.0 ** -12, device="cuda")
    sets = [(cuda(operand(M, K, g)), cuda(operand(N, K, g))) for _ in range(2)]
    alone = [run(a, b, one, one, torch.float32)[0].clone() for a, b in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(5):
        for st, (a, b), o in zip(streams, sets, outs):
            with torch.cuda.stream(st):
                o.append(run(a, b, one, one, torch.float32)[0])
    torch.cuda.synchronize()
    for o, want in zip(outs, alone):
        assert all(torch.equal(c, want) for c in o)


def test_an_operand_with_itself():
    bb = B()
    g = torch.Generator().manual_seed(3)
    for rows in (200, 1300):
        a = (*cuda(operand(rows, 320, g)), torch.full((1,), 0.01, device="cuda"))
        check(bb.linear_nvfp4(a, a, torch.float32), a[:2], a[:2], a[2], a[2])

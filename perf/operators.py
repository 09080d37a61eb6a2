"""The NVFP4 linear layer's operators, as cases to be measured.

Four operators make up a linear layer with 4-bit operands, forward and
backward: the NVFP4 x NVFP4 product, the quantizer along the rows (for the two
gradient products, which contract over the other axis), the RMS norm with the
residual's addition and a quantized output, and that norm's gradient.

``run`` computes a case in its plain form (elementary torch operations) or,
where ``own`` is true, with the framework's calls.  Quantized results are
returned as the values they stand for.  The quantizers' arithmetic is fixed
step by step in binary32 (include/if4.h), so the plain form takes the same
roundings, and binary64 where a value sits next to a border: the norm's sum of
squares, and IF4's choice between its two candidates.
"""
import math

import torch


own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# ---------------------------------------------------------------- cases ---

def listed():
    return [
        # one token through a 4096 x 4096 projection: latency and the weight's bytes
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "out": "bf16"},
        # a decode batch
        {"name": "linear_batch", "op": "linear", "M": 48, "N": 8192, "K": 4096, "out": "f16"},
        # odd sizes: K not a multiple of the MMA's 64, N not of 8
        {"name": "linear_ragged", "op": "linear", "M": 1001, "N": 1555, "K": 4128, "out": "bf16"},
        # the framework's own linear workload
        {"name": "linear_prefill", "op": "linear", "M": 8192, "N": 4096, "K": 4096, "out": "bf16"},
        # the framework's small workload, both directions
        {"name": "quant_t_small", "op": "quant_t", "rows": 256, "cols": 1024, "x": "f32",
         "mode": "if4", "both": True},
        # a weight's transposed form, for dX = dY W
        {"name": "quant_t_weight", "op": "quant_t", "rows": 4096, "cols": 4096, "x": "bf16",
         "mode": "nvfp4", "both": False},
        # the framework's activation workload, both directions
        {"name": "quant_t_activation", "op": "quant_t", "rows": 8192, "cols": 8192, "x": "bf16",
         "mode": "if4", "both": True},
        # a decode step's norm in front of a projection, and the projection
        {"name": "norm_linear_decode", "op": "norm_linear", "M": 16, "N": 4096, "K": 4096,
         "x": "bf16"},
        # prefill of the framework's activation size
        {"name": "norm_prefill", "op": "norm", "rows": 8192, "cols": 8192, "x": "bf16",
         "mode": "if4", "residual": True},
        # few ragged rows, no residual
        {"name": "norm_few", "op": "norm", "rows": 37, "cols": 5008, "x": "f16",
         "mode": "nvfp4", "residual": False},
        # the norm's gradient over a training batch
        {"name": "norm_backward", "op": "norm_back", "rows": 16384, "cols": 4096, "x": "bf16",
         "dres": True},
        # one training step of one linear: y, dX and dW, all operands quantized both ways
        {"name": "linear_step", "op": "step", "M": 4096, "N": 4096, "K": 4096},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "quant_t", "norm", "norm_back", "norm_linear", "step"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 8192), _log(rng, 16, 16384), _log(rng, 32, 16384, 32)
            if M * N * K <= 8192 * 4096 * 4096:
                return {"op": op, "M": M, "N": N, "K": K, "out": rng.choice(["bf16", "f16"])}
    if op == "norm_linear":
        return {"op": op, "M": _log(rng, 1, 512), "N": _log(rng, 256, 8192),
                "K": _log(rng, 256, 8192, 32), "x": rng.choice(["bf16", "f16"])}
    if op == "step":
        return {"op": op, "M": _log(rng, 64, 4096, 32), "N": _log(rng, 64, 4096, 32),
                "K": _log(rng, 64, 4096, 32)}
    while True:
        rows, cols = _log(rng, 1, 16384), _log(rng, 16, 16384, 16)
        if op == "quant_t":
            rows = max(16, rows // 16 * 16)
        if rows * cols <= 8192 * 8192:
            break
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quant_t":
        return {"op": op, "rows": rows, "cols": cols, "x": x, "mode": rng.choice(["if4", "nvfp4"]),
                "both": rng.random() < 0.5}
    if op == "norm":
        return {"op": op, "rows": rows, "cols": cols, "x": x, "mode": rng.choice(["if4", "nvfp4"]),
                "residual": rng.random() < 0.7}
    return {"op": op, "rows": rows, "cols": cols, "x": x, "dres": rng.random() < 0.7}


# ------------------------------------------------- formats, plain form ----

def _f(v, like):
    """A binary32 constant on the device: torch divides by a host number
    through its reciprocal, which rounds twice."""
    return torch.full((), v, dtype=torch.float32, device=like.device)


def _e4m3(t):
    """Nearest E4M3 value, saturating at 448."""
    return t.clamp(max=448.0).to(torch.float8_e4m3fn).float()


def _e2m1(a):
    """Nearest E2M1 magnitude of a >= 0, ties to the even code."""
    return (0.5 * ((a > 0.25).float() + (a >= 0.75) + (a > 1.25) + (a >= 1.75))
            + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5.0))


def _tensor_scale(x):
    amax = x.abs().amax().float()
    return torch.where(amax == 0, _f(1.0, x), (amax / _f(2688.0, x)).clamp(min=2.0 ** -117))


def _encode(x, ts, mode):
    """x binary32 [..., 16]: (q, block scale) with the group's values q * scale * ts."""
    s = _e4m3(x.abs().amax(-1, keepdim=True) / _f(6.0, x) / ts)
    eff = s * ts
    inv = torch.where(s == 0, _f(0.0, x), _f(1.0, x) / eff)
    v = x * inv
    fp = torch.copysign(_e2m1(v.abs()), v)
    if mode == "if4":
        k = (v.double() * _f(7.0 / 6.0, x).double()).round().clamp(-7, 7).float()
        it = 6.0 * k / _f(7.0, x)
        e_fp = (v.double() - fp.double()).square_().sum(-1, keepdim=True)
        e_int = (v.double() - it.double()).square_().sum(-1, keepdim=True)
        fp = torch.where(e_int < e_fp, it, fp)
    return torch.where(s == 0, _f(0.0, x), fp), s


def _values(x, ts, mode):
    """Quantized and decoded along the last axis, binary32."""
    g = x.float().reshape(*x.shape[:-1], -1, 16)
    q, s = _encode(g, ts, mode)
    return (q * (s * ts)).reshape(x.shape)


def _nvfp4_operand(x):
    """A made NVFP4 operand of a product: (codes, scales, ts)."""
    ts = _tensor_scale(x).reshape(1)
    q, s = _encode(x.float().reshape(x.shape[0], -1, 16), ts, "nvfp4")
    mags = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=x.device)
    n = torch.searchsorted(mags, q.abs().contiguous()).to(torch.uint8)
    n = (n + 8 * torch.signbit(q).to(torch.uint8)).reshape(x.shape[0], -1)
    codes = n[:, 0::2] + 16 * n[:, 1::2]
    scales = s.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape[0], -1)
    return codes.contiguous(), scales.contiguous(), ts


def _decode(codes, scales):
    """NVFP4 values without the tensor scale, binary32."""
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                       device=codes.device)
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1, 16)
    v = lut[n.long()] * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return v.reshape(codes.shape[0], -1)


# --------------------------------------------------------------- inputs ---

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(g, rows, cols, dt):
    """Activations: N(0, 1), one channel in a hundred twenty times larger."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    loud = torch.rand((cols,), generator=g, device="cuda") < 0.01
    return x.mul_(torch.where(loud, 20.0, 1.0)).to(dt)


def _weight(g, rows, cols):
    """Weights: Student-t with three degrees of freedom, standard deviation 0.02."""
    z = torch.randn((4, rows, cols), generator=g, device="cuda")
    t = z[0] / (z[1:].square().sum(0) / 3.0).sqrt()
    return (t * (0.02 / math.sqrt(3.0))).bfloat16()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = dict(case, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if op == "linear":
        st["a"] = _nvfp4_operand(_acts(g, case["M"], case["K"], torch.bfloat16))
        st["b"] = _nvfp4_operand(_weight(g, case["N"], case["K"]))
    elif op == "quant_t":
        st["x_"] = _acts(g, case["rows"], case["cols"], _DT[case["x"]])
    elif op == "step":
        st["x_"] = _acts(g, case["M"], case["K"], torch.bfloat16)
        st["w"] = _weight(g, case["N"], case["K"])
        st["dy"] = (1e-3 * torch.randn((case["M"], case["N"]), generator=g,
                                       device="cuda")).bfloat16()
    else:
        rows, cols = (case["M"], case["K"]) if op == "norm_linear" else (case["rows"], case["cols"])
        dt = _DT[case["x"]]
        st["x_"] = _acts(g, rows, cols, dt)
        st["w"] = (1.0 + 0.1 * torch.randn((cols,), generator=g, device="cuda")).to(dt)
        if op == "norm_back":
            st["dy"] = (1e-2 * torch.randn((rows, cols), generator=g, device="cuda")).to(dt)
            st["dres"] = ((1e-2 * torch.randn((rows, cols), generator=g, device="cuda")).to(dt)
                          if case["dres"] else None)
            s = st["x_"].double().square().mean(-1) + _f(EPS, st["x_"]).double()
            st["rstd"] = (1.0 / s.sqrt()).float()
        else:
            st["r"] = (torch.randn((rows, cols), generator=g, device="cuda").to(dt)
                       if case.get("residual", True) else None)
            # the running tensor scale of the norm's output, as with delayed scaling
            st["ts"] = torch.full((1,), 32.0 / 2688.0, device="cuda")
            if op == "norm_linear":
                st["b"] = _nvfp4_operand(_weight(g, case["N"], case["K"]))
    return st


# ------------------------------------------------------------------ run ---

def _norm(st, mode):
    """(h, rstd, quantized values) of the norm in its plain form."""
    x, r = st["x_"], st["r"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    s = h.double().square().mean(-1, keepdim=True) + _f(EPS, x).double()
    rstd = (1.0 / s.sqrt()).float()
    y = h.float() * rstd * st["w"].float()
    return h, rstd.squeeze(-1), _values(y, st["ts"], mode)


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    op = st["op"]
    if op == "linear":
        (ac, asc, ats), (bc, bs, bts) = st["a"], st["b"]
        c = (ats * bts) * (_decode(ac, asc) @ _decode(bc, bs).T)
        return c.to(_DT[st["out"]])
    if op == "quant_t":
        x, dt = st["x_"], _DT[st["x"]]
        ts = _tensor_scale(x)
        out = {"t": _values(x.T.contiguous(), ts, st["mode"]).to(dt), "ts": ts.reshape(1)}
        if st["both"]:
            out["rows"] = _values(x, ts, st["mode"]).to(dt)
        return out
    if op == "norm":
        h, rstd, y = _norm(st, st["mode"])
        return {"h": h, "rstd": rstd, "y": y.to(h.dtype)}
    if op == "norm_linear":
        h, _, y = _norm(st, "nvfp4")
        bc, bs, bts = st["b"]
        return {"h": h, "c": (y @ (_decode(bc, bs) * bts).T).bfloat16()}
    if op == "norm_back":
        x, dy, w, rs = st["x_"].float(), st["dy"].float(), st["w"].float(), st["rstd"].unsqueeze(-1)
        n = x * rs
        gy = dy * w
        dx = rs * (gy - n * (gy * n).mean(-1, keepdim=True))
        if st["dres"] is not None:
            dx = dx + st["dres"].float()
        return {"dx": dx.to(st["x_"].dtype), "dw": (dy * n).double().sum(0).float()}
    x, w, dy = st["x_"], st["w"], st["dy"]
    tx, tw, ty = _tensor_scale(x), _tensor_scale(w), _tensor_scale(dy)
    y = _values(x, tx, "nvfp4") @ _values(w, tw, "nvfp4").T
    dx = _values(dy, ty, "nvfp4") @ _values(w.T.contiguous(), tw, "nvfp4").T
    dw = _values(dy.T.contiguous(), ty, "nvfp4") @ _values(x.T.contiguous(), tx, "nvfp4").T
    return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw.bfloat16()}


def _run_own(st):
    from adaptive_block_scaled_b200 import binding as if4
    op, err = st["op"], st["err"]
    if op == "linear":
        return if4.linear_nvfp4(st["a"], st["b"], dtype=_DT[st["out"]], err_flag=err)
    if op == "quant_t":
        x, dt = st["x_"], _DT[st["x"]]
        if st["both"]:
            codes, scales, codes_t, scales_t, ts = if4.quantize_t(x, st["mode"], with_rows=True,
                                                                  err_flag=err)
            return {"t": if4.dequantize(codes_t, scales_t, ts, dt), "ts": ts,
                    "rows": if4.dequantize(codes, scales, ts, dt)}
        codes_t, scales_t, ts = if4.quantize_t(x, st["mode"], err_flag=err)
        return {"t": if4.dequantize(codes_t, scales_t, ts, dt), "ts": ts}
    if op == "norm":
        x = st["x_"]
        codes, scales, h, rstd = if4.rms_norm_quantize(x, st["w"], st["ts"], residual=st["r"],
                                                       eps=EPS, mode=st["mode"], err_flag=err)
        return {"h": h, "rstd": rstd, "y": if4.dequantize(codes, scales, st["ts"], x.dtype)}
    if op == "norm_linear":
        codes, scales, h, _ = if4.rms_norm_quantize(st["x_"], st["w"], st["ts"], residual=st["r"],
                                                    eps=EPS, mode="nvfp4", err_flag=err)
        c = if4.linear_nvfp4((codes, scales, st["ts"]), st["b"], err_flag=err)
        return {"h": h, "c": c}
    if op == "norm_back":
        dx, dw = if4.rms_norm_backward(st["dy"], st["x_"], st["w"], st["rstd"], dres=st["dres"])
        return {"dx": dx, "dw": dw}
    x, w, dy = st["x_"], st["w"], st["dy"]
    xc, xs, xct, xst, tx = if4.quantize_t(x, "nvfp4", with_rows=True, err_flag=err)
    wc, ws, wct, wst, tw = if4.quantize_t(w, "nvfp4", with_rows=True, err_flag=err)
    yc, ys, yct, yst, ty = if4.quantize_t(dy, "nvfp4", with_rows=True, err_flag=err)
    return {"y": if4.linear_nvfp4((xc, xs, tx), (wc, ws, tw), err_flag=err),
            "dx": if4.linear_nvfp4((yc, ys, ty), (wct, wst, tw), err_flag=err),
            "dw": if4.linear_nvfp4((yct, yst, ty), (xct, xst, tx), err_flag=err)}


# ----------------------------------------------------------------- work ---

def work(case):
    op, Q = case["op"], 0.5625                      # bytes of a quantized value and its scale
    if op in ("linear", "norm_linear"):
        M, N, K = case["M"], case["N"], case["K"]
        by = (M + N) * K * Q + 2 * M * N if op == "linear" else N * K * Q + 2 * M * N + 3 * 2 * M * K
        return {"bytes": by, "flops": 2.0 * M * N * K}
    if op == "step":
        M, N, K = case["M"], case["N"], case["K"]
        e = M * K + N * K + M * N
        return {"bytes": 2.0 * e + 2.0 * e, "flops": 6.0 * M * N * K}
    n, b = case["rows"] * case["cols"], _SIZE[case["x"]]
    if op == "quant_t":      # x once; codes, scales and the values they stand for, each way
        return {"bytes": n * (b + (2 if case["both"] else 1) * (Q + b)), "flops": 20.0 * n}
    if op == "norm":         # x and the residual; h if there is one; codes, scales, values
        return {"bytes": n * (b * (3 if case["residual"] else 1) + Q + b), "flops": 20.0 * n}
    return {"bytes": n * b * (4 if case["dres"] else 3) + 8.0 * case["cols"], "flops": 12.0 * n}


# ---------------------------------------------- the definition, 64 bits ---

def _r32(t):
    """One rounding of a binary64 value to binary32, back in binary64."""
    return t.to(torch.float32).to(torch.float64)


def _grid(t, emin, emax, frac, top):
    """Nearest value of a small float (ties to even): exponents emin..emax, frac bits."""
    e = torch.frexp(t.abs())[1].double() - 1.0
    step = torch.exp2(e.clamp(emin, emax) - frac)
    return (torch.round(t / step) * step).clamp(-top, top)


def _exact_values(x, ts, mode):
    """Quantized along the last axis and decoded, from the format's definition."""
    g = x.double().reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    top = g.abs().max(-1, keepdim=True).values
    scale = _grid(_r32(_r32(top / 6) / ts), -6, 8, 3, 448.0)
    eff = _r32(scale * ts)
    v = _r32(g * torch.where(scale > 0, _r32(1 / eff), torch.zeros_like(eff)))
    del g
    q = _grid(v, 0, 2, 1, 6.0)
    if mode == "if4":
        c = float(torch.tensor(7.0 / 6.0, dtype=torch.float32))
        z = _r32(torch.round(v * c).clamp(-7, 7) * 6 / 7)
        gain = ((v - q) ** 2).sum(-1, keepdim=True) - ((v - z) ** 2).sum(-1, keepdim=True)
        q = torch.where(gain > 0, z, q)
    return _r32(q * eff).reshape(x.shape)


def _exact_scale(x):
    top = x.double().abs().max()
    return torch.where(top > 0, _r32(top / 2688).clamp(min=2.0 ** -117), torch.ones_like(top))


def _exact_operand(t):
    codes, scales, ts = t
    b = scales.int() & 127
    e, m = b >> 3, (b & 7).double()
    s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    lo, hi = (codes & 15).int(), (codes >> 4).int()
    n = torch.cat([lo.unsqueeze(-1), hi.unsqueeze(-1)], -1).flatten(1)
    ex, fr = (n >> 1) & 3, (n & 1).double()
    v = torch.where(ex > 0, (1 + fr / 2) * torch.exp2(ex.double() - 1), fr / 2)
    v = torch.where(n >= 8, -v, v)
    return v * s.repeat_interleave(16, 1), ts.double()


def _exact_norm(st, mode):
    x, r = st["x_"], st["r"]
    h = x.double() if r is None else _r32(x.double() + r.double()).to(x.dtype).double()
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    rstd = _r32(torch.rsqrt((h * h).sum(-1) / h.shape[-1] + eps))
    y = _r32(_r32(h * rstd.unsqueeze(-1)) * st["w"].double())
    return h, rstd, _exact_values(y, st["ts"].double(), mode)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "linear":
        (a, ta), (b, tb) = _exact_operand(st["a"]), _exact_operand(st["b"])
        return torch.mm(a, b.T) * (ta * tb)
    if op == "quant_t":
        x = st["x_"]
        ts = _exact_scale(x)
        out = {"t": _exact_values(x.T.contiguous(), ts, case["mode"]), "ts": ts.reshape(1)}
        if case["both"]:
            out["rows"] = _exact_values(x, ts, case["mode"])
        return out
    if op == "norm":
        h, rstd, y = _exact_norm(st, case["mode"])
        return {"h": h, "rstd": rstd, "y": y}
    if op == "norm_linear":
        h, _, y = _exact_norm(st, "nvfp4")
        b, tb = _exact_operand(st["b"])
        return {"h": h, "c": torch.mm(y, b.T) * tb}
    if op == "norm_back":
        h, dy, w = st["x_"].double(), st["dy"].double(), st["w"].double()
        rs = st["rstd"].double().unsqueeze(-1)
        along = (dy * w * h).sum(-1, keepdim=True) / h.shape[-1]
        dx = dy * w * rs - h * along * rs ** 3
        return {"dx": dx if st["dres"] is None else dx + st["dres"].double(),
                "dw": (dy * h * rs).sum(0)}
    x, w, dy = st["x_"], st["w"], st["dy"]
    tx, tw, ty = _exact_scale(x), _exact_scale(w), _exact_scale(dy)

    def rows(t, ts):
        return _exact_values(t, ts, "nvfp4")

    def down(t, ts):
        return _exact_values(t.T.contiguous(), ts, "nvfp4")

    return {"y": torch.mm(rows(x, tx), rows(w, tw).T), "dx": torch.mm(rows(dy, ty), down(w, tw).T),
            "dw": torch.mm(down(dy, ty), down(x, tx).T)}

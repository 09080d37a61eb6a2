"""Which device and stream the binding's calls run on (no GPU needed: the C
calls and the device lookup are replaced)."""
import contextlib
import os
import re
from types import SimpleNamespace

import pytest
import torch

U8, F32, BF16 = torch.uint8, torch.float32, torch.bfloat16


def z(*shape, dtype=U8):
    return torch.zeros(shape, dtype=dtype)


U8_32, U8_4 = z(32, 32), z(32, 4)


def entries(b):
    """name -> a call of that entry point with every tensor on the CPU."""
    x, ts, err = z(32, 64, dtype=BF16), z(1, dtype=F32), z(1, dtype=torch.int32)
    c, s, sync = z(32, 32), z(32, 4), z(64, dtype=torch.int32)
    y, h = z(32, 64, dtype=BF16), z(32, 64, dtype=torch.float16)
    w = z(1 << 20)
    wc, ws, o = z(64, 32), z(64, 4), z(32, 64, dtype=BF16)
    op = (c, s, ts, wc, ws, ts)
    calls = {
        "if4_tensor_amax": lambda **k: b.if4_tensor_amax(x, ts, err, **k),
        "if4_tensor_scale": lambda **k: b.if4_tensor_scale(ts, ts, **k),
        "if4_tensor_amax_rht": lambda **k: b.if4_tensor_amax_rht(x, 5, ts, err, **k),
        "if4_quantize_rht": lambda **k: b.if4_quantize_rht(x, 5, c, s, ts, 0, err, **k),
        "if4_quantize_fused": lambda **k: b.if4_quantize_fused(x, c, s, None, None, ts, sync, err, **k),
        "if4_quantize_fused_rht":
            lambda **k: b.if4_quantize_fused(x, c, s, c, s, ts, sync, err, signs=3, **k),
        "if4_quantize_fused_shared":
            lambda **k: b.if4_quantize_fused_shared(x, c, s, None, None, ts, sync, 2, err, **k),
        "if4_quantize_fused_rht_shared":
            lambda **k: b.if4_quantize_fused_shared(x, c, s, c, s, ts, sync, 2, err, signs=3, **k),
        "if4_quantize_fused_dequant":
            lambda **k: b.if4_quantize_fused_dequant(x, c, s, None, None, ts, sync, y, err, **k),
        "if4_quantize_fused_dequant_shared":
            lambda **k: b.if4_quantize_fused_dequant_shared(x, c, s, c, s, ts, sync, y, 2, err, **k),
        "if4_dequantize": lambda **k: b.if4_dequantize(c, s, ts, y, **k),
        "if4_decode_f16": lambda **k: b.if4_decode_f16(c, s, h, **k),
        "if4_gemm_f16": lambda **k: b.if4_gemm_f16(h, z(64, 64, dtype=torch.float16), ts, ts, o, err, **k),
        "if4_linear": lambda **k: b.if4_linear(*op, w, o, err, **k),
        "if4_linear_fused": lambda **k: b.if4_linear_fused(*op, o, err, **k),
        "if4_linear_noalloc": lambda **k: b.if4_linear_noalloc(*op, o, err, **k),
        "if4_linear_quantized": lambda **k: b.if4_linear_quantized(*op, w, c, s, ts, o, err, **k),
        "nvfp4_linear": lambda **k: b.nvfp4_linear(*op, None, o, err, **k),
        "if4_rms_norm_backward":
            lambda **k: b.if4_rms_norm_backward(y, y, z(64, dtype=F32), z(32, dtype=F32), None, y,
                                                z(64, dtype=F32), w, **k),
    }
    for n in ("if4_quantize", "nvfp4_quantize", "nvint4_quantize", "nvfp4_4over6_quantize"):
        calls[n] = lambda n=n, **k: getattr(b, n)(x, c, s, ts, 0, err, **k)
    for n in ("if4_quantize_t", "nvfp4_quantize_t"):
        calls[n] = lambda n=n, **k: getattr(b, n)(x, c, s, z(64, 16), z(64, 2), ts, 0, err, **k)
    for n in ("if4_rms_norm_quantize", "nvfp4_rms_norm_quantize"):
        calls[n] = lambda n=n, **k: getattr(b, n)(x, None, z(64, dtype=F32), 1e-6, None, None, c, s,
                                                  ts, None, err, **k)
    for bits in (6, 3):
        wide = z(32, 64 * bits // 8)
        calls[f"if{bits}_quantize"] = \
            lambda bits=bits, wide=wide, **k: b.ifw_quantize(x, bits, 0, wide, s, ts, 0, err, **k)
        calls[f"if{bits}_dequantize"] = \
            lambda bits=bits, wide=wide, **k: b.ifw_dequantize(wide, s, ts, bits, y, **k)
    return calls


def binding():
    from adaptive_block_scaled_b200 import build
    build.build()
    from adaptive_block_scaled_b200 import binding as b
    return b


NAMES = sorted(entries(None))


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA"):
        entries(binding())[name]()


@pytest.mark.parametrize("name", NAMES)
def test_calls_run_on_the_tensors_device_and_the_given_stream(name, monkeypatch):
    b = binding()
    seen = []
    monkeypatch.setattr(b, "_device", lambda n, *t: 3)
    monkeypatch.setattr(b, "_call", lambda n, dev, stream, *a: seen.append((n, dev, stream, len(a))))
    side = object()
    entries(b)[name](stream=side)
    assert seen == [(name, 3, side, len(getattr(b.lib, name).argtypes) - 1)]


class Recorded:
    """In place of torch.cuda.stream: whether a stream is current."""
    def __init__(self):
        self.now, self.inside = None, []

    @contextlib.contextmanager
    def stream(self, st):
        self.now, before = st, self.now
        yield
        self.now = before


def helpers(b):
    x, ts = z(32, 64, dtype=BF16), z(1, dtype=F32)
    q = (z(32, 32), z(32, 4), ts)
    w = (z(64, 32), z(64, 4), ts)
    wn, rstd, wide = z(64, dtype=F32), z(32, dtype=F32), z(32, 48)
    return {
        "quantize": lambda st: [b.quantize(x, m, stream=st) for m in ("if4", "nvfp4", "nvint4", "4over6")],
        "quantize given ts": lambda st: b.quantize(x, "if4", ts, None, st),
        "quantize_rht": lambda st: b.quantize_rht(x, 7, stream=st),
        "quantize_w": lambda st: [b.quantize_w(x, n, stream=st) for n in (6, 3)],
        "dequantize_w": lambda st: b.dequantize_w(wide, q[1], ts, 6, stream=st),
        "quantize_fused": lambda st: [b.quantize_fused(x, stream=st),
                                      b.quantize_fused(x, False, stream=st, signs=9)],
        "quantize_fused_dequant": lambda st: b.quantize_fused_dequant(x, stream=st),
        "dequantize": lambda st: b.dequantize(*q, stream=st),
        "decode_f16": lambda st: b.decode_f16(*q[:2], stream=st),
        "linear_nvfp4": lambda st: b.linear_nvfp4(q, w, stream=st),
        "quantize_t": lambda st: b.quantize_t(x, "nvfp4", with_rows=True, stream=st),
        "rms_norm_quantize": lambda st: b.rms_norm_quantize(x, wn, ts, residual=x, stream=st),
        "rms_norm_backward": lambda st: b.rms_norm_backward(x, x, wn, rstd, stream=st),
    }


@pytest.mark.parametrize("name", sorted(helpers(None)))
def test_helpers_allocate_and_launch_on_the_given_stream(name, monkeypatch):
    b, rec = binding(), Recorded()
    side = SimpleNamespace(device_index=-1)          # the device of host tensors
    monkeypatch.setattr(torch.cuda, "stream", rec.stream)
    monkeypatch.setattr(b, "_device", lambda n, *t: 0)
    launches = []
    monkeypatch.setattr(b, "_call", lambda n, dev, stream, *a: launches.append((rec.now, stream)))
    made = []
    for f in ("empty", "empty_like", "empty_strided", "zeros"):
        real = getattr(torch, f)
        monkeypatch.setattr(torch, f, lambda *a, real=real, **k: (made.append(rec.now), real(*a, **k))[1])
    call = helpers(b)[name]
    made.clear()
    call(side)
    # whatever the helper takes from the allocator comes under the stream, and the
    # launch goes to the stream that is current then
    assert launches and all(l == (side, None) for l in launches)
    assert made and all(m is side for m in made)
    launches.clear()
    call(None)
    assert launches and all(l == (None, None) for l in launches)


@pytest.mark.parametrize("name", NAMES)
def test_streams_of_another_device_are_refused(name, monkeypatch):
    b = binding()
    monkeypatch.setattr(b, "_device", lambda n, *t: 3)
    with pytest.raises(ValueError, match="cuda:1.*cuda:3"):
        entries(b)[name](stream=SimpleNamespace(device_index=1, cuda_stream=0))


@pytest.mark.parametrize("name", sorted(helpers(None)))
def test_helpers_refuse_streams_of_another_device(name, monkeypatch):
    b, rec = binding(), Recorded()
    monkeypatch.setattr(torch.cuda, "stream", rec.stream)
    monkeypatch.setattr(b, "_device", lambda n, *t: 0)
    monkeypatch.setattr(b, "_call", lambda *a: None)
    with pytest.raises(ValueError, match="stream belongs to cuda:1"):
        helpers(b)[name](SimpleNamespace(device_index=1))


def test_overlapping_rows_are_refused(monkeypatch):
    """An expanded tensor has the memory of one row: no call may take it for a
    matrix of its shape, whether it reads or writes it."""
    b = binding()
    monkeypatch.setattr(b, "_device", lambda n, *t: 0)
    monkeypatch.setattr(b, "_call", lambda *a: pytest.fail("the call went through"))
    one = z(1, 64, dtype=BF16)
    ts, c, s, sync = z(1, dtype=F32), z(32, 32), z(32, 4), z(64, dtype=torch.int32)
    for x in (one.expand(32, 64), torch.as_strided(z(2048, dtype=BF16), (32, 64), (32, 1))):
        for call in (lambda: b.if4_quantize(x, c, s, ts), lambda: b.if4_tensor_amax(x, ts),
                     lambda: b.if4_quantize_rht(x, 1, c, s, ts), lambda: b.quantize(x),
                     lambda: b.if4_quantize_fused(x, c, s, None, None, ts, sync),
                     lambda: b.if4_dequantize(c, s, ts, x), lambda: b.quantize_w(x, 6),
                     lambda: b.ifw_dequantize(z(32, 48), s, ts, 6, x)):
            with pytest.raises(ValueError, match="overlap"):
                call()
    seen = []
    monkeypatch.setattr(b, "_call", lambda *a: seen.append(a))
    b.if4_quantize(one, z(1, 32), z(1, 4), ts)
    b.if4_quantize(z(64, 128, dtype=BF16)[::2, :64], c, s, ts)        # rows 256 apart
    assert [a[5:8] for a in seen] == [(1, 64, 64), (32, 64, 256)]


def refused(b, monkeypatch, match, *calls):
    monkeypatch.setattr(b, "_device", lambda n, *t: 0)
    monkeypatch.setattr(b, "_call", lambda *a: pytest.fail("the call went through"))
    for call in calls:
        with pytest.raises(ValueError, match=match):
            call()


def test_expanded_workspaces_are_refused(monkeypatch):
    """Its elements count as bytes of memory that it does not have."""
    b = binding()
    ts, err = z(1, dtype=F32), z(1, dtype=torch.int32)
    op, o = (z(32, 32), z(32, 4), ts, z(64, 32), z(64, 4), ts), z(32, 64, dtype=BF16)
    y, rstd, wn = z(32, 64, dtype=BF16), z(32, dtype=F32), z(64, dtype=F32)
    ws = z(1).expand(1 << 20)
    refused(b, monkeypatch, "workspace must be contiguous",
            lambda: b.nvfp4_linear(*op, ws, o, err),
            lambda: b.if4_rms_norm_backward(y, y, wn, rstd, None, y, z(64, dtype=F32), ws),
            lambda: b.if4_linear(*op, ws, o, err),
            lambda: b.if4_linear_quantized(*op, ws, op[0], op[1], ts, o, err))
    sync = z(1, dtype=torch.int32).expand(64)
    x = z(32, 64, dtype=BF16)
    refused(b, monkeypatch, "sync_words must be a contiguous",
            lambda: b.if4_quantize_fused(x, op[0], op[1], None, None, ts, sync),
            lambda: b.if4_quantize_fused_shared(x, op[0], op[1], None, None, ts, sync, 2),
            lambda: b.if4_quantize_fused_dequant(x, op[0], op[1], None, None, ts, sync, y))


def test_words_of_another_type_are_refused(monkeypatch):
    """A float or an int that a kernel reads or writes through its address."""
    b = binding()
    x, c, s, y = z(32, 64, dtype=BF16), z(32, 32), z(32, 4), z(32, 64, dtype=BF16)
    ts, sync, wide = z(1, dtype=F32), z(64, dtype=torch.int32), z(32, 48)
    for bad in (z(1), z(1, dtype=torch.float64), z(0, dtype=F32)):
        refused(b, monkeypatch, "ts|amax",
                lambda: b.if4_tensor_amax(x, bad), lambda: b.if4_tensor_scale(ts, bad),
                lambda: b.if4_tensor_scale(bad, ts), lambda: b.if4_tensor_amax_rht(x, 1, bad),
                lambda: b.if4_quantize_rht(x, 1, c, s, bad), lambda: b.if4_quantize(x, c, s, bad),
                lambda: b.if4_quantize_fused(x, c, s, None, None, bad, sync),
                lambda: b.if4_quantize_fused_dequant(x, c, s, None, None, bad, sync, y),
                lambda: b.if4_dequantize(c, s, bad, y), lambda: b.ifw_dequantize(wide, s, bad, 6, y),
                lambda: b.ifw_quantize(x, 6, 0, wide, s, bad))
    for bad in (z(1), z(1, dtype=torch.int64), z(0, dtype=torch.int32)):
        refused(b, monkeypatch, "err_flag",
                lambda: b.if4_tensor_amax(x, ts, bad), lambda: b.if4_quantize(x, c, s, ts, 0, bad),
                lambda: b.if4_quantize_rht(x, 1, c, s, ts, 0, bad),
                lambda: b.if4_quantize_fused(x, c, s, None, None, ts, sync, bad),
                lambda: b.ifw_quantize(x, 6, 0, wide, s, ts, 0, bad),
                lambda: b.if4_linear_fused(c, s, ts, c, s, ts, z(32, 32, dtype=BF16), bad))


def test_a_product_without_an_error_word_says_so_and_fills_none(monkeypatch):
    b = binding()
    assert "errors are lost" in " ".join(b.linear_nvfp4.__doc__.split())
    ts = z(1, dtype=F32)
    monkeypatch.setattr(b, "_device", lambda n, *t: 0)
    seen = []
    monkeypatch.setattr(b, "_call", lambda *a: seen.append(a))
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: pytest.fail("a kernel for a word nobody reads"))
    b.linear_nvfp4((U8_32, U8_4, ts), (U8_32, U8_4, ts))
    assert seen[0][0] == "nvfp4_linear" and seen[0][-1]          # an address, never NULL


def test_the_readme_reads_its_error_word():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "README.md")).read()
    for block in re.findall(r"```python\n(.*?)```", text, flags=re.S):
        calls = re.findall(r"linear_nvfp4\((?:[^()]|\([^()]*\))*\)", block)
        assert all("err_flag=" in c for c in calls)
        assert not calls or "err.item()" in block

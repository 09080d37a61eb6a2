"""Helpers that are given a stream, and tensors on another device than the
current one, through every quantizer, dequantizer and width."""
import pytest
import torch

pytestmark = pytest.mark.gpu

R, C = 256, 1024


def B():
    from adaptive_block_scaled_b200 import binding
    return binding


def calls(device="cuda"):
    """name -> helper(stream) on fixed inputs."""
    bb = B()
    g = torch.Generator().manual_seed(4)
    x = torch.randn((R, C), generator=g).bfloat16().to(device)
    q = bb.quantize(x)
    w = {n: bb.quantize_w(x, n) for n in (6, 3)}
    torch.cuda.synchronize(device)
    return {
        "quantize if4": lambda st: bb.quantize(x, stream=st),
        "quantize nvfp4 given": lambda st: bb.quantize(x, "nvfp4", q[2], stream=st),
        "quantize nvint4": lambda st: bb.quantize(x, "nvint4", stream=st),
        "quantize 4over6": lambda st: bb.quantize(x, "4over6", stream=st),
        "quantize_rht": lambda st: bb.quantize_rht(x, 0x1234, stream=st),
        "quantize_fused": lambda st: bb.quantize_fused(x, stream=st),
        "quantize_fused rht": lambda st: bb.quantize_fused(x, False, stream=st, signs=5),
        "quantize_fused_dequant": lambda st: bb.quantize_fused_dequant(x, stream=st),
        "dequantize": lambda st: (bb.dequantize(*q, stream=st),),
        "decode_f16": lambda st: (bb.decode_f16(*q[:2], stream=st),),
        "quantize_w 6": lambda st: bb.quantize_w(x, 6, stream=st),
        "quantize_w 3": lambda st: bb.quantize_w(x, 3, stream=st),
        "dequantize_w 6": lambda st: (bb.dequantize_w(*w[6], 6, stream=st),),
        "dequantize_w 3": lambda st: (bb.dequantize_w(*w[3], 3, torch.float32, stream=st),),
    }


NAMES = ["quantize if4", "quantize nvfp4 given", "quantize nvint4", "quantize 4over6", "quantize_rht",
         "quantize_fused", "quantize_fused rht", "quantize_fused_dequant", "dequantize", "decode_f16",
         "quantize_w 6", "quantize_w 3", "dequantize_w 6", "dequantize_w 3"]


@pytest.mark.parametrize("name", NAMES)
def test_results_of_a_given_stream_are_not_handed_out_on_the_current_one(name):
    """The results are dropped while the side stream has not begun to write them;
    the current stream then takes blocks of their sizes and fills them."""
    run = calls()[name]
    want = run(None)
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want] + [256, 512]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(30_000_000)
    got = run(side)
    del got
    fill = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool(torch.all(f == 0xA5)) for f in fill)
    got = run(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second device")
@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_device_than_the_current_one(name):
    want = calls()[name](None)
    got = calls("cuda:1")[name](None)
    assert all(p.device == torch.device("cuda:1") and torch.equal(p.cpu(), q.cpu())
               for p, q in zip(got, want))

"""Source rules of kernels that may start before their predecessor has finished.

Launched programmatically, such a kernel waits (griddepcontrol.wait) before it
reads anything.  A load keeps its place behind that wait only if the compiler
may not move it (volatile) and the hardware may not take its data for constant
(no ld.global.nc): an earlier kernel of the stream may have just written it.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "adaptive_block_scaled_b200", "csrc")
FILES = ["nvfp4_linear.cu", "if4_norm.cu", "if4_quant_t.cu", "if4_quant.cu", "ifw_quant.cu",
         "if4_linear.cu", "if4_device.cuh", "if4_load.cuh", "if4_encode.cuh", "if4_decode.cuh"]


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", FILES)
def test_no_load_that_takes_memory_for_constant(name):
    text = code(name)
    assert "ld.global.nc" not in text and "__ldg" not in text


@pytest.mark.parametrize("name", FILES + ["if4_tc.cuh", "nvfp4_scales.cuh"])
def test_every_load_instruction_keeps_its_place(name):
    text = code(name)
    for m in re.finditer(r'asm\s*(volatile)?\s*\(\s*"((?:[^"\\]|\\.)*)"', text):
        if "ld.global" in m.group(2) or "ld.shared" in m.group(2):
            assert m.group(1), m.group(2)

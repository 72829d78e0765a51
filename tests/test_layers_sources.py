"""What the sources of the kernels that update in place, or are launched early, may not contain. Runs without a GPU."""

import re

from test_llm_sources import kernels, statements


def test_operands_are_loaded_coherently():
    """A non-coherent load is for memory that nothing writes while the kernel runs. Outputs may take their inputs' places, and
    a kernel that is launched early runs beside the one whose results it reads, so their operands take the coherent path. (The
    products' epilogue reads a bias, which no output may overlap.)"""
    loads = {name for name, s in statements() if "ld.global" in s}
    assert {"rows.h", "clip.cu", "reduce.cu"} <= loads
    for name, s in statements():
        assert "ld.global.nc" not in s or name == "tc_ptx.h", (name, s)


def test_early_kernels_wait_before_anything_else():
    """What a kernel that is launched early reads may still be written until its wait has ended."""
    text = {}
    for name, kernel, body in kernels():
        text[kernel] = body
    for kernel in ("k_expert_dispatch", "k_clip_scale", "k_layernorm_dweight"):
        body = text[kernel][text[kernel].index("{\n") + 2:]
        before = body[:body.index("await_launches();")]
        assert not re.search(r"[\[\]]|->|\(", re.sub(r"__shared__[^;]*;", "", before)), kernel

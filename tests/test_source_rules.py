"""Rules of the kernels' sources that no run can show."""
import re

from quantized_matmul_speculative_gb300 import build


def test_dependent_kernels_do_not_use_the_read_only_path():
    """A kernel that starts while its predecessor may still write (griddepcontrol.wait) reads what that one writes with
    loads that stay where they are: no __ldg, no ld.global.nc and no asm load that the compiler may move.  Weights, which
    no such predecessor writes, are loaded by ld_stream (qmm_device.cuh)."""
    found = []
    sources = sorted([*build.CSRC.glob("*.cu"), *build.CSRC.glob("*.cuh")])
    assert any("griddep_wait" in p.read_text() for p in sources)
    for p in sources:
        text = re.sub(r"//[^\n]*", "", p.read_text())
        if p.name == "qmm_device.cuh":
            text = re.sub(r"void ld_stream<\d>\(.*?\n}", "", text, flags=re.S)
        elif "griddep_wait" not in text and "stage_x" not in text:
            continue  # a kernel that its launch orders
        found += [(p.name, m.group(0)) for m in re.finditer(r"__ldg|ld\.global\.nc|asm\(\s*\"ld\.global", text)]
    assert not found, found

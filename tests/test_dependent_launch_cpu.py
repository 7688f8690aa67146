"""Kernels launched while the kernel ahead of them still runs must read what it writes by loads
that the wait orders (csrc/pdl.cuh): ld.global.nc, __ldg and const __restrict__ pointers promise
that nobody writes the memory while the kernel lives.  A source check, without a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_dequant_matmul_gb300", "csrc")
NON_COHERENT = re.compile(r"__ldg\s*\(|ld\.global\.nc|\bldg_stream\w*\s*\(|const\s+[\w:]+\s*(?:<[^<>]*>)?\s*\*\s*(?:const\s+)?__restrict__")


def code(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["mx_quant.cu", "mx_mm.cu", "moe_route.cu", "elem.cuh", "pdl.cuh"])
def test_no_non_coherent_loads(name):
    assert not NON_COHERENT.findall(code(name))


# (file, kernel, where its dependent reads begin; mxfp4_mv's weights are read ahead of the wait,
# and with launch overlap the caller promises that nothing ahead writes them)
@pytest.mark.parametrize("name,kernel,after", [("moe_tc.cu", "k_moe_split", ""), ("moe_tc.cu", "k_moe_tc", ""),
                                               ("moe.cu", "k_moe_combine", ""), ("mv_tc.cu", "k_mv_tc", "griddepcontrol.wait")])
def test_kernels_of_the_routed_layer_and_the_overlapped_matvec(name, kernel, after):
    text = code(name)
    start = re.search(r"\b%s\((?=const)" % kernel, text).start()
    depth, end = 0, text.index("{", text.index(")", start))
    for end in range(end, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            break
    body = text[start:end]
    assert "griddepcontrol.wait" in body
    assert not NON_COHERENT.findall(body[body.index(after):])


def test_the_check_sees_each_form():
    for text in ("v = __ldg(p);", "ld.global.nc.L1::no_allocate.v4.u32", "ldg_stream32(p, v)", "const T* __restrict__ x",
                 "const Pack<T, N>* __restrict__ o"):
        assert NON_COHERENT.search(text), text
    assert not NON_COHERENT.search("ld_dep(p); ld_dep_stream(p); const A a, T* __restrict__ y; ld.global.v4.u32")

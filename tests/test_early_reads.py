"""What a kernel may read before the grid that it depends on has completed:
laid-out weights, which no kernel that lets dependents start early writes, and
nothing else (include/qmm.h, stream order)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gguf_block_quantized_qmatmul_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_router_is_read_after_the_wait():
    """It is a tensor of floats, which the call before may make."""
    body = source("qmm_moe_layer.cu").split("moe_router_kernel(", 1)[1]
    before = body.split("grid_dep_wait();", 1)[0]
    assert "router_load8(" not in before


def test_what_an_earlier_grid_may_write_is_not_read_as_constant():
    """ld.global.nc (__ldg) is for data that nobody writes while the kernel runs, and a kernel that was started early runs
    while the grid before it writes activations, scales and sums: only what is in the laid-out weights (sw: their scales) goes that way."""
    for name in ("qmm_q8c_rows.cu", "qmm_q8c_quant.cu", "qmm_q8c_gemm.cu", "qmm_moe_layer.cu", "qmm_moe_layer.cuh", "qmm_moe_route.cuh", "qmm_norm.cuh"):
        for use in re.findall(r"__ldg\(([^;]*);", source(name)):
            assert re.match(r"sw \+ n|reinterpret_cast<const uint32_t\*>\(w\.data \+ w\.norm_off\)", use), (name, use)

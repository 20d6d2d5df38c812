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

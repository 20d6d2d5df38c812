"""What the sources of the 4-bit and mixture-of-experts kernels must not hold,
because no run of one compiler's code can show that it is sound."""
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gguf_block_quantized_qmatmul_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))))
def test_no_shuffle_mask_from_the_lanes_that_happen_to_be_together(name):
    """__activemask() promises nothing about lanes that left a loop at different trips: a shuffle by its mask may
    read a lane that does not take part."""
    with open(os.path.join(CSRC, name)) as f:
        assert "__activemask" not in f.read()

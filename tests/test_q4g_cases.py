"""4-bit group-scale products and mixture-of-experts operators where sizes,
magnitudes and handles are at their edges.  Tolerances are those of
test_q4g.py unless a test says otherwise."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    import gguf_block_quantized_qmatmul_gb300 as q
    return q


def rng(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ routing


@pytest.mark.parametrize("E,k", [(9, 2), (256, 8), (300, 5), (512, 32)])
@pytest.mark.parametrize("T", [33, 40, 41, 500, 1217, 4863, 10007, 33333])
def test_route_order_of_uneven_tiles(q, T, E, k):
    """Numbers of tiles that two half warps, 16 warps and the order's blocks do not divide evenly."""
    r = q.moe_route(torch.randn((T, E), generator=rng(T + E)).cuda(), k)
    flat = r.ids.cpu().numpy().reshape(-1)
    order = np.argsort(flat, kind="stable")
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.offsets.cpu().numpy(), np.searchsorted(flat[order], np.arange(E + 1)))

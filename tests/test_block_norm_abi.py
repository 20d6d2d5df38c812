"""Which places qmm_block_norm takes for its results (no GPU needed: calls that
pass the checks end at an injected launch failure, before any CUDA call)."""
import ctypes

import pytest

pytest.importorskip("torch")

SHAPE, CUDA = 2, 6
Y, R, OTHER = 0x100000, 0x200000, 0x300000  # addresses that are never read


@pytest.fixture(scope="module")
def call():
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    import gguf_block_quantized_qmatmul_gb300 as q
    from gguf_block_quantized_qmatmul_gb300 import q8c

    def f(T=2, K=64, **k):
        a = dict(y=Y, residual=R, weight=0x10000, h=0x400000, ldy=64, ldr=64, ldg=64, ldro=64, ldh=64)
        a.update(k)
        n = q8c._Norm(**a)
        q.test_inject("launch_failure", 1)
        try:
            return q8c._lib().qmm_block_norm(ctypes.addressof(n), T, K, 0)
        finally:
            q.test_inject("off")
    return f


@pytest.mark.parametrize("out,ld", [("residual_out", "ldro"), ("h", "ldh")])
@pytest.mark.parametrize("at,ld_in", [(Y, "ldy"), (R, "ldr")])
def test_in_place_rows_are_the_same_distance_apart(call, out, ld, at, ld_in):
    """At another distance a row's result would lie on another row's input, which may not have been read yet."""
    assert call(**{out: at}) == CUDA and call(**{out: at, ld: 80, ld_in: 80}) == CUDA
    assert call(**{out: at, ld: 80}) == SHAPE and call(**{out: at, ld_in: 80}) == SHAPE
    assert call(**{out: at, ld: 80, "T": 1}) == CUDA and call(**{out: OTHER, ld: 80}) == CUDA
    # y and residual are one tensor: a result in its place follows both distances
    assert call(**{out: Y, "residual": Y}) == CUDA and call(**{out: Y, "residual": Y, "ldr": 80}) == SHAPE


def test_codes_lie_in_no_other_tensors_place(call):
    ok = dict(h=0, codes=0x500000, scales=0x600000)
    assert call(**ok) == CUDA and call(**{**ok, "residual_out": R}) == CUDA
    assert call(**{**ok, "residual_out": OTHER, "codes": OTHER}) == SHAPE
    for at in (Y, R):
        assert call(**{**ok, "codes": at}) == SHAPE

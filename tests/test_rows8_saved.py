"""Quantized rows are kept like any tensors, whoever made them."""
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


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 100), (16, 4096), (300, 2000), (0, 64)])
@pytest.mark.parametrize("given", [False, True])
def test_a_norms_rows_can_be_saved(q, tmp_path, T, K, dt, given):
    """With r' beside them: no storage is seen as two types."""
    x = torch.randn((T, K), device="cuda").to(dt)
    r, rows = q.block_norm(x, torch.ones(K, device="cuda", dtype=dt), residual=x, quantize=True, residual_out=torch.empty_like(x) if given else None)
    assert r.data_ptr() == 0 or len({t.untyped_storage().data_ptr() for t in (r, *rows)}) == 3
    ref = q.block_norm(x, torch.ones(K, device="cuda", dtype=dt), residual=x)
    assert torch.equal(r, ref[0]) and rows.codes.shape == (T, K) and rows.scales.shape == (T,) and rows.codes.stride() in ((-(-K // 16) * 16, 1), (K, 1))
    for kept in ({"rows": tuple(rows)}, {"r": r, "codes": rows.codes, "scales": rows.scales}, {"codes": rows.codes}):
        torch.save(kept, tmp_path / "k.pt")
        back = torch.load(tmp_path / "k.pt", weights_only=True)
        if "rows" in kept:
            assert all(torch.equal(a, b) for a, b in zip(back["rows"], rows))
            if T:
                w = q.q8c_pack(rows.codes.clone(), torch.ones(T, device="cuda"))
                assert torch.equal(q.q8c_matmul(w, q.Rows8(*back["rows"])), q.q8c_matmul(w, rows))
        else:
            assert all(torch.equal(back[k], kept[k]) for k in kept)


def test_a_quantizers_rows_and_float_results_too(q, tmp_path):
    x = torch.randn((5, 100), device="cuda")
    rows = q.q8c_quantize(x)
    r, h = q.block_norm(x, x[0], residual=x)
    torch.save({"rows": tuple(rows), "r": r, "h": h}, tmp_path / "k.pt")
    back = torch.load(tmp_path / "k.pt", weights_only=True)
    assert all(torch.equal(a, b) for a, b in zip(back["rows"], rows)) and torch.equal(back["r"], r) and torch.equal(back["h"], h)

"""Results of 8-bit products in places that are aligned as their elements are
and no further, between guard values: the same bits as anywhere else, and
nothing around them is touched."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    import gguf_block_quantized_qmatmul_gb300 as q
    return q


# the row kernel; single blocks, K slices; pairs of blocks, K slices, tiles of 128 K; N in whole fours and not
SIZES = [(1, 64, 128), (3, 1300, 576), (5, 64, 128), (40, 1300, 576), (40, 1302, 576), (33, 400, 8192), (300, 2052, 1024),
         (200, 9000, 192), (300, 1300, 8192), (1024, 14336, 128), (1024, 14333, 128), (6, 4, 64), (7, 5, 64)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_results_on_no_boundary(q, M, N, K, dt):
    g = torch.Generator().manual_seed(M + N)
    codes = torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda()
    w = q.q8c_pack(codes, (0.001 + torch.rand(N, generator=g)).cuda())
    x = torch.randn((M, K), generator=g).to(DT[dt]).cuda()
    ref = q.q8c_matmul(w, x)
    for shift in (1, 2, 3, 4, 8):
        buf = torch.full((M * N + 32,), 7.0, dtype=DT[dt], device="cuda")
        out = buf[shift:shift + M * N].view(M, N)
        assert q.q8c_matmul(w, x, out=out).data_ptr() == out.data_ptr()
        assert torch.equal(out, ref)
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + M * N:] == 7).all())
    assert q.last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(3, 500, 9001), (40, 1300, 576), (64, 4096, 4096), (300, 2052, 1024), (1024, 9000, 192)])
def test_workspace_on_any_16_byte_boundary(q, M, N, K):
    g = torch.Generator().manual_seed(M)
    w = q.q8c_pack(torch.randint(-127, 128, (N, K), generator=g).to(torch.int8).cuda(), torch.rand(N, generator=g).cuda())
    x = torch.randn((M, K), generator=g).half().cuda()
    ref, n = q.q8c_matmul(w, x), q.q8c_matmul_workspace(w, M)
    assert n > 0
    for shift in (16, 48):
        buf = torch.full((n + 80,), 0xA5, dtype=torch.uint8, device="cuda")
        assert torch.equal(q.q8c_matmul(w, x, workspace=buf[shift:shift + n]), ref)
        assert bool((buf[:shift] == 0xA5).all()) and bool((buf[shift + n:] == 0xA5).all())
    assert q.last_device_error() == 0

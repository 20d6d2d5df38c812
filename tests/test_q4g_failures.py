"""Failure paths of the 4-bit and mixture-of-experts calls, exercised without
faulting the GPU (as test_gpu_failures.py does for the block formats): an
injected launch failure makes no CUDA call; an injected stall, one block's
weight copies ending early, runs every other role of that block and of its
pair into its bounded wait, and with the limit lowered to 2^22 SM clocks (2
ms) the call ends, reports QMM_ERR_TIMEOUT, and the next one is right."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

QMM_ERR_CUDA, QMM_ERR_TIMEOUT = 6, 7
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    import gguf_block_quantized_qmatmul_gb300 as q
    return q


def weights(q, E, N, K, gate_up=False):
    g = torch.Generator().manual_seed(E + N + K)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scales = (0.01 * (0.5 + torch.rand((E, N, K // 64), generator=g))).half()
    return q.q4g_pack(codes.cuda(), scales.cuda(), gate_up=gate_up)


def call(q, op, dt, M):
    """A call of the GEMM, and what it makes."""
    g = torch.Generator().manual_seed(M)
    if op == "matmul":
        w, x = weights(q, 1, 4100, 4096), torch.randn((M, 4096), generator=g).to(DT[dt]).cuda()
        return lambda **kw: q.q4g_matmul(w, x, **kw)
    route = q.moe_route(torch.randn((M, 4), generator=g).cuda(), 2)
    if op == "gate_up":
        w, x = weights(q, 4, 1040, 1024, True), torch.randn((M, 1024), generator=g).to(DT[dt]).cuda()
        return lambda **kw: q.moe_gate_up(w, x, route, **kw)
    w, h = weights(q, 4, 1040, 1024), torch.randn((M, 2, 1024), generator=g).to(DT[dt]).cuda()
    return lambda **kw: q.moe_down(w, h, route, **kw)


# pairs of blocks with one weight piece and with two, single blocks (f32); dense and by expert
CALLS = [("matmul", "bf16", 300), ("matmul", "f16", 1000), ("matmul", "f32", 100), ("gate_up", "f16", 500), ("gate_up", "bf16", 500),
         ("gate_up", "f32", 200), ("down", "f16", 500), ("down", "f32", 200)]


@pytest.mark.parametrize("tiles", [0, 1, 5])
@pytest.mark.parametrize("op,dt,M", CALLS)
def test_injected_stall_times_out_and_recovers(q, op, dt, M, tiles):
    run = call(q, op, dt, M)
    ref = run()
    torch.cuda.synchronize()
    assert q.last_device_error() == 0
    q.test_set_wait_limit(22)
    try:
        q.test_inject("stall", 1, tiles)
        run()
        torch.cuda.synchronize()  # the call ends: every wait is bounded
        assert q.last_device_error() == QMM_ERR_TIMEOUT
    finally:
        q.test_inject("off")
        q.test_set_wait_limit(0)
    assert torch.equal(run(), ref)
    assert q.last_device_error() == 0


@pytest.mark.parametrize("op,dt,M", [("matmul", "bf16", 2), ("gate_up", "f32", 1), ("down", "f16", 3)] + CALLS)
def test_injected_launch_failure_touches_nothing(q, op, dt, M):
    run = call(q, op, dt, M)
    ref = run()
    out = torch.full_like(ref, 7.0)
    q.test_inject("launch_failure", 1)
    try:
        with pytest.raises(q.QmmError) as e:
            run(out=out)
        assert e.value.status == QMM_ERR_CUDA
    finally:
        q.test_inject("off")
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    assert torch.equal(run(out=out), ref)


def test_injected_launch_failure_of_a_routing(q):
    logits = torch.randn((5, 16), generator=torch.Generator().manual_seed(1)).cuda()
    q.test_inject("launch_failure", 1)
    try:
        with pytest.raises(q.QmmError) as e:
            q.moe_route(logits, 3)
        assert e.value.status == QMM_ERR_CUDA
    finally:
        q.test_inject("off")
    assert torch.equal(q.moe_route(logits, 3).ids.long(), logits.topk(3).indices)

"""A layer whose inputs the library's own calls make just before it, in the same
stream: kernels that let the next ones start early."""
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


def layer_weights(q, E, N, K, F, dt):
    g = torch.Generator().manual_seed(1)
    def pack(rows, cols, gate_up):  # noqa: E306
        codes = torch.randint(0, 256, (E, rows, cols // 2), generator=g).to(torch.uint8).cuda()
        return q.q4g_pack(codes, (0.01 + 0.01 * torch.rand((E, rows, cols // 32), generator=g)).to(dt).cuda(), gate_up=gate_up)
    return pack(2 * F, K, True), pack(N, F, False)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,E,K,T", [(64, 64, 2048, 1), (300, 16, 4096, 5), (4096, 64, 1024, 9), (20000, 64, 576, 3)])
def test_a_router_and_tokens_that_a_norm_has_just_made(q, rows, E, K, T, dt):
    """The norm's last rows are the router, its first ones the tokens."""
    up, down = layer_weights(q, E, 96, K, 64, torch.bfloat16 if dt == torch.bfloat16 else torch.float16)
    g = torch.Generator().manual_seed(2)
    y, residual = (torch.randn((rows, K), generator=g).to(dt).cuda() for _ in range(2))
    weight = torch.ones(K, device="cuda", dtype=dt)
    made, h = q.block_norm(y, weight, residual=residual, scale=0.1)
    torch.cuda.synchronize()
    ref, route = q.moe_layer(up, down, made[-E:], h[:T], 4, route=True)
    torch.cuda.synchronize()

    def run():
        q.block_norm(y, weight, residual=residual, scale=0.1, residual_out=made, out=h)
        return q.moe_layer(up, down, made[-E:], h[:T], 4, route=True)
    for _ in range(20):
        made.fill_(float("nan"))
        h.fill_(float("nan"))
        z, r = run()
        assert torch.equal(z, ref) and torch.equal(r.ids, route.ids) and torch.equal(r.weights, route.weights)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, r = run()
    for _ in range(5):
        made.fill_(float("nan"))
        h.fill_(float("nan"))
        graph.replay()
        assert torch.equal(z, ref) and torch.equal(r.ids, route.ids) and torch.equal(r.weights, route.weights)
    assert q.last_device_error() == 0

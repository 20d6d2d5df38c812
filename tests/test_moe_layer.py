"""The whole mixture-of-experts layer against the calls that it stands for, and
against 64 bits.

The layer's routing and products are those of moe_route, moe_gate_up and
moe_down.  Its logits are f32 sums in an order of its own, so the comparison
takes its ids and weights and checks them by themselves: the ids are the best
by 64-bit logits unless picks are closer than the logits' error, K 2^-24 sum
|x r| at most; a weight's relative error is then 2 top_k exp'(l) of that, and a
few roundings.  Tolerances of y, from the formats, with T = sum_j p_j sum |h_j| |w| and u the
type's unit roundoff: the products' 1e-5 of test_q4g.py for each of the two
(the first's, through silu, at most 2.2 of it), what h loses as two pieces
(two truncations to 8 bits in bf16, two roundings to 11 in f16, three pieces in
f32) and u |y| for the result's rounding."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
UH = {"f32": 2.0 ** -24, "f16": 2.0 ** -22, "bf16": 2.0 ** -16}


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


def expert_weights(q, E, N, K, G, zeros, sdt, seed, gate_up=False):
    g = rng(seed)
    q4 = torch.randint(0, 16, (E, N, K), generator=g)
    s = ((0.5 + torch.rand((E, N, K // G), generator=g)) * (0.3 / K ** 0.5)).to(DT[sdt])
    z = torch.randint(0, 16, (E, N, K // G), generator=g) if zeros else None
    zd = 8.0 if z is None else z.double().repeat_interleave(G, 2)
    codes = (q4[..., 0::2] | (q4[..., 1::2] << 4)).to(torch.uint8)
    w = q.q4g_pack(codes.cuda(), s.cuda(), None if z is None else z.to(torch.uint8).cuda(), gate_up=gate_up)
    return w, s.double().repeat_interleave(G, 2) * (q4.double() - zd)


def make(q, T, E, K, F, N, G, G2, dt, seed=1, zeros=True):
    sdt = "bf16" if dt == "bf16" else "f16"
    up, wu = expert_weights(q, E, 2 * F, K, G, zeros, sdt, seed, True)
    down, wd = expert_weights(q, E, N, F, G2, zeros, sdt, seed + 1)
    x = torch.randn((T, K), generator=rng(seed + 2)).to(DT[dt])
    router = (torch.randn((E, K), generator=rng(seed + 3)) * (1.5 / K ** 0.5)).to(DT[dt])
    return up, wu, down, wd, x, router


def exact(x, ids, weights, wu, wd, dt):
    """y in 64 bits with this routing, and how far it may be off."""
    T, F = x.shape[0], wd.shape[2]
    y, tol = torch.zeros((T, wd.shape[1]), dtype=torch.float64), torch.zeros((T, wd.shape[1]), dtype=torch.float64)
    for t in range(T):
        xt = x[t].double()
        for e, p in zip(ids[t].tolist(), weights[t].double().tolist()):
            both, size = wu[e] @ xt, wu[e].abs() @ xt.abs()
            g, u = both[:F], both[F:]
            s = torch.sigmoid(g)
            h = g * s * u
            # silu' <= 1.1, |silu(g)| <= |g|
            dh = 1e-5 * (1.1 * size[:F] * u.abs() + (g * s).abs() * size[F:]) + 8 * 2.0 ** -22 * h.abs() + UH[dt] * h.abs() + (2.0 ** -25 if dt == "f16" else 0)
            y[t] += p * (wd[e] @ h)
            tol[t] += p * (wd[e].abs() @ (dh + 1e-5 * h.abs()))
    return y, tol + U[dt] * y.abs() + (2.0 ** -25 if dt == "f16" else 0)


CASES = [
    # T, E, k, K, F, N, G, G2, dt, score
    (1, 8, 2, 128, 64, 128, 32, 32, "bf16", "softmax"), (1, 64, 8, 2048, 1024, 2048, 128, 128, "bf16", "softmax"), (1, 16, 4, 576, 192, 576, 64, 64, "f32", "sigmoid"),
    (2, 5, 5, 96, 96, 50, 32, 96, "f16", "softmax"), (3, 128, 6, 512, 256, 500, 64, 32, "f32", "sigmoid"), (4, 64, 8, 1024, 128, 1024, 128, 64, "f16", "softmax"),
    (4, 512, 3, 64, 32, 64, 32, 32, "bf16", "sigmoid"), (5, 64, 8, 512, 256, 512, 128, 128, "bf16", "softmax"), (5, 3, 1, 32, 32, 1, 32, 32, "f32", "softmax"),
    (7, 100, 7, 320, 160, 333, 32, 32, "f16", "sigmoid"), (16, 64, 8, 1024, 512, 1024, 64, 64, "f16", "softmax"), (16, 8, 8, 256, 128, 256, 128, 64, "f32", "softmax"),
    (17, 8, 2, 512, 256, 512, 64, 128, "bf16", "sigmoid"), (32, 16, 4, 576, 192, 576, 64, 64, "bf16", "softmax"), (32, 300, 8, 256, 128, 256, 64, 32, "f32", "sigmoid"),
    (32, 1, 1, 160, 96, 100, 32, 32, "f16", "softmax"), (9, 32, 32, 128, 64, 128, 64, 64, "f16", "softmax"), (32, 512, 32, 64, 32, 40, 32, 32, "f16", "softmax"),
    (32, 33, 32, 96, 64, 64, 32, 64, "f32", "sigmoid"), (20, 8, 1, 4096, 64, 100, 128, 64, "f32", "softmax"), (1, 40, 32, 256, 64, 300, 32, 64, "bf16", "softmax")]


@pytest.mark.parametrize("T,E,k,K,F,N,G,G2,dt,score", CASES)
def test_layer(q, T, E, k, K, F, N, G, G2, dt, score):
    up, wu, down, wd, x, router = make(q, T, E, K, F, N, G, G2, dt, zeros=E % 2 == 0)
    bias = 0.1 * torch.randn(E, generator=rng(9)) if score == "sigmoid" and T % 2 else None
    c = dict(score=score, bias=None if bias is None else bias.cuda())
    y, r = q.moe_layer(up, down, router.cuda(), x.cuda(), k, route=True, **c)
    ids, weights = r.ids.cpu(), r.weights.cpu()
    # the routing
    l, size = x.double() @ router.double().T, x.double().abs() @ router.double().abs().T
    err = (K * 2.0 ** -24 * size).max()
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    pick = s + bias.double() if bias is not None else l
    mine = pick.gather(1, ids.long())
    best = pick.sort(1, descending=True).values[:, :k]
    assert ((mine - best).abs() <= 2 * err + 1e-6).all() and all(len(set(i.tolist())) == k for i in ids)
    w = s.gather(1, ids.long())
    w = w / w.sum(1, keepdim=True)
    assert ((weights - w).abs() <= w * (4 * err + 1e-5)).all()
    # the products, with this routing
    ref, tol = exact(x, ids, weights, wu, wd, dt)
    bad = ~((y.double().cpu() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst at {torch.nonzero(bad)[0].tolist()}"
    # the same on every run, and without the routing
    assert torch.equal(y, q.moe_layer(up, down, router.cuda(), x.cuda(), k, **c))
    # and what the calls that it stands for make of this routing, which round h to the type, and f16 weights of many rows too
    order = torch.sort(ids.flatten(), stable=True)
    off = torch.searchsorted(order.values, torch.arange(E + 1, dtype=torch.int32)).int()
    full = q.Route(r.ids, r.weights, off.cuda(), order.indices.int().cuda())
    z = q.moe_down(down, q.moe_gate_up(up, x.cuda(), full), full)
    assert float((y.double() - z.double()).norm().cpu()) <= (4 * U[dt] + 4e-5) * float(ref.norm())
    assert q.last_device_error() == 0


@pytest.mark.parametrize("E,groups,top_groups,group_score", [(64, 8, 3, "max"), (64, 8, 4, "top2"), (60, 5, 2, "top2"), (256, 8, 4, "top2"), (96, 3, 2, "max")])
def test_groups_are_routed_as_moe_route_does(q, E, groups, top_groups, group_score):
    """Logits that both sides form exactly: small integers."""
    T, K, F, N, k = 6, 64, 32, 64, 4
    up, wu, down, wd, _, _ = make(q, T, E, K, F, N, 32, 32, "bf16")
    x = torch.randint(-3, 4, (T, K), generator=rng(5)).bfloat16().cuda()
    router = (torch.randint(-3, 4, (E, K), generator=rng(6)) / 16).bfloat16().cuda()
    bias = (torch.randint(-100, 101, (E,), generator=rng(7)) * 0.001).cuda()
    c = dict(score="sigmoid", bias=bias, groups=groups, top_groups=top_groups, group_score=group_score, scale=2.5, renorm=False)
    y, r = q.moe_layer(up, down, router, x, k, route=True, **c)
    ref = q.moe_route(x.float() @ router.float().T, k, **c)
    assert torch.equal(r.ids, ref.ids) and torch.equal(r.weights, ref.weights)
    y64, tol = exact(x.cpu(), r.ids.cpu(), r.weights.cpu(), wu, wd, "bf16")
    assert ((y.double().cpu() - y64).abs() <= tol).all()


def test_tokens_that_agree_and_masked_experts(q):
    """Every token takes the same experts (one item has all rows); experts with a bias of -inf are never taken."""
    T, E, K, F, N, k = 32, 16, 128, 64, 128, 2
    up, wu, down, wd, x, router = make(q, T, E, K, F, N, 64, 64, "f16")
    bias = torch.full((E,), -float("inf"))
    bias[[3, 11]] = 0.0
    y, r = q.moe_layer(up, down, router.cuda(), x.cuda(), k, score="sigmoid", bias=bias.cuda(), route=True)
    assert set(r.ids.flatten().tolist()) == {3, 11}
    ref, tol = exact(x, r.ids.cpu(), r.weights.cpu(), wu, wd, "f16")
    assert ((y.double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dt,rdt", [("bf16", "f32"), ("f16", "bf16"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("T", [1, 3, 11])
def test_routers_of_other_types(q, T, dt, rdt):
    E, K, F, N, k = 24, 192, 64, 96, 3
    up, wu, down, wd, x, _ = make(q, T, E, K, F, N, 64, 64, dt)
    router = (torch.randint(-8, 9, (E, K), generator=rng(4)) / 64).to(DT[rdt])  # exact in each
    y, r = q.moe_layer(up, down, router.cuda(), x.cuda(), k, route=True)
    l = x.double() @ router.double().T
    best = l.sort(1, descending=True).values[:, :k]
    err = (K * 2.0 ** -24 * (x.double().abs() @ router.double().abs().T)).max()
    assert ((l.gather(1, r.ids.cpu().long()) - best).abs() <= 2 * err).all()
    ref, tol = exact(x, r.ids.cpu(), r.weights.cpu(), wu, wd, dt)
    assert ((y.double().cpu() - ref).abs() <= tol).all()


def test_bad_tokens_stay_to_themselves(q):
    T, E, K, F, N, k = 7, 16, 128, 64, 128, 3
    up, _, down, _, x, router = make(q, T, E, K, F, N, 64, 64, "f32")
    x, router = x.cuda(), router.cuda()
    y = q.moe_layer(up, down, router, x, k)
    x[2, 5] = float("nan")
    z = q.moe_layer(up, down, router, x, k)
    keep = [i for i in range(T) if i != 2]
    assert not torch.isfinite(z[2]).any() and torch.isfinite(z[keep]).all()
    assert torch.allclose(z[keep], y[keep], rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("T", [1, 3, 20])
def test_rows_apart_canary_stream_graph_and_workspace(q, T):
    E, K, F, N, k = 32, 256, 128, 200, 4
    up, _, down, _, x, router = make(q, T, E, K, F, N, 64, 64, "bf16")
    x, router = x.cuda(), router.cuda()
    y = q.moe_layer(up, down, router, x, k)
    wide = torch.full((T, K + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 32:32 + K] = x
    buf = torch.full((T * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    n = q.moe_layer_workspace(up, down, torch.bfloat16, T, k)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    q.moe_layer(up, down, router, wide[:, 32:32 + K], k, out=buf[:T * N].view(T, N), workspace=ws[:n])
    assert torch.equal(buf[:T * N].view(T, N), y) and bool((buf[T * N:] == 7).all()) and bool((ws[n:] == 0xFF).all())
    with pytest.raises(q.QmmError) as e:
        q.moe_layer(up, down, router, x, k, workspace=ws[:n - 16])
    assert e.value.status == 5
    # two calls at once, on two streams
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    got = [[q.moe_layer(up, down, router, x, k, stream=s) for s in sides] for _ in range(10)]
    for s in sides:
        s.synchronize()
    assert all(torch.equal(z, y) for pair in got for z in pair)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = q.moe_layer(up, down, router, x, k)
        z2 = q.moe_layer(up, down, router, x, k)
    x2 = torch.randn((T, K), generator=rng(8)).bfloat16().cuda()
    ref = q.moe_layer(up, down, router, x2, k)
    x.copy_(x2)
    for _ in range(3):
        z.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, ref) and torch.equal(z2, ref)


def test_the_block_of_a_decoder(q):
    """What these operators are for, as a decode step calls them: norm to 8-bit rows, a projection, norm and residual, the
    mixture-of-experts layer, norm and residual.  Each against 64 bits from the step before it as it came out, and in a
    graph the same again."""
    T, K, E, F, k = 6, 512, 16, 128, 4
    up, wu, down, wd, x, router = make(q, T, E, K, F, K, 64, 64, "bf16")
    proj = torch.randn((K, K), generator=rng(20)) / K ** 0.5
    wp = q.q8c_pack(*q.q8c_quantize(proj.cuda()))
    n1, n2, n3, post = ((1 + 0.2 * torch.randn(K, generator=rng(21 + i))).bfloat16().cuda() for i in range(4))
    router, x = router.cuda(), x.cuda()

    def block(x):
        r0, rows = q.block_norm(x, n1, quantize=True)
        a = q.q8c_matmul(wp, rows, dtype=torch.bfloat16)
        r1, h = q.block_norm(a, n2, residual=r0, post_weight=post)
        m, route = q.moe_layer(up, down, router, h, k, route=True)
        r2, out = q.block_norm(m, n3, residual=r1, scale=0.5)
        return rows, a, r1, h, route, m, r2, out

    rows, a, r1, h, route, m, r2, out = block(x)
    norm = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    near = lambda got, ref, tol: float((got.double() - ref).norm()) <= tol * float(ref.norm())  # noqa: E731
    u = U["bf16"]
    # the projection: integers, exactly; the norms: one rounding of each result
    w = q.q8c_dequantize(wp).double()
    assert near(a, (rows.codes.double() * rows.scales.double()[:, None]) @ w.T, u)
    assert near(r1, x.double() + norm(a.double()) * post.double(), u)
    assert near(h, norm(x.double() + norm(a.double()) * post.double()) * n2.double(), u)
    ref, tol = exact(h.cpu(), route.ids.cpu(), route.weights.cpu(), wu, wd, "bf16")
    assert ((m.double().cpu() - ref).abs() <= tol).all()
    assert near(r2, r1.double() + 0.5 * m.double(), u) and near(out, norm(r1.double() + 0.5 * m.double()) * n3.double(), u)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = block(x)[-1]
    for _ in range(2):
        again.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)
    assert q.last_device_error() == 0


def test_refusals_and_empty(q):
    E, K, F, N = 8, 64, 32, 64
    up, _, down, _, x, router = make(q, 4, E, K, F, N, 32, 32, "f16")
    x, router = x.cuda(), router.cuda()
    assert q.moe_layer(up, down, router, x[:0], 2).shape == (0, N)
    for bad in (dict(x=x.repeat(9, 1)), dict(top_k=0), dict(top_k=9), dict(gate_up=down), dict(down=up), dict(groups=3), dict(groups=8, top_groups=1, top_k=2)):
        with pytest.raises((q.QmmError, ValueError)):
            q.moe_layer(**{**dict(gate_up=up, down=down, router=router, x=x, top_k=2), **bad})
    with pytest.raises(q.QmmError) as e:  # rows on no 16-byte boundary
        q.moe_layer(up, down, router, torch.empty((4, K + 1), dtype=torch.float16, device="cuda")[:, 1:], 2)
    assert e.value.status == 4
    for bad in (dict(router=router[:7]), dict(router=router.t().contiguous().t()), dict(router=router.cpu()), dict(x=x[:, :32]), dict(bias=torch.zeros(7, device="cuda")),
                dict(out=torch.empty((4, N), device="cuda"))):
        with pytest.raises(ValueError):
            q.moe_layer(**{**dict(gate_up=up, down=down, router=router, x=x, top_k=2), **bad})


@pytest.mark.parametrize("T", [1, 20])
def test_injected_failures(q, T):
    E, K, F, N, k = 32, 256, 128, 200, 4
    up, _, down, _, x, router = make(q, T, E, K, F, N, 64, 64, "f16")
    x, router = x.cuda(), router.cuda()
    ref = q.moe_layer(up, down, router, x, k)
    torch.cuda.synchronize()
    assert q.last_device_error() == 0
    q.test_set_wait_limit(22)
    try:
        q.test_inject("stall", 1, 0)
        q.moe_layer(up, down, router, x, k)
        torch.cuda.synchronize()  # the call ends: every wait is bounded
        assert q.last_device_error() == 7
    finally:
        q.test_inject("off")
        q.test_set_wait_limit(0)
    out = torch.full_like(ref, 7.0)
    q.test_inject("launch_failure", 1)
    try:
        with pytest.raises(q.QmmError) as e:
            q.moe_layer(up, down, router, x, k, out=out)
        assert e.value.status == 6
    finally:
        q.test_inject("off")
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())
    assert torch.equal(q.moe_layer(up, down, router, x, k), ref) and q.last_device_error() == 0

"""4-bit group-scale products and mixture-of-experts operators against plain
64-bit implementations, element by element and in the 2-norm.

Tolerances, derived from the formats.  With T = sum |x| |w| of an element and
u the output type's unit roundoff (2^-24, 2^-11, 2^-8):
  - every product: u |y| for the one rounding of the output, and 1e-5 T for
    the f32 sums (the bound of this library's other f32 products);
  - the GEMM with f16 or bf16 activations rounds each weight to f16: 2^-11 T;
    bf16 values below 2^-29 of their row's largest lose bits: 2^-29 T too.
In the 2-norm the weights' roundings are independent, so their sum's relative
error is at most 2^-11 (and the output's u): u + 2^-11, or 1e-5 for f32.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


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


def make(E, N, K, G, zeros, sdt, seed, scale=0.01):
    """Checkpoint tensors on the CPU, and the weights in 64 bits."""
    g = rng(seed)
    q4 = torch.randint(0, 16, (E, N, K), generator=g)
    s = (scale * (0.25 + torch.rand((E, N, K // G), generator=g))).to(DT[sdt])
    s[0, 0] = -s[0, 0]
    z = torch.randint(0, 16, (E, N, K // G), generator=g) if zeros else None
    zd = 8.0 if z is None else z.double().repeat_interleave(G, 2)
    w = s.double().repeat_interleave(G, 2) * (q4.double() - zd)
    codes = (q4[..., 0::2] | (q4[..., 1::2] << 4)).to(torch.uint8)
    return codes, s, None if z is None else z.to(torch.uint8), w


def pack(q, t, gate_up=False):
    codes, s, z, _ = t
    return q.q4g_pack(codes.cuda(), s.cuda(), None if z is None else z.cuda(), gate_up=gate_up)


def tolerance(dt, y, T, gemm):
    e = U[dt] * y.abs() + 1e-5 * T
    return e + (2.0 ** -11 + 2.0 ** -29) * T if gemm and dt != "f32" else e


def norm_tolerance(dt, gemm):
    return 1e-5 if dt == "f32" else U[dt] + (2.0 ** -11 if gemm else 1e-5)


def check(got, ref, tol, norm):
    got = got.double().cpu()
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst at {torch.nonzero(bad)[0].tolist()}: {got[bad][:3]} for {ref[bad][:3]}"
    assert float((got - ref).norm()) <= norm * float(ref.norm()) + 1e-30


# ------------------------------------------------------------------ layout


@pytest.mark.parametrize("E,N,K,G,zeros,sdt,gate_up", [
    (1, 1, 32, 32, False, "f16", False), (1, 17, 96, 32, True, "bf16", False), (3, 40, 192, 64, True, "f16", False),
    (2, 50, 256, 128, True, "bf16", True), (2, 18, 160, 32, False, "f16", True), (1, 33, 512, 512, True, "f16", False),
    (1, 20, 192, 96, True, "f16", False)])
def test_pack_keeps_every_weight(q, E, N, K, G, zeros, sdt, gate_up):
    t = make(E, N, K, G, zeros, sdt, 1)
    w = pack(q, t, gate_up)
    assert torch.equal(q.q4g_dequantize(w).double().cpu(), t[3])


def test_pack_q4_0_is_the_block_format(q):
    x = torch.randn((2, 48, 320), generator=rng(3)).cuda()
    wq = q.quantize_weights(x.reshape(96, 320).contiguous(), "q4_0")
    ref = q.dequantize(wq, "q4_0", 320)
    w = q.q4g_pack_q4_0(wq.reshape(2, 48, -1), 320)
    assert torch.equal(q.q4g_dequantize(w).reshape(96, 320), ref)


# ------------------------------------------------------------------ dense product

DENSE = [
    # M, N, K, G, zeros, dt: few rows or a small matrix
    (1, 576, 576, 32, False, "f32"), (1, 1, 32, 32, True, "f16"), (1, 15, 64, 64, False, "bf16"), (2, 17, 96, 32, True, "f32"),
    (3, 100, 1536, 128, True, "bf16"), (7, 33, 160, 32, True, "f16"), (8, 192, 576, 64, False, "bf16"), (9, 48, 128, 128, True, "f16"),
    (10, 40, 320, 64, True, "f32"), (16, 300, 1024, 128, False, "f16"), (31, 70, 192, 64, True, "bf16"), (32, 576, 576, 32, True, "f16"),
    (1, 96, 16384, 128, True, "f32"), (5, 40, 14336, 128, True, "f32"), (32, 24, 14336, 64, True, "bf16"), (1, 9000, 128, 128, True, "f16"),
    (1, 5000, 256, 64, False, "bf16"),
    # more
    (33, 128, 256, 128, True, "f16"), (33, 17, 32, 32, True, "bf16"), (64, 130, 96, 32, False, "f16"), (100, 576, 576, 64, True, "bf16"),
    (129, 257, 320, 64, True, "f16"), (257, 300, 1536, 128, True, "bf16"), (300, 129, 160, 32, True, "f16"), (1000, 64, 128, 128, False, "bf16"),
    (11, 40, 64, 64, True, "f32"), (37, 300, 1024, 32, True, "f32"), (130, 200, 576, 64, True, "f32"), (300, 144, 1600, 32, False, "f32"),
    (33, 40, 14336, 128, True, "f32"), (40, 2500, 320, 64, True, "f16"), (530, 2000, 256, 128, True, "bf16"),
    (17, 4100, 4096, 64, True, "f16"), (12, 6000, 2048, 32, True, "f32"), (260, 4000, 1088, 64, True, "f16"), (65, 9000, 320, 64, True, "bf16"),
    (200, 1030, 4160, 32, False, "bf16"), (70, 4500, 672, 32, True, "f32"), (1100, 500, 2048, 128, True, "f16"), (700, 3000, 96, 32, True, "bf16")]


@pytest.mark.parametrize("M,N,K,G,zeros,dt", DENSE)
def test_matmul(q, M, N, K, G, zeros, dt):
    t = make(1, N, K, G, zeros, "f16" if dt == "f16" else "bf16", 7)
    x = torch.randn((M, K), generator=rng(8)).to(DT[dt])
    if M > 2:
        x[1] = 0
        x[2] *= 100
    w = pack(q, t)
    y = q.q4g_matmul(w, x.cuda())
    W, xd = t[3][0], x.double()
    ref, T = xd @ W.T, xd.abs() @ W.abs().T
    gemm = M > 8 and M * N * K > 160_000_000  # else no weight is rounded
    check(y, ref, tolerance(dt, ref, T, gemm), norm_tolerance(dt, gemm))
    assert torch.equal(y, q.q4g_matmul(w, x.cuda()))  # the same on every run
    assert q.last_device_error() == 0


@pytest.mark.parametrize("M,dt", [(3, "f16"), (9, "f32"), (300, "f16"), (300, "bf16"), (300, "f32")])
def test_matmul_rows_apart_and_canary(q, M, dt):
    N, K = 1900, 320
    t = make(1, N, K, 64, True, "f16", 9)
    w = pack(q, t)
    wide = torch.full((M, K + 64), float("nan"), dtype=DT[dt], device="cuda")
    x = torch.randn((M, K), generator=rng(1)).to(DT[dt])
    wide[:, 32:32 + K] = x.cuda()
    buf = torch.full((M * N + 64,), 7.0, dtype=DT[dt], device="cuda")
    out = buf[:M * N].view(M, N)
    q.q4g_matmul(w, wide[:, 32:32 + K], out=out)
    assert torch.equal(out, q.q4g_matmul(w, x.cuda()))
    assert bool((buf[M * N:] == 7).all())


@pytest.mark.parametrize("M,dt", [(4, "f16"), (4, "bf16"), (4, "f32"), (600, "f16"), (600, "bf16"), (600, "f32")])
def test_matmul_keeps_bad_rows_to_themselves(q, M, dt):
    N, K = 1500, 192
    w = pack(q, make(1, N, K, 64, True, "bf16", 4))
    x = torch.randn((M, K), generator=rng(2)).to(DT[dt]).cuda()
    bad = x.clone()
    bad[1, 5] = float("nan")
    bad[3, 7] = float("inf")
    y, z = q.q4g_matmul(w, x), q.q4g_matmul(w, bad)
    assert torch.isnan(z[1]).all() and not torch.isfinite(z[3]).any()
    keep = [i for i in range(M) if i not in (1, 3)]
    assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("dt,M", [("f32", 2), ("bf16", 2), ("bf16", 700), ("f32", 700), ("f16", 2), ("f16", 700)])
def test_matmul_extreme_magnitudes(q, dt, M):
    """Scales and activations near the ends of their types' ranges."""
    N, K = 1000, 256
    sdt = "f16" if dt == "f16" else "bf16"
    for scale, xs in ((1e-4, 1e3), (100.0, 1e-3)) if dt == "f16" else ((1e-25, 1e20), (1e20, 1e-25)):
        t = make(1, N, K, 64, True, sdt, 5, scale)
        x = (xs * torch.randn((M, K), generator=rng(6))).to(DT[dt])
        ref, T = x.double() @ t[3][0].T, x.double().abs() @ t[3][0].abs().T
        tiny = 2.0 ** -24 if dt == "f16" else 0.0  # an f16 output may be subnormal
        check(q.q4g_matmul(pack(q, t), x.cuda()), ref, tolerance(dt, ref, T, M > 10) + tiny, norm_tolerance(dt, M > 10) + tiny)


def test_matmul_empty_and_streams(q):
    w = pack(q, make(1, 64, 128, 64, True, "f16", 4))
    assert q.q4g_matmul(w, torch.empty((0, 128), dtype=torch.float16, device="cuda")).shape == (0, 64)
    for M in (3, 20000):
        x = torch.randn((M, 128), generator=rng(2)).to(torch.bfloat16).cuda()
        y = q.q4g_matmul(w, x)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        z = q.q4g_matmul(w, x, stream=side)
        side.synchronize()
        assert torch.equal(y, z)


@pytest.mark.parametrize("M", [2, 400])
def test_matmul_in_a_graph(q, M):
    w = pack(q, make(1, 2000, 256, 64, True, "f16", 4))
    x = torch.randn((M, 256), generator=rng(2)).cuda()
    y = q.q4g_matmul(w, x)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q.q4g_matmul(w, x)
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(g):
        z = q.q4g_matmul(w, x)
    x.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, 2 * y)


# ------------------------------------------------------------------ routing


def plain_route(l, k, score, bias, groups, top_groups, group_score, renorm, scale):
    """Loops in 64 bits over picks that are apart or equal."""
    l = np.where(np.isnan(l), -np.inf, l)
    T, E = l.shape
    ids, wts = np.zeros((T, k), np.int32), np.zeros((T, k))
    rows = {}  # a row's answer: long calls repeat rows
    for t in range(T):
        key = l[t].tobytes()
        if key in rows:
            ids[t], wts[t] = rows[key]
            continue
        if score == "softmax":
            m = l[t].max()
            e = np.where(l[t] == m, 1.0, np.exp(l[t] - m) if np.isfinite(m) else 0.0) if m > -np.inf else np.zeros(E)
            s = e / e.sum() if e.sum() > 0 else e
            pick = l[t] if bias is None else s + bias
        else:
            s = 1 / (1 + np.exp(-l[t]))
            pick = s if bias is None else s + bias
        pick = pick.copy()
        if groups > 1:
            parts = pick.reshape(groups, -1)
            val = [sum(sorted(p)[-2:]) if group_score == "top2" else max(p) for p in parts]
            kept = sorted(range(groups), key=lambda g: (-val[g], g))[:top_groups]
            out = np.ones(groups, bool)
            out[kept] = False
            allowed = ~np.repeat(out, E // groups)
        else:
            allowed = np.ones(E, bool)
        best = sorted((e for e in range(E) if allowed[e]), key=lambda e: (-pick[e], e))[:k]
        ids[t] = best
        w = s[best]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        wts[t] = scale * w
        rows[key] = ids[t], wts[t]
    return ids, wts


def plain_order(ids, E):
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    return np.searchsorted(flat[order], np.arange(E + 1)), order


ROUTES = [
    # T, E, k, score, bias, groups, top_groups, group_score, renorm, dt
    (1, 1, 1, "softmax", False, 1, 1, "max", True, "f32"), (1, 64, 6, "softmax", False, 1, 1, "max", True, "f32"),
    (5, 8, 2, "softmax", False, 1, 1, "max", False, "bf16"), (33, 60, 4, "sigmoid", False, 1, 1, "max", True, "f16"),
    (300, 256, 8, "sigmoid", True, 8, 4, "top2", True, "bf16"), (70, 160, 6, "softmax", False, 8, 3, "max", False, "f32"),
    (40, 512, 32, "sigmoid", True, 32, 8, "top2", True, "f32"), (129, 33, 33 - 1, "softmax", False, 1, 1, "max", True, "f16"),
    (50, 12, 3, "softmax", True, 3, 2, "max", True, "f32"), (64, 24, 5, "sigmoid", False, 12, 5, "top2", False, "f32"), (200, 64, 6, "sigmoid", False, 4, 2, "max", True, "f16"),
    (31, 7, 7, "sigmoid", True, 7, 7, "max", True, "f32"), (2000, 96, 8, "softmax", False, 1, 1, "max", True, "bf16"),
    (9000, 16, 2, "softmax", False, 1, 1, "max", True, "f16"), (32, 300, 8, "softmax", False, 1, 1, "max", True, "f32"),
    (70000, 9, 1, "softmax", False, 1, 1, "max", True, "f32"), (4099, 500, 3, "sigmoid", False, 1, 1, "max", True, "f16"),
    (70000, 512, 2, "softmax", False, 1, 1, "max", True, "bf16")]


@pytest.mark.parametrize("T,E,k,score,bias,groups,top_groups,group_score,renorm,dt", ROUTES)
def test_route(q, T, E, k, score, bias, groups, top_groups, group_score, renorm, dt):
    g = rng(T + E)
    # logits in steps of 1/8: ties, and else picks that no f32 rounding can swap
    l = (torch.randint(-24, 25, (T, E), generator=g).float() / 8).to(DT[dt])
    l = l[torch.arange(T) % 1500]
    b = torch.randint(-8, 9, (E,), generator=g).float() / 16 if bias else None
    if bias:  # redraw rows with picks closer than 1e-5 that are not equal
        for _ in range(50):
            d = l.double()
            p = (torch.sigmoid(d) if score == "sigmoid" else torch.softmax(d, 1)) + b.double()
            gap = p.sort(1).values.diff(dim=1)
            near = ((gap > 1e-12) & (gap < 1e-5)).any(1)
            if groups > 1:
                v = p.unflatten(1, (groups, -1)).sort(2, descending=True).values[..., :2 if group_score == "top2" else 1].sum(2)
                gap = v.sort(1).values.diff(dim=1)
                near |= ((gap > 1e-12) & (gap < 1e-5)).any(1)
            if not near.any():
                break
            l[near] = (torch.randint(-24, 25, (int(near.sum()), E), generator=g).float() / 8).to(DT[dt])
        l = l[~near]
        T = l.shape[0]
        assert T > 0
    r = q.moe_route(l.cuda(), k, score=score, bias=None if b is None else b.cuda(), groups=groups, top_groups=top_groups,
                    group_score=group_score, renorm=renorm, scale=1.5)
    ids, wts = plain_route(l.double().numpy(), k, score, None if b is None else b.double().numpy(), groups, top_groups, group_score, renorm, 1.5)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.abs(r.weights.double().cpu().numpy() - wts).max() <= 1e-6
    off, order = plain_order(ids, E)
    assert np.array_equal(r.offsets.cpu().numpy(), off) and np.array_equal(r.order.cpu().numpy(), order)
    bare = q.moe_route(l.cuda(), k, score=score, bias=None if b is None else b.cuda(), groups=groups, top_groups=top_groups,
                       group_score=group_score, renorm=renorm, scale=1.5, order=False)
    assert bare.order is None and torch.equal(bare.ids, r.ids) and torch.equal(bare.weights, r.weights)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_rows(q, score):
    """-inf, NaN, the type's lowest value, +inf and rows that the mask leaves empty."""
    inf = float("inf")
    l = torch.zeros((7, 40))
    l[0] = -inf
    l[1] = float("nan")
    l[2, :38] = -inf
    l[3] = torch.finfo(torch.float32).min
    l[4, 5] = inf
    l[5, 3] = float("nan")
    l[6, :] = -0.0
    l[6, 20:] = 0.0
    r = q.moe_route(l.cuda(), 4, score=score)
    ids, wts = plain_route(l.double().numpy(), 4, score, None, 1, 1, "max", True, 1.0)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.abs(r.weights.double().cpu().numpy() - wts).max() <= 1e-6


def test_route_rows_apart_and_no_tokens(q):
    l = torch.randn((50, 48), generator=rng(1)).cuda()
    wide = torch.full((50, 100), 50.0, device="cuda")
    wide[:, 9:57] = l
    for a, b in zip(q.moe_route(wide[:, 9:57], 5), q.moe_route(l, 5)):
        assert torch.equal(a, b)
    r = q.moe_route(l[:0], 5)
    assert r.ids.shape == (0, 5) and bool((r.offsets == 0).all()) and r.order.numel() == 0


# ------------------------------------------------------------------ experts


def routing(q, T, E, k, kind, seed):
    g = rng(seed)
    if kind == "even":
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    elif kind == "one":  # every token's first expert is the last one
        ids = torch.stack([torch.cat([torch.tensor([E - 1]), torch.randperm(max(E - 1, 1), generator=g)[:k - 1]]) for _ in range(T)])
    else:  # skipped slots, a token without experts
        ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
        ids[torch.rand((T, k), generator=g) < 0.3] = -1
        ids[T // 2] = E
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    sorted_ids = flat[order]
    order = order[(sorted_ids >= 0) & (sorted_ids < E)]
    off = torch.searchsorted(flat[order].contiguous(), torch.arange(E + 1))
    order = torch.cat([order, torch.zeros(T * k - order.numel(), dtype=torch.int64)])
    w = torch.rand((T, k), generator=g) + 0.1
    i32 = lambda t: t.to(torch.int32).contiguous().cuda()  # noqa: E731
    return ids, w, q.Route(i32(ids), w.cuda(), i32(off), i32(order))


EXPERTS = [
    # T, E, k, K, F, G, zeros, dt, routing
    (1, 8, 2, 256, 64, 64, True, "bf16", "even"), (1, 16, 6, 96, 33, 32, True, "f16", "even"), (2, 4, 4, 192, 40, 64, False, "f32", "even"),
    (3, 5, 2, 160, 17, 32, True, "bf16", "skip"), (7, 12, 3, 320, 50, 64, True, "f16", "even"), (16, 128, 8, 256, 40, 128, True, "bf16", "even"),
    (20, 6, 2, 128, 70, 128, True, "f32", "one"), (33, 8, 3, 96, 64, 32, False, "f16", "skip"), (60, 4, 2, 256, 100, 64, True, "bf16", "one"),
    (100, 4, 3, 320, 129, 64, True, "f16", "even"), (100, 1, 1, 192, 64, 64, True, "bf16", "even"), (150, 8, 4, 576, 72, 32, True, "f32", "even"),
    (300, 6, 2, 160, 130, 32, True, "bf16", "skip"), (700, 4, 2, 256, 72, 128, True, "f16", "one"), (90, 3, 2, 1600, 24, 64, True, "f32", "skip"),
    (40, 512, 8, 64, 16, 32, True, "f16", "even"), (1500, 6, 4, 128, 20, 64, True, "bf16", "even")]


def slot_products(xr, W, ids, E):
    """Per slot: x . W_e^T and sum |x| |W_e| in 64 bits (zeros where skipped)."""
    T, k = ids.shape
    y = torch.zeros((T, k, W.shape[1]), dtype=torch.float64)
    A = torch.zeros_like(y)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            x = xr[t, j]
            y[t, j], A[t, j] = x @ W[e].T, x.abs() @ W[e].abs().T
    return y, A


@pytest.mark.parametrize("T,E,k,K,F,G,zeros,dt,kind", EXPERTS)
def test_gate_up(q, T, E, k, K, F, G, zeros, dt, kind):
    t = make(E, 2 * F, K, G, zeros, "f16" if dt == "f16" else "bf16", 11)
    w = pack(q, t, gate_up=True)
    ids, _, route = routing(q, T, E, k, kind, 12)
    x = torch.randn((T, K), generator=rng(13)).to(DT[dt])
    out = torch.full((T, k, F), 3.0, dtype=DT[dt], device="cuda")
    h = q.moe_gate_up(w, x.cuda(), route, out=out)
    y, A = slot_products(x.double()[:, None].expand(T, k, K), t[3], ids, E)
    g, u = y[..., :F], y[..., F:]
    e = tolerance("f32", torch.zeros_like(A), A, False) if dt == "f32" else (1e-5 + 2.0 ** -11 + 2.0 ** -29) * A
    eg, eu = e[..., :F], e[..., F:]
    s = g * torch.sigmoid(g)
    ref = s * u
    tol = 1.1 * u.abs() * eg + s.abs() * eu + 1.1 * eg * eu + (U[dt] + 1e-6) * ref.abs() + (2.0 ** -24 if dt == "f16" else 0)
    on = ((ids >= 0) & (ids < E))[..., None].expand(T, k, F)
    got = h.double().cpu()
    assert bool((got[~on] == 3).all())  # skipped slots are not written
    # the product of two sums: twice the relative error of one (silu's slope is at most 1.1)
    check(got[on], ref[on], tol[on], 2.2 * norm_tolerance(dt, True))
    assert torch.equal(h, q.moe_gate_up(w, x.cuda(), route, out=out.clone()))
    assert q.last_device_error() == 0


@pytest.mark.parametrize("T,E,k,K,F,G,zeros,dt,kind", EXPERTS)
def test_down(q, T, E, k, K, F, G, zeros, dt, kind):
    N = 2 * F + 1
    t = make(E, N, K, G, zeros, "f16" if dt == "f16" else "bf16", 14)
    w = pack(q, t)
    ids, wt, route = routing(q, T, E, k, kind, 15)
    h = torch.randn((T, k, K), generator=rng(16)).to(DT[dt])
    y = q.moe_down(w, h.cuda(), route)
    p, A = slot_products(h.double(), t[3], ids, E)
    ref, A = (p * wt.double()[..., None]).sum(1), (A * wt.double()[..., None]).sum(1)
    check(y, ref, tolerance(dt, ref, A, True), norm_tolerance(dt, True))
    assert torch.equal(y, q.moe_down(w, h.cuda(), route))
    assert q.last_device_error() == 0


def test_layer_together(q):
    """Router, experts and a dense linear as a model runs them, from GGUF Q4_0 experts, with strided activations."""
    T, E, k, D, F = 37, 16, 4, 576, 192
    g = rng(20)
    x = torch.randn((T, 2 * D), generator=g).to(torch.bfloat16).cuda()[:, :D]
    wr = torch.randn((E, D), generator=g).cuda()
    w1 = (0.04 * torch.randn((E, 2 * F, D), generator=g)).cuda()
    w2 = (0.07 * torch.randn((E, D, F), generator=g)).cuda()
    q1 = q.quantize_weights(w1.view(-1, D), "q4_0")
    q2 = q.quantize_weights(w2.view(-1, F), "q4_0")
    p1 = q.q4g_pack_q4_0(q1.view(E, 2 * F, -1), D, gate_up=True)
    p2 = q.q4g_pack_q4_0(q2.view(E, D, -1), F)
    route = q.moe_route(x.float() @ wr.T, k)
    h = q.moe_gate_up(p1, x, route)
    y = q.moe_down(p2, h, route).double()
    W1, W2 = q.dequantize(q1, "q4_0", D).view(E, 2 * F, D).double(), q.dequantize(q2, "q4_0", F).view(E, D, F).double()
    both = torch.einsum("td,tknd->tkn", x.double(), W1[route.ids.long()])
    ref = both[..., :F] * torch.sigmoid(both[..., :F]) * both[..., F:]
    assert float((h.double() - ref).norm() / ref.norm()) < 2.0 ** -8 + 2 * 2.0 ** -11
    ref = (torch.einsum("tkf,tknf->tkn", h.double(), W2[route.ids.long()]) * route.weights.double()[..., None]).sum(1)
    assert float((y - ref).norm() / ref.norm()) < 2.0 ** -8 + 2.0 ** -11


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_gemm_keeps_the_precision(q, dt, G):
    """The norm of the error of many rows.  f16: gate_up rounds its output (2^-11 / sqrt(3) at most in the mean) and
    hardly anything else, one weight matrix adds its weights' rounding (as much again).  f32: activations of 22 bits,
    and sums that truncate over no more than 128 K."""
    T, E, k, D, F = 700, 8, 2, 1536, 640
    t = make(E, 2 * F, D, G, True, "f16", 31, scale=0.02)
    x = torch.randn((T, D), generator=rng(32)).to(DT[dt])
    route = q.moe_route(torch.randn((T, E), generator=rng(33)).cuda(), k)
    h = q.moe_gate_up(pack(q, t, gate_up=True), x.cuda(), route).double().cpu()
    ref = torch.empty((T, k, F), dtype=torch.float64)
    for e in range(E):
        at = (route.ids == e).nonzero().cpu()
        both = x[at[:, 0]].double() @ t[3][e].T
        ref[at[:, 0], at[:, 1]] = both[:, :F] * torch.sigmoid(both[:, :F]) * both[:, F:]
    half = 2.0 ** -11 / 3 ** 0.5
    assert float((h - ref).norm() / ref.norm()) < (2e-6 if dt == "f32" else 1.05 * half)
    w = tuple(None if v is None else v[:1] for v in t)
    ref = x.double() @ t[3][0].T
    y = q.q4g_matmul(pack(q, w), x.cuda()).double().cpu()
    assert float((y - ref).norm() / ref.norm()) < (1e-6 if dt == "f32" else 2 ** 0.5 * half)
    assert q.last_device_error() == 0


def test_matmul_of_many_tiles(q):
    """More tiles to a block than it looks up at its start."""
    M, N, K = 40000, 2050, 32
    t = make(1, N, K, 32, True, "f16", 41)
    x = torch.randn((M, K), generator=rng(42)).cuda()
    y = q.q4g_matmul(pack(q, t), x)
    ref = x.double() @ t[3][0].cuda().T
    T = x.double().abs() @ t[3][0].cuda().abs().T
    assert bool(((y.double() - ref).abs() <= 1e-5 * T).all())
    assert float((y.double() - ref).norm() / ref.norm()) < 1e-6
    assert q.last_device_error() == 0


def test_route_tensors_are_ordinary(q):
    """Parts of one allocation: apart, 16-byte aligned, and alive by themselves."""
    r = q.moe_route(torch.randn((5, 7), generator=rng(50)).cuda(), 3)
    spans = sorted((v.data_ptr(), v.data_ptr() + 4 * v.numel()) for v in r)
    assert all(a % 16 == 0 for a, _ in spans) and all(x[1] <= y[0] for x, y in zip(spans, spans[1:]))
    assert [v.dtype for v in r] == [torch.int32, torch.float32, torch.int32, torch.int32]
    assert all(v.is_contiguous() and v._version == 0 and not v.requires_grad for v in r)
    ids, kept = r.ids, r.ids.clone()
    del r
    torch.full((4096,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(ids, kept) and torch.equal(ids.add(1).sub_(1), kept) and torch.equal(ids.t().contiguous(), kept.t().contiguous())
    one = q.moe_route(torch.randn((5, 7), generator=rng(50)).cuda(), 3, order=False)
    assert one.offsets is None and one.order is None and torch.equal(one.ids, kept)


def test_refused_tensors(q):
    w = pack(q, make(1, 64, 128, 64, True, "f16", 4))
    x = torch.zeros((2, 128), dtype=torch.float16, device="cuda")
    for bad in (x.double(), x[:, :64], x.cpu(), x.t(), x[None]):
        with pytest.raises(ValueError):
            q.q4g_matmul(w, bad)
    with pytest.raises(q.QmmError):  # rows that do not start on 16 bytes
        q.q4g_matmul(w, torch.zeros((2, 132), dtype=torch.float16, device="cuda")[:, 1:129])
    with pytest.raises(ValueError):
        q.q4g_matmul(w, x, out=torch.empty((2, 63), dtype=torch.float16, device="cuda"))
    y = torch.zeros((20000, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(q.QmmError) as err:
        q.q4g_matmul(w, y, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert err.value.status == 5
    r = q.moe_route(torch.zeros((2, 4), device="cuda"), 2)
    with pytest.raises(q.QmmError):  # not packed as gate and up rows
        q.moe_gate_up(pack(q, make(4, 64, 128, 64, True, "f16", 4)), x, r)
    with pytest.raises(ValueError):  # another number of experts
        q.moe_gate_up(pack(q, make(5, 64, 128, 64, True, "f16", 4), gate_up=True), x, r)

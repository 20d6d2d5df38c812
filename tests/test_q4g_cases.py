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


# ------------------------------------------------------------------ what a caller hands over


def make(E, N, K, G, zeros, sdt, seed, scale=0.01):
    """Checkpoint tensors on the CPU, and the weights in 64 bits."""
    g = rng(seed)
    q4 = torch.randint(0, 16, (E, N, K), generator=g)
    s = (scale * (0.25 + torch.rand((E, N, K // G), generator=g))).to(sdt)
    z = torch.randint(0, 16, (E, N, K // G), generator=g) if zeros else None
    zd = 8.0 if z is None else z.double().repeat_interleave(G, 2)
    w = s.double().repeat_interleave(G, 2) * (q4.double() - zd)
    codes = (q4[..., 0::2] | (q4[..., 1::2] << 4)).to(torch.uint8)
    return codes, s, None if z is None else z.to(torch.uint8), w


def pack(q, t, gate_up=False):
    codes, s, z, _ = t
    return q.q4g_pack(codes.cuda(), s.cuda(), None if z is None else z.cuda(), gate_up=gate_up)


def test_refused_workspaces(q):
    """Memory of the host, and views whose bytes are not one piece: refused before any launch."""
    T, E, k, F = 600, 4, 2, 64
    x = torch.zeros((T, 128), dtype=torch.bfloat16, device="cuda")
    h = torch.zeros((T, k, F), dtype=torch.bfloat16, device="cuda")
    logits = torch.zeros((T, E), device="cuda")
    wm = pack(q, make(1, 5000, 128, 64, True, torch.float16, 4))
    wg, wd = pack(q, make(E, 2 * F, 128, 64, True, torch.float16, 4), True), pack(q, make(E, 128, F, 64, True, torch.float16, 4))
    r = q.moe_route(logits, k)
    calls = (lambda ws: q.q4g_matmul(wm, x, workspace=ws), lambda ws: q.moe_route(logits, k, workspace=ws),
             lambda ws: q.moe_gate_up(wg, x, r, workspace=ws), lambda ws: q.moe_down(wd, h, r, workspace=ws))
    n = 1 << 22  # bytes, enough for each of them
    good = torch.empty(n, dtype=torch.uint8, device="cuda")
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty((n, 2), dtype=torch.uint8, device="cuda")[:, 0],
                torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), torch.empty((16, n // 16), dtype=torch.uint8, device="cuda").t(),
                good.tolist()[:3]):
        for f in calls:
            with pytest.raises(ValueError):
                f(bad)
    for f in calls:
        a, b = f(None), f(good)
        for u, v in zip(a, b) if isinstance(a, tuple) else ((a, b),):
            assert torch.equal(u, v)
        assert torch.equal(f(good.view(torch.float32))[0], f(None)[0])


def test_weights_are_read_where_they_are_now(q):
    """Reassigned, moved, copied and saved weights give the same products; on the CPU they are refused."""
    import copy
    import io
    t = make(1, 200, 256, 64, True, torch.float16, 5)
    x = torch.randn((300, 256), generator=rng(6)).half().cuda()
    w = pack(q, t)
    ref = q.q4g_matmul(w, x)
    old = w.data
    w.data = old.clone()
    old.zero_()
    assert torch.equal(q.q4g_matmul(w, x), ref) and torch.equal(q.q4g_matmul(w, x[:1]), q.q4g_matmul(pack(q, t), x[:1]))
    kept = w.data
    w.data.data = kept.clone()  # the storage under the same tensor
    assert torch.equal(q.q4g_matmul(w, x), ref) and torch.equal(q.q4g_dequantize(w).double().cpu(), t[3])
    c = copy.deepcopy(w)
    w.data.zero_()
    assert torch.equal(q.q4g_matmul(c, x), ref)
    f = io.BytesIO()
    torch.save(c, f)
    f.seek(0)
    c = torch.load(f, weights_only=False, map_location="cpu")
    for call in (lambda: q.q4g_matmul(c, x), lambda: q.q4g_dequantize(c), lambda: q.q4g_matmul_workspace(c, torch.float16, 9)):
        with pytest.raises(ValueError):
            call()
    c.data = c.data.cuda()
    assert torch.equal(q.q4g_matmul(c, x), ref)
    c.data.resize_(16)  # no longer whole
    with pytest.raises(ValueError):
        q.q4g_matmul(c, x)


# ------------------------------------------------------------------ magnitudes
# Tolerances: those of test_q4g.py (u |y| + 1e-5 T, and 2^-11 T for weights that the GEMM rounds),
# and 2^-140 for f32 sums of results near the end of the f32 range: 2^11 times the smallest f32 number,
# which is the unit of the row kernel's sums for results that are below 2^-115.

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def near(y, ref, T, dt, gemm):
    tol = U[dt] * ref.abs() + 1e-5 * T + (2.0 ** -11 * T if gemm and dt != torch.float32 else 0) + 2.0 ** -138
    y = y.double().cpu()
    bad = ~((y - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first {y[bad][:3]} for {ref[bad][:3]}"


# the scales' magnitude, the activations'
MAGNITUDES = [(1e-5, 1e37), (1e-6, 3e37), (1e-2, 1e35), (1e-25, 1e-10), (1e-20, 1e3), (1e20, 1e-30), (1e3, 1e-30)]


@pytest.mark.parametrize("scale,xs", MAGNITUDES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("G", [32, 128])
def test_magnitudes_of_few_rows(q, scale, xs, dt, G):
    """Every way through the row kernel: dense, by slot, by token, by expert."""
    E, k, K, N = 4, 2, 256, 96
    t = make(E, N, K, G, True, torch.bfloat16, 21, scale)
    x = (xs * torch.randn((20, k, K), generator=rng(22)).clamp(-3, 3)).to(dt)
    xd = x.double()
    w1 = pack(q, tuple(v if v is None else v[:1] for v in t))
    for M in (1, 2, 9):
        near(q.q4g_matmul(w1, x[:M, 0].cuda()), xd[:M, 0] @ t[3][0].T, xd[:M, 0].abs() @ t[3][0].abs().T, dt, False)
    w = pack(q, t)
    for T in (1, 16, 20):  # 40 slots of four experts: the GEMM in bf16
        r = q.moe_route(torch.randn((T, E), generator=rng(23)).cuda(), k)
        W = t[3][r.ids.long().cpu()]
        wt = r.weights.double().cpu()[..., None]
        ref, A = (wt * (W @ xd[:T, :, :, None])[..., 0]).sum(1), (wt * (W.abs() @ xd[:T, :, :, None].abs())[..., 0]).sum(1)
        near(q.moe_down(w, x[:T].cuda(), r), ref, A, dt, T == 20)


SMALL_AND_LARGE = MAGNITUDES + [(1e-25, 1e-13), (1e-25, 1e-14), (1e-30, 1e-7), (1e-12, 1e-25), (1e30, 1e5), (1e37, 1e-3)]


@pytest.mark.parametrize("scale,xs", SMALL_AND_LARGE)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_magnitudes_of_many_rows(q, scale, xs, dt):
    """The GEMM, dense and by expert: results down to the end of the f32 range."""
    E, k, K, N, T = 3, 2, 256, 1000, 700
    t = make(E, N, K, 64, True, torch.bfloat16, 24, scale)
    x = (xs * torch.randn((T, k, K), generator=rng(25)).clamp(-3, 3)).to(dt)
    xd = x.double()
    w1 = pack(q, tuple(v if v is None else v[:1] for v in t))
    near(q.q4g_matmul(w1, x[:, 0].contiguous().cuda()), xd[:, 0] @ t[3][0].T, xd[:, 0].abs() @ t[3][0].abs().T, dt, True)
    r = q.moe_route(torch.randn((T, E), generator=rng(26)).cuda(), k)
    ids, wt = r.ids.long().cpu(), r.weights.double().cpu()
    ref, A = torch.zeros((T, N), dtype=torch.float64), torch.zeros((T, N), dtype=torch.float64)
    for e in range(E):
        a, j = torch.nonzero(ids == e, as_tuple=True)
        ref.index_add_(0, a, wt[a, j, None] * (xd[a, j] @ t[3][e].T))
        A.index_add_(0, a, wt[a, j, None] * (xd[a, j].abs() @ t[3][e].abs().T))
    near(q.moe_down(pack(q, t), x.cuda(), r), ref, A, dt, True)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_large_rows_of_weights_and_activations_that_do_not_meet(q, dt):
    """Weights of 1e25 and activations of 1e25, where each is zero beside the other: the results are exactly zero."""
    N, K, T = 600, 256, 500
    codes, s, z, _ = make(1, N, K, 64, True, torch.bfloat16, 27, 1e25)
    codes[..., :64] = 0x55  # the first 128 weights of a row are 5 - 5
    z[..., :2] = 5
    x = torch.zeros((T, K))
    x[:, :128] = 1e25 * torch.randn((T, 128), generator=rng(28)).clamp(-3, 3)
    for M in (2, T):
        assert bool((q.q4g_matmul(pack(q, (codes, s, z, None)), x[:M].to(dt).cuda()) == 0).all())
    w = pack(q, (codes, s, z, None), gate_up=True)
    for M in (2, T):
        r = q.moe_route(torch.zeros((M, 1)).cuda(), 1)
        assert bool((q.moe_gate_up(w, x[:M].to(dt).cuda(), r) == 0).all())


def test_route_refuses_numbers_that_do_not_fit(q):
    """Integers past 32 bits are not cut to fewer, and no memory is asked for a routing that is refused."""
    l = torch.zeros((5, 8), device="cuda")
    many = torch.zeros((1 << 20, 8), device="cuda")
    for call in (lambda: q.moe_route(l, (1 << 32) + 2), lambda: q.moe_route(l, 2, groups=(1 << 32) + 1), lambda: q.moe_route(l, 2, groups=2, top_groups=(1 << 32) + 1),
                 lambda: q.moe_route(l, -(1 << 32) + 2), lambda: q.moe_route(l, 0), lambda: q.moe_route(l, 9), lambda: q.moe_route(many, 1 << 21),
                 lambda: q.moe_route(torch.zeros((5, 513), device="cuda"), 2), lambda: q.moe_route(l[:, :0], 1)):
        with pytest.raises(q.QmmError) as e:
            call()
        assert e.value.status == 2
    with pytest.raises(RuntimeError):  # a tensor that is neither true nor false
        q.moe_route(l, 2, order=torch.zeros(2))
    with pytest.raises(RuntimeError):
        q.moe_route(l, 2, renorm=torch.zeros(2))
    assert torch.equal(q.moe_route(l, 2).ids.cpu(), torch.tensor([[0, 1]] * 5, dtype=torch.int32))


def test_a_route_can_be_saved(q, tmp_path):
    """With and without the sorted slots, as a tuple and in parts."""
    l = torch.randn((37, 16), generator=rng(60)).cuda()
    for order in (True, False):
        r = q.moe_route(l, 3, order=order)
        torch.save(tuple(r), tmp_path / "r.pt")
        for a, b in zip(torch.load(tmp_path / "r.pt"), r):
            assert b is None and a is None or torch.equal(a, b)
        torch.save({"route": r._asdict()}, tmp_path / "r.pt")
        assert torch.equal(torch.load(tmp_path / "r.pt")["route"]["weights"], r.weights)


# ------------------------------------------------------------------ sizes at which a kernel takes another way


@pytest.mark.parametrize("M", [9, 10, 11, 12])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_nine_to_twelve_rows_round_no_weight(q, dt, M):
    """Over a matrix that takes the row kernel one pass (where it would take two, as of 5000 x 4096, the GEMM is used)."""
    N, K = 9000, 2048
    t = make(1, N, K, 64, True, torch.float16, 31)
    x = torch.randn((M, K), generator=rng(32)).to(dt)
    y = q.q4g_matmul(pack(q, t), x.cuda()).double().cpu()
    ref, T = x.double() @ t[3][0].T, x.double().abs() @ t[3][0].abs().T
    u = 2.0 ** -11 if dt == torch.float16 else 2.0 ** -8
    assert bool(((y - ref).abs() <= u * ref.abs() + 1e-5 * T).all())


@pytest.mark.parametrize("dt,top_k", [("f32", 8), ("f32", 32), ("f16", 7), ("f16", 17), ("f16", 32), ("bf16", 31), ("bf16", 32)])
@pytest.mark.parametrize("T", [1, 4])
def test_down_of_a_token_with_many_experts(q, dt, top_k, T):
    """A token's experts end to end (f32: as far as their activations fit)."""
    E, K, N = 40, 96 if dt == "f32" else 352, 75
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt]
    t = make(E, N, K, 32, True, torch.float16, 33)
    h = torch.randn((T, top_k, K), generator=rng(34)).to(dt)
    r = q.moe_route(torch.randn((T, E), generator=rng(35)).cuda(), top_k)
    y = q.moe_down(pack(q, t), h.cuda(), r).double().cpu()
    W, wt = t[3][r.ids.long().cpu()], r.weights.double().cpu()[..., None]
    ref, A = (wt * (W @ h.double()[..., None])[..., 0]).sum(1), (wt * (W.abs() @ h.double().abs()[..., None])[..., 0]).sum(1)
    u = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    assert bool(((y - ref).abs() <= u * ref.abs() + 1e-5 * A).all())


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32])
def test_pairs_with_more_units_than_are_looked_up(q, dt):
    """More than 64 units a pair of blocks: later ones are looked up when they are taken."""
    M, N, K = 40000, 9000, 32
    t = make(1, N, K, 32, True, torch.float16, 36)
    x = torch.randn((M, K), generator=rng(37)).to(dt).cuda()
    y = q.q4g_matmul(pack(q, t), x)
    W = t[3][0].cuda()
    u = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    for m in range(0, M, 4000):
        xd = x[m:m + 4000].double()
        ref, T = xd @ W.T, xd.abs() @ W.abs().T
        assert bool(((y[m:m + 4000].double() - ref).abs() <= u * ref.abs() + (1e-5 + (0 if dt == torch.float32 else 2.0 ** -11)) * T).all())
    assert q.last_device_error() == 0


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32])
def test_experts_with_more_units_than_are_looked_up(q, dt):
    """The same for gate_up and down, with experts of very different numbers of rows, one without any."""
    T, E, K, F = 40000, 5, 32, 4100
    g = rng(38)
    pick = torch.tensor([0] * 5 + [1] * 3 + [2] + [4])[torch.randint(0, 10, (T,), generator=g)]
    logits = torch.zeros((T, E)).scatter_(1, pick[:, None], 4.0).cuda()
    r = q.moe_route(logits, 1)
    assert torch.equal(r.ids[:, 0].cpu().long(), pick)
    x = torch.randn((T, K), generator=g).to(dt).cuda()
    u = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    w = 1e-5 + (0 if dt == torch.float32 else 2.0 ** -11)
    t = make(E, 2 * F, K, 32, True, torch.float16, 39)
    h = q.moe_gate_up(pack(q, t, True), x, r)
    d = q.moe_down(pack(q, t), x[:, None], r)
    for m in range(0, T, 4000):
        e = pick[m:m + 4000]
        y, A = torch.empty((len(e), 2 * F), dtype=torch.float64, device="cuda"), torch.empty((len(e), 2 * F), dtype=torch.float64, device="cuda")
        for i in range(E):
            at, W = (e == i).nonzero()[:, 0].cuda(), t[3][i].cuda()
            y[at], A[at] = x[m + at].double() @ W.T, x[m + at].double().abs() @ W.abs().T
        assert bool(((d[m:m + 4000].double() - y).abs() <= u * y.abs() + w * A).all())
        eg, eu, gate, up = w * A[:, :F], w * A[:, F:], y[:, :F], y[:, F:]
        s = gate * torch.sigmoid(gate)
        tol = 1.1 * up.abs() * eg + s.abs() * eu + 1.1 * eg * eu + (u + 1e-6) * (s * up).abs() + 2.0 ** -24
        assert bool(((h[m:m + 4000, 0].double() - s * up).abs() <= tol).all())
    assert q.last_device_error() == 0

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

"""8-bit channel-scaled products and the quantizer that feeds them against
plain implementations: integer sums in 64 bits, then the f32 steps that the
header states, each rounded.  There is nothing to tolerate: codes, scales and
results are equal bit for bit, on every kernel."""
import numpy as np
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


def rng(seed):
    return torch.Generator().manual_seed(seed)


def plain_codes(x):
    """Codes (int64) and scales (f32) of the rows of x, in f32 steps."""
    v = x.float().numpy()
    with np.errstate(all="ignore"):
        top = np.abs(v).max(1, initial=0)
        d = (top / np.float32(127)).astype(np.float32)
        inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
        p = (v * inv[:, None]).astype(np.float32)
        c = np.trunc(p)
        c = c + np.where(np.abs(p - c) >= np.float32(0.5), np.sign(p), 0)
        c = np.clip(np.where(np.isnan(c), 0, c), -127, 127).astype(np.int64)
    bad = ~np.isfinite(v).all(1)
    c[bad] = 0
    d[bad] = np.nan
    return c, d


def plain_product(codes, sx, w, sw, bias, dt):
    """y from int64 codes: exact sums, then (sum sw) sx + bias in f32 steps."""
    total = (codes.astype(np.float64) @ w.astype(np.float64).T)  # integers below 2^53: exact
    with np.errstate(all="ignore"):
        y = total.astype(np.float32) * sw[None] * sx[:, None] + (np.float32(0) if bias is None else bias[None])
    return torch.from_numpy(y.astype(np.float32)).to(DT[dt])


def weights(q, N, K, seed=3, spread=30.0):
    g = rng(seed)
    codes = torch.clamp(torch.round(spread * torch.randn((N, K), generator=g)), -128, 127).to(torch.int8)
    scales = 0.001 * (0.5 + torch.rand(N, generator=g))
    return codes, scales, q.q8c_pack(codes.cuda(), scales.cuda())


def same(a, b):
    a, b = a.cpu(), b.cpu()
    assert a.dtype == b.dtype and a.shape == b.shape
    ok = (a == b) | (torch.isnan(a) & torch.isnan(b))
    assert ok.all(), f"{int((~ok).sum())} of {ok.numel()} differ, first at {torch.nonzero(~ok)[0].tolist()}: {a[~ok][:3]} for {b[~ok][:3]}"


# ------------------------------------------------------------------ layout and quantizer


@pytest.mark.parametrize("N,K", [(1, 1), (1, 16), (17, 127), (16, 128), (40, 129), (33, 576), (5, 1000)])
def test_pack_keeps_every_weight(q, N, K):
    codes, scales, w = weights(q, N, K)
    assert torch.equal(q.q8c_dequantize(w).cpu(), codes.float() * scales[:, None])
    wide = torch.zeros((N, K + 5), dtype=torch.int8, device="cuda")
    wide[:, 3:3 + K] = codes.cuda()
    again = q.q8c_pack(wide[:, 3:3 + K], scales.cuda().reshape(N, 1))
    assert torch.equal(again.data[:w.data.numel() - 12], w.data[:w.data.numel() - 12])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,K", [(1, 1), (3, 8), (2, 77), (5, 576), (1, 4096), (4, 9001), (1, 131071), (600, 64)])
def test_quantize(q, M, K, dt):
    x = torch.randn((M, K), generator=rng(K)).to(DT[dt])
    if M > 2:
        x[1] = 0
        x[2] = torch.round(x[2] * 4) / 2  # ties
    r = q.q8c_quantize(x.cuda())
    c, d = plain_codes(x)
    assert np.array_equal(r.codes.cpu().numpy(), c) and np.array_equal(r.scales.cpu().numpy(), d)


@pytest.mark.parametrize("dt", list(DT))
def test_quantize_special_rows(q, dt):
    x = torch.randn((9, 200), generator=rng(5))
    x[0] = 0
    x[1, 3], x[2, 100], x[3, 199] = float("nan"), float("inf"), -float("inf")
    x[4] *= 1e-38
    x[5] = 0
    x[5, 7] = 1e-45  # the scale is 0 in f32
    x[6] *= 1e37 if dt != "f16" else 1e4
    x[7, 9], x[7, 10] = -0.0, -127.0
    x[8] = 3.0
    x = x.to(DT[dt])
    r = q.q8c_quantize(x.cuda())
    c, d = plain_codes(x)
    assert np.array_equal(r.codes.cpu().numpy(), c) and np.array_equal(r.scales.cpu().numpy(), d, equal_nan=True)


# ------------------------------------------------------------------ products

SIZES = [
    # the row kernel: one row, a few, more than a pass holds; rows of any length
    (1, 1, 1), (1, 16, 16), (1, 576, 576), (1, 17, 100), (2, 40, 129), (3, 100, 1536), (7, 33, 160), (8, 192, 576), (9, 48, 128), (16, 300, 1024), (17, 50, 333),
    (31, 70, 192), (33, 64, 576), (100, 40, 64), (1, 96, 16384), (5, 40, 14336), (16, 24, 14336), (1, 9000, 128), (3, 20, 100000), (1, 5000, 4095), (40, 333, 200),
    # the GEMM: single blocks and pairs, K slices, a last tile of few rows, N and K past a tile's end
    (17, 4100, 4096), (37, 4096, 1536), (129, 2570, 640), (257, 3000, 1536), (300, 1290, 1601), (600, 640, 1000), (1000, 700, 1088), (1100, 500, 2048), (64, 9000, 576),
    (200, 1030, 4160), (33, 400, 14336), (530, 2000, 256), (40, 6000, 777), (193, 4000, 320), (2100, 1000, 128)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(q, M, N, K):
    codes, scales, w = weights(q, N, K)
    dt = ("f32", "f16", "bf16")[(M + N + K) % 3]
    x = torch.randn((M, K), generator=rng(M)).to(DT[dt])
    if M > 2:
        x[1] = 0
        x[2] *= 100
    bias = torch.randn(N, generator=rng(9)) if N % 2 else None
    c, d = plain_codes(x)
    ref = plain_product(c, d, codes.numpy(), scales.numpy(), None if bias is None else bias.numpy(), dt)
    b = None if bias is None else bias.cuda()
    y = q.q8c_matmul(w, x.cuda(), bias=b)
    same(y, ref)
    same(q.q8c_matmul(w, q.q8c_quantize(x.cuda()), bias=b, dtype=DT[dt]), ref)
    assert q.last_device_error() == 0


@pytest.mark.parametrize("xdt", list(DT))
@pytest.mark.parametrize("ydt", list(DT))
@pytest.mark.parametrize("M", [3, 300])
def test_matmul_types(q, M, xdt, ydt):
    N, K = 1300, 576
    codes, scales, w = weights(q, N, K)
    x = torch.randn((M, K), generator=rng(M)).to(DT[xdt])
    c, d = plain_codes(x)
    y = q.q8c_matmul(w, x.cuda(), dtype=DT[ydt])
    same(y, plain_product(c, d, codes.numpy(), scales.numpy(), None, ydt))


@pytest.mark.parametrize("M,N,K", [(3, 128, 640), (40, 1300, 576), (300, 2052, 1024), (33, 400, 8192), (40, 1302, 576)])
@pytest.mark.parametrize("dt", list(DT))
def test_bias(q, M, N, K, dt):
    """The bias is added to the rounded product: no contraction."""
    codes, scales, w = weights(q, N, K)
    x = torch.randn((M, K), generator=rng(M)).to(DT[dt])
    bias = torch.randn(N, generator=rng(9))
    c, d = plain_codes(x)
    same(q.q8c_matmul(w, x.cuda(), bias=bias.cuda()), plain_product(c, d, codes.numpy(), scales.numpy(), bias.numpy(), dt))


@pytest.mark.parametrize("M,K", [(4, 20736), (3, 28672), (4, 32768), (2, 32768), (1, 100000)])
def test_few_long_rows_of_codes(q, M, K):
    """Rows whose codes fill most of a block's shared memory; up to 32768 K they need no workspace, as the header says."""
    N = 40
    codes, scales, w = weights(q, N, K, spread=12.0)
    rows = torch.randint(-127, 128, (M, K), generator=rng(M)).to(torch.int8)
    sx = 0.5 + torch.rand(M, generator=rng(5))
    ref = plain_product(rows.numpy().astype(np.int64), sx.numpy(), codes.numpy(), scales.numpy(), None, "f32")
    x = q.Rows8(rows.cuda(), sx.cuda())
    same(q.q8c_matmul(w, x), ref)
    if K <= 32768:
        same(q.q8c_matmul(w, x, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")), ref)


def test_offsets_past_32_bits(q):
    """Results and activations of more than 2^31 elements: rows of the end and around the boundary against calls of their own."""
    N, K, M = 2048, 64, 1100000
    _, _, w = weights(q, N, K)
    x = torch.randn((M, K), generator=rng(2)).half().cuda()
    y = q.q8c_matmul(w, x)
    edge = 2 ** 31 // N
    for m in (0, edge - 4, edge, M - 8):
        assert torch.equal(y[m:m + 8], q.q8c_matmul(w, x[m:m + 8]))
    far = torch.empty((70, 1 << 25), dtype=torch.float16, device="cuda")[:, :K]  # rows 2^25 elements apart
    far.copy_(x[:70])
    assert torch.equal(q.q8c_matmul(w, far), y[:70]) and torch.equal(q.q8c_matmul(w, far[-4:]), y[66:70])
    r = q.q8c_quantize(far)
    assert torch.equal(q.q8c_matmul(w, r, dtype=torch.float16), y[:70])


def test_a_row_does_not_depend_on_the_others(q):
    N, K = 2000, 1536
    _, _, w = weights(q, N, K)
    x = torch.randn((700, K), generator=rng(1)).bfloat16().cuda()
    y = q.q8c_matmul(w, x)
    for m in (1, 5, 16, 17, 40, 130, 300):
        assert torch.equal(q.q8c_matmul(w, x[700 - m:]), y[700 - m:])


@pytest.mark.parametrize("M,K", [(1, 16384), (16, 4096), (40, 2048), (70, 14336), (300, 14336), (300, 1024), (513, 2500)])
def test_largest_sums(q, M, K):
    """Codes at the ends of their range and of one sign: sums far past 2^24, on each kernel, in rows beside ordinary ones."""
    N = 1300
    g = rng(2)
    codes = torch.randint(-128, 128, (N, K), generator=g).to(torch.int8)
    codes[0], codes[1], codes[2], codes[-1] = 127, -128, 126, -128
    scales = torch.full((N,), 2.0 ** -20)
    w = q.q8c_pack(codes.cuda(), scales.cuda())
    rows = torch.randint(-128, 128, (M, K), generator=g).to(torch.int8)
    rows[0] = -128
    if M > 5:
        rows[1], rows[2], rows[5] = 127, -127, -128
        rows[3] = 127 * (1 - 2 * (torch.arange(K) % 2))
        rows[4, :K // 2], rows[4, K // 2:] = 127, -127
    sx = 0.5 + torch.rand(M, generator=g)
    ref = plain_product(rows.numpy().astype(np.int64), sx.numpy(), codes.numpy(), scales.numpy(), None, "f32")
    same(q.q8c_matmul(w, q.Rows8(rows.cuda(), sx.cuda())), ref)
    assert q.last_device_error() == 0


@pytest.mark.parametrize("M", [2, 9, 300])
def test_bad_rows_stay_to_themselves(q, M):
    N, K = 1500, 192
    _, _, w = weights(q, N, K)
    x = torch.randn((M, K), generator=rng(2)).cuda()
    bad = x.clone()
    bad[0, 5] = float("nan")
    bad[-1, 7] = float("inf")
    y, z = q.q8c_matmul(w, x), q.q8c_matmul(w, bad)
    assert torch.isnan(z[0]).all() and torch.isnan(z[-1]).all()
    assert torch.equal(y[1:-1], z[1:-1])


@pytest.mark.parametrize("M", [3, 20, 300])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_rows_apart_and_canary(q, M, shift):
    N, K = 1900, 320
    _, _, w = weights(q, N, K)
    x = torch.randn((M, K), generator=rng(1)).half()
    wide = torch.full((M, K + 67 - 3 * (shift == 0)), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, shift:shift + K] = x.cuda()
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[:M * N].view(M, N)
    y = q.q8c_matmul(w, x.cuda())
    q.q8c_matmul(w, wide[:, shift:shift + K], out=out)
    assert torch.equal(out, y) and bool((buf[M * N:] == 7).all())
    r = q.q8c_quantize(wide[:, shift:shift + K])
    codes = torch.full((M, K + 35), 77, dtype=torch.int8, device="cuda")
    codes[:, shift:shift + K] = r.codes
    assert torch.equal(q.q8c_matmul(w, q.Rows8(codes[:, shift:shift + K], r.scales), dtype=torch.float16), y)


def test_overlapping_rows_are_refused(q):
    _, _, w = weights(q, 64, 128)
    x = torch.randn(1000, device="cuda").as_strided((4, 128), (64, 1))
    with pytest.raises(ValueError):
        q.q8c_matmul(w, x)


@pytest.mark.parametrize("M", [2, 400])
def test_in_a_graph_and_on_a_stream(q, M):
    _, _, w = weights(q, 2000, 256)
    x = torch.randn((M, 256), generator=rng(2)).cuda()
    y = q.q8c_matmul(w, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = q.q8c_matmul(w, x, stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = q.q8c_matmul(w, x)
    x.mul_(2.0)
    for _ in range(2):
        z.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, 2 * y)


@pytest.mark.parametrize("M,N,K", [(2, 2000, 4096), (4, 500, 9000), (40, 1000, 8192), (300, 2000, 1024)])
def test_calls_at_once(q, M, N, K):
    """On two streams, and a captured call replayed beside an eager one: each has a workspace of its own."""
    _, _, w = weights(q, N, K)
    xs = [torch.randn((M, K), generator=rng(i)).half().cuda() for i in range(3)]
    ref = [q.q8c_matmul(w, x) for x in xs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        z = q.q8c_matmul(w, xs[2])
    sides = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got += [(i, q.q8c_matmul(w, xs[i], stream=sides[i])) for i in range(2)]
        with torch.cuda.stream(sides[2]):
            z.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref[i]) for i, y in got) and torch.equal(z, ref[2])
    assert q.last_device_error() == 0


def test_empty(q):
    _, _, w = weights(q, 64, 128)
    assert q.q8c_matmul(w, torch.empty((0, 128), device="cuda")).shape == (0, 64)
    e = q.q8c_pack(torch.empty((0, 128), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    assert q.q8c_matmul(e, torch.ones((3, 128), device="cuda")).shape == (3, 0)
    r = q.q8c_quantize(torch.empty((0, 128), device="cuda"))
    assert r.codes.shape == (0, 128) and q.q8c_matmul(w, r).shape == (0, 64)
    assert q.q8c_quantize(torch.empty((0, 5), device="cuda")).codes.shape == (0, 5)


def test_workspace(q):
    _, _, w = weights(q, 2000, 1024)
    x = torch.randn((200, 1024), generator=rng(2)).cuda()
    n = q.q8c_matmul_workspace(w, 200)
    assert n > 0
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    y = q.q8c_matmul(w, x)
    assert torch.equal(q.q8c_matmul(w, x, workspace=ws[:n]), y) and bool((ws[n:] == 0xA5).all())
    with pytest.raises(q.QmmError) as e:
        q.q8c_matmul(w, x, workspace=ws[:n - 16])
    assert e.value.status == 5
    r = q.q8c_quantize(x)
    assert torch.equal(q.q8c_matmul(w, r, workspace=ws[:q.q8c_matmul_workspace(w, 200, True)]), y)


QMM_ERR_CUDA, QMM_ERR_TIMEOUT = 6, 7


@pytest.mark.parametrize("tiles", [0, 1, 5])
@pytest.mark.parametrize("M,N", [(1000, 4100), (70, 4100), (40, 9000)])
def test_injected_stall_times_out_and_recovers(q, M, N, tiles):
    _, _, w = weights(q, N, 4096)
    x = torch.randn((M, 4096), generator=rng(2)).cuda()
    ref = q.q8c_matmul(w, x)
    torch.cuda.synchronize()
    assert q.last_device_error() == 0
    q.test_set_wait_limit(22)
    try:
        q.test_inject("stall", 1, tiles)
        q.q8c_matmul(w, x)
        torch.cuda.synchronize()  # the call ends: every wait is bounded
        assert q.last_device_error() == QMM_ERR_TIMEOUT
    finally:
        q.test_inject("off")
        q.test_set_wait_limit(0)
    assert torch.equal(q.q8c_matmul(w, x), ref)
    assert q.last_device_error() == 0


@pytest.mark.parametrize("M", [2, 300])
def test_injected_launch_failure_touches_nothing(q, M):
    _, _, w = weights(q, 2000, 1024)
    x = torch.randn((M, 1024), generator=rng(2)).cuda()
    out = torch.full((M, 2000), 7.0, device="cuda")
    for f in (lambda: q.q8c_matmul(w, x, out=out), lambda: q.q8c_quantize(x), lambda: q.block_norm(x, x[0], out=out[:, :1024])):
        q.test_inject("launch_failure", 1)
        try:
            with pytest.raises(q.QmmError) as e:
                f()
            assert e.value.status == QMM_ERR_CUDA
        finally:
            q.test_inject("off")
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())

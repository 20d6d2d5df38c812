"""The norms around a block against the formula in 64 bits.

Tolerances, from the kernel's f32 steps, e = 2^-24.  A sum of K squares is at
most 32 additions in a thread and 10 among them, each off by e, so sqrt and the
reciprocal of (mean + eps) are off by at most 43 e / 2 + 4 e < 26 e; v takes
three more products (29 e), gate and scale two more: r' is off by 31 e |s g v|
+ e |r'|, delta below.  The second norm's root is off by 26 e and by what delta
does to the sum (|delta| / |r'| in the 2-norm), h = r' root w takes three more
roundings: |h| (29 e + |delta| / |r'|) + delta root |w|.  On top comes the one
rounding to the output's type."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
E = 2.0 ** -24


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    import gguf_block_quantized_qmatmul_gb300 as q
    return q


def make(T, K, dt, wdt, residual=True, post=True, gate="channel", seed=1):
    g = torch.Generator().manual_seed(seed)
    t = dict(y=torch.randn((T, K), generator=g).to(DT[dt]), weight=(1 + 0.3 * torch.randn(K, generator=g)).to(DT[wdt]))
    if residual:
        t["residual"] = (3 * torch.randn((T, K), generator=g)).to(DT[dt])
    if post:
        t["post_weight"] = (1 + 0.3 * torch.randn(K, generator=g)).to(DT[wdt])
    if gate != "none":
        t["gate"] = torch.rand((K,) if gate == "channel" else (T, K), generator=g).to(DT[dt])
    return t


def plain(t, scale, eps, offset):
    """r', h in 64 bits and how far the kernel's, unrounded, may be off."""
    d = {k: v.double() for k, v in t.items()}
    v = d["y"]
    if "post_weight" in d:
        v = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * (offset + d["post_weight"])
    a = scale * v * d.get("gate", 1.0)
    r = d.get("residual", 0.0) + a
    root = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    h = r * root * (offset + d["weight"])
    delta = 31 * E * a.abs() + E * r.abs()
    norm = r.norm(dim=1, keepdim=True)
    ratio = torch.where(norm > 0, delta.norm(dim=1, keepdim=True) / norm, torch.zeros_like(norm))
    return r, h, delta, h.abs() * (29 * E + ratio) + delta * root * (offset + d["weight"]).abs()


def near(got, ref, tol, dt):
    tol = tol + U[dt] * (ref.abs() + tol) + (2.0 ** -25 if dt == "f16" else 2.0 ** -149)
    bad = ~((got.double().cpu() - ref).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst at {torch.nonzero(bad)[0].tolist()}: {got.cpu()[bad][:3]} for {ref[bad][:3]}"


CASES = [
    # T, K, dt, wdt, residual, post, gate, scale, offset
    (1, 1, "f32", "f32", True, True, "channel", 1.0, 0.0), (1, 576, "f32", "f32", True, False, "none", 1.0, 0.0), (3, 7, "bf16", "f32", True, True, "token", 0.5, 1.0),
    (2, 100, "f16", "f16", False, True, "channel", 0.25, 0.0), (5, 255, "f32", "bf16", True, True, "none", 1.0, 1.0), (4, 256, "bf16", "bf16", False, False, "none", 1.0, 0.0),
    (2, 2048, "bf16", "bf16", True, True, "token", -1.5, 0.0), (2, 2049, "f16", "f32", True, True, "channel", 1.0, 0.0), (3, 4096, "f16", "f16", True, True, "channel", 0.7, 0.0),
    (2, 4100, "f32", "f32", True, True, "token", 1.0, 0.0), (2, 8192, "bf16", "f32", True, True, "channel", 1.0, 1.0), (2, 8200, "f32", "f16", True, True, "token", 0.3, 0.0),
    (1, 32768, "f16", "bf16", True, True, "channel", 1.0, 0.0), (2, 20001, "bf16", "bf16", True, False, "token", 1.0, 0.0), (1030, 64, "f32", "f32", True, True, "channel", 1.0, 0.0),
    (1100, 1000, "bf16", "bf16", True, True, "token", 0.5, 0.0), (1025, 1024, "f16", "f32", True, True, "none", 1.0, 0.0), (700, 576, "bf16", "f32", True, True, "channel", 1.0, 0.0)]


@pytest.mark.parametrize("T,K,dt,wdt,residual,post,gate,scale,offset", CASES)
def test_against_the_formula(q, T, K, dt, wdt, residual, post, gate, scale, offset):
    t = make(T, K, dt, wdt, residual, post, gate)
    if T > 2:
        t["y"][1] = 0
    r, h, dr, dh = plain(t, scale, 1e-5, offset)
    c = {k: v.cuda() for k, v in t.items()}
    gr, gh = q.block_norm(**c, scale=scale, eps=1e-5, weight_offset=offset)
    near(gr, r, dr, dt)
    near(gh, h, dh, dt)
    again = q.block_norm(**c, scale=scale, eps=1e-5, weight_offset=offset)
    assert torch.equal(gr, again[0]) and torch.equal(gh, again[1])
    # as codes: the same h, quantized
    cr, rows = q.block_norm(**c, scale=scale, eps=1e-5, weight_offset=offset, quantize=True)
    assert torch.equal(cr, gr)
    if dt == "f32":  # whose h is kept as it is
        ref = q.q8c_quantize(gh)
        assert torch.equal(rows.codes, ref.codes) and torch.equal(rows.scales, ref.scales)
    d = rows.scales.double().cpu()[:, None]
    top = h.abs().amax(1, keepdim=True)
    assert ((d - top / 127).abs() <= (dh.amax(1, keepdim=True) + E * top) / 127 + 2.0 ** -149).all()
    # a code is off by half a step, and by two roundings of a product of up to 127
    assert ((rows.codes.cpu().double() * d - h).abs() <= dh + d * (0.5 + 2 * 128 * E) + top * 2 * E).all()


def test_rows_apart_in_place_and_canary(q):
    T, K = 40, 600
    t = {k: v.cuda() for k, v in make(T, K, "bf16", "f32", gate="token").items()}
    r, h = q.block_norm(**t)
    for shift, extra in ((0, 8), (3, 5), (8, 16)):
        wide = {k: torch.full((T, K + extra + shift), 5.0, dtype=torch.bfloat16, device="cuda") for k in ("y", "residual", "gate", "out", "residual_out")}
        view = {k: v[:, shift:shift + K] for k, v in wide.items()}
        for k in ("y", "residual", "gate"):
            view[k].copy_(t[k])
        q.block_norm(**view, weight=t["weight"], post_weight=t["post_weight"])
        assert torch.equal(view["residual_out"], r) and torch.equal(view["out"], h)
        for k in ("out", "residual_out"):
            assert bool((wide[k][:, :shift] == 5).all()) and bool((wide[k][:, shift + K:] == 5).all())
    q.block_norm(**t, residual_out=t["residual"], out=t["y"])
    assert torch.equal(t["residual"], r) and torch.equal(t["y"], h)


@pytest.mark.parametrize("T,K", [(1, 577), (9, 577), (300, 1001), (5, 5001), (3, 14336), (7, 20001), (2, 28672), (400, 9)])
@pytest.mark.parametrize("dt", list(DT))
def test_in_place(q, T, K, dt):
    """r' and h where y and the residual were, rows that share words among them."""
    t = {k: v.cuda() for k, v in make(T, K, dt, "f32", gate="token").items()}
    r, h = q.block_norm(**t, scale=0.7)
    c = {k: v.clone() for k, v in t.items()}
    q.block_norm(**c, scale=0.7, residual_out=c["residual"], out=c["y"])
    assert torch.equal(c["residual"], r) and torch.equal(c["y"], h)
    c = {k: v.clone() for k, v in t.items()}
    q.block_norm(**c, scale=0.7, residual_out=c["y"], out=c["residual"])
    assert torch.equal(c["y"], r) and torch.equal(c["residual"], h)


def test_rows_that_are_not_finite(q):
    t = {k: v.cuda() for k, v in make(5, 300, "f32", "f32").items()}
    r, h = q.block_norm(**t)
    t["y"][1, 7] = float("nan")
    t["residual"][3, 2] = float("inf")
    r2, h2 = q.block_norm(**t)
    for i in (0, 2, 4):
        assert torch.equal(r[i], r2[i]) and torch.equal(h[i], h2[i])
    assert torch.isnan(r2[1]).all() and torch.isnan(h2[1]).all() and not torch.isfinite(h2[3, 2])
    rows = q.block_norm(**t, quantize=True)[1]
    assert torch.isnan(rows.scales[[1, 3]]).all() and not rows.codes[[1, 3]].any()


def test_zero_rows(q):
    t = {k: v.cuda() for k, v in make(3, 64, "f32", "f32", residual=False).items()}
    t["y"].zero_()
    r, h = q.block_norm(**t)
    assert not r.any() and not h.any()
    rows = q.block_norm(**t, quantize=True)[1]
    assert not rows.codes.any() and not rows.scales.any()


def test_stream_graph_and_empty(q):
    t = {k: v.cuda() for k, v in make(20, 640, "f16", "f16").items()}
    r, h = q.block_norm(**t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r2, h2 = q.block_norm(**t, stream=side)
    side.synchronize()
    assert torch.equal(r, r2) and torch.equal(h, h2)
    y = t["y"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r2, rows = q.block_norm(**t, quantize=True)
    ref = q.block_norm(**{**t, "y": y * 2}, quantize=True)
    t["y"].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r2, ref[0]) and torch.equal(rows.codes, ref[1].codes) and torch.equal(rows.scales, ref[1].scales)
    e = q.block_norm(t["y"][:0], t["weight"])
    assert e[0].shape == e[1].shape == (0, 640)


@pytest.mark.parametrize("K", [1, 31, 200, 256, 400, 577, 760, 1000, 2041, 4096, 5000, 9000])
@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f16")])
def test_a_row_does_not_depend_on_its_place(q, K, dt, wdt):
    """The same bits on every kernel: beside many rows or few, on any alignment, in any row."""
    T = max(700, 5000 // K)
    t = {k: v.cuda() for k, v in make(T, K, dt, wdt, gate="token").items()}
    r, h = q.block_norm(**t, scale=0.7)
    cr, rows = q.block_norm(**t, scale=0.7, quantize=True)
    assert torch.equal(cr, r)
    per_row = ("y", "residual", "gate")
    for first, n in ((0, 1), (3, 1), (T - 7, 7), (5, 300)):
        for extra, shift in ((0, 0), (8 - K % 8 + 8, 8), (3, 1)):
            some = dict(t)
            for k in per_row:
                wide = torch.full((n, K + extra), 3.0, dtype=DT[dt], device="cuda")
                some[k] = wide[:, shift:shift + K]
                some[k].copy_(t[k][first:first + n])
            if shift == 1:
                for k in ("weight", "post_weight"):
                    some[k] = torch.cat([t[k][:1], t[k]])[1:]
            a, b = q.block_norm(**some, scale=0.7)
            assert torch.equal(a, r[first:first + n]) and torch.equal(b, h[first:first + n])
            a, b = q.block_norm(**some, scale=0.7, quantize=True)
            assert torch.equal(a, r[first:first + n]) and torch.equal(b.codes, rows.codes[first:first + n]) and torch.equal(b.scales, rows.scales[first:first + n])


def test_offsets_past_32_bits(q):
    """More than 2^31 values, and rows far apart: rows around the boundary against calls of their own."""
    T, K = 530000, 4096
    y = torch.empty((T, K), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    w = torch.rand(K, device="cuda").bfloat16()
    r, h = q.block_norm(y, w, residual=y, post_weight=w)
    for t in (0, 2 ** 31 // K - 2, T - 4):
        a, b = q.block_norm(y[t:t + 4], w, residual=y[t:t + 4], post_weight=w)
        assert torch.equal(r[t:t + 4], a) and torch.equal(h[t:t + 4], b)
    del r, h
    far = y.view(-1).as_strided((60, 576), (1 << 25, 1))
    a, b = q.block_norm(far, w[:576])
    near = q.block_norm(far.clone(), w[:576])
    assert torch.equal(a, near[0]) and torch.equal(b, near[1])


def test_refusals(q):
    t = {k: v.cuda() for k, v in make(4, 64, "f16", "f32").items()}
    for bad in (dict(y=t["y"].float()), dict(y=t["y"][:3]), dict(weight=t["weight"][:63]), dict(post_weight=t["weight"].half()), dict(gate=t["gate"].float()),
                dict(gate=torch.ones((2, 64), dtype=torch.float16, device="cuda")), dict(residual=t["residual"].cpu()), dict(out=t["y"].float()),
                dict(residual_out=t["y"].t()), dict(out=t["y"], quantize=True), dict(y=t["y"].t())):
        with pytest.raises(ValueError):
            q.block_norm(**{**t, **bad})
    with pytest.raises(q.QmmError) as e:  # both results in one place
        q.block_norm(**t, out=t["y"], residual_out=t["y"])
    assert e.value.status == 2
    with pytest.raises(q.QmmError) as e:
        x = torch.zeros((1, 32769), device="cuda")
        q.block_norm(x, x[0])
    assert e.value.status == 2


def test_norm_and_product_together(q):
    """What a decoder runs between its attention and its projections: the 8-bit rows go straight into the product."""
    T, K, N = 45, 1536, 2000
    t = {k: v.cuda() for k, v in make(T, K, "bf16", "bf16").items()}
    g = torch.Generator().manual_seed(4)
    wq = q.q8c_quantize(torch.randn((N, K), generator=g).cuda())
    w = q.q8c_pack(*wq)
    r, rows = q.block_norm(**t, quantize=True)
    y = q.q8c_matmul(w, rows, dtype=torch.bfloat16)
    total = rows.codes.cpu().double() @ wq.codes.cpu().double().T
    ref = (total.float() * wq.scales.cpu() * rows.scales.cpu()[:, None]).bfloat16()
    assert torch.equal(y.cpu(), ref)


@pytest.mark.parametrize("T,K,dt,wdt,residual,post,gate", [
    (10000, 256, "bf16", "bf16", True, True, "channel"), (5001, 576, "f16", "f32", True, False, "token"), (20000, 136, "f32", "f32", False, True, "none"),
    (9000, 392, "bf16", "f32", True, True, "token"), (3000, 1000, "f16", "f16", True, True, "channel"), (2000, 1544, "bf16", "bf16", True, False, "none"),
    (1300, 2048, "f32", "f32", True, True, "token"), (700, 4096, "bf16", "bf16", True, True, "channel"), (650, 4096, "f32", "f32", False, True, "token"),
    (400, 6400, "f16", "f32", True, True, "none"), (350, 8192, "f32", "f32", True, True, "token"), (330, 8184, "bf16", "bf16", False, False, "channel"),
    (4000, 704, "f32", "bf16", True, True, "channel"), (2500, 1020, "bf16", "bf16", True, True, "channel")])
def test_many_rows(q, T, K, dt, wdt, residual, post, gate):
    """The kernels that take many rows: every row against the formula, in place and as codes too."""
    t = make(T, K, dt, wdt, residual, post, gate)
    r, h, dr, dh = plain(t, 0.7, 1e-5, 0.5)
    c = {k: v.cuda() for k, v in t.items()}
    gr, gh = q.block_norm(**c, scale=0.7, eps=1e-5, weight_offset=0.5)
    near(gr, r, dr, dt)
    near(gh, h, dh, dt)
    cr, rows = q.block_norm(**c, scale=0.7, eps=1e-5, weight_offset=0.5, quantize=True)
    assert torch.equal(cr, gr)
    if dt == "f32":
        ref = q.q8c_quantize(gh)
        assert torch.equal(rows.codes, ref.codes) and torch.equal(rows.scales, ref.scales)
    d = rows.scales.double().cpu()[:, None]
    assert ((rows.codes.cpu().double() * d - h).abs() <= dh + d * (0.5 + 2 * 128 * E) + h.abs().amax(1, keepdim=True) * 2 * E).all()
    if residual:
        c["y"][3, 5] = float("nan")
        q.block_norm(**c, scale=0.7, eps=1e-5, weight_offset=0.5, residual_out=c["residual"], out=c["y"])
        keep = torch.arange(T, device="cuda") != 3
        assert torch.equal(c["residual"][keep], gr[keep]) and torch.equal(c["y"][keep], gh[keep]) and torch.isnan(c["y"][3]).all()
    assert q.last_device_error() == 0

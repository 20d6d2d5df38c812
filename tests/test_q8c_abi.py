"""Argument errors and sizes of the 8-bit products and the norms (no GPU needed:
every call here returns before touching the device), and the weights' object."""
import copy
import ctypes
import pickle

import pytest

torch = pytest.importorskip("torch")

NULL, SHAPE, TYPE, ALIGN = 1, 2, 3, 4
P = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module")
def m():
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    from gguf_block_quantized_qmatmul_gb300 import q8c
    return q8c


@pytest.fixture(scope="module")
def lib(m):
    return m._lib()


def test_bytes(lib):
    # 16-row blocks of 128-K segments of 2048 bytes, a scale per row, the largest sum of squares
    assert lib.qmm_q8c_bytes(16, 128) == 2048 + 64 + 16
    assert lib.qmm_q8c_bytes(17, 129) == 2 * 2 * 2048 + 128 + 16
    assert lib.qmm_q8c_bytes(1, 1) == 2048 + 64 + 16
    assert lib.qmm_q8c_bytes(28672, 8192) == 1792 * 64 * 2048 + 4 * 28672 + 16
    for bad in ((0, 16), (16, 0), (-1, 16), (16, 1 << 17), ((1 << 23) + 1, 16)):
        assert lib.qmm_q8c_bytes(*bad) == 0


def test_pack_and_quantize_refusals(lib):
    ok = dict(codes=P, ldc=128, scales=P, N=16, K=128, out=P)

    def pack(**k):
        return lib.qmm_q8c_pack(*{**ok, **k}.values(), 0)
    assert pack(codes=0) == NULL and pack(scales=0) == NULL and pack(out=0) == NULL
    assert pack(ldc=127) == SHAPE and pack(K=0) == SHAPE and pack(N=-1) == SHAPE and pack(K=1 << 17, ldc=1 << 17) == SHAPE
    assert pack(out=P + 8) == ALIGN and pack(scales=P + 2) == ALIGN
    assert pack(N=0) == 0
    ok = dict(xtype=0, x=P, ldx=128, M=2, K=128, codes=P, ldc=128, scales=P)

    def quantize(**k):
        return lib.qmm_q8c_quantize(*{**ok, **k}.values(), 0)
    assert quantize(xtype=3) == TYPE and quantize(xtype=-1) == TYPE
    assert quantize(ldx=127) == SHAPE and quantize(ldc=127) == SHAPE and quantize(K=0) == SHAPE and quantize(M=-1) == SHAPE and quantize(M=1 << 31) == SHAPE
    assert quantize(x=0) == NULL and quantize(codes=0) == NULL and quantize(scales=0) == NULL
    assert quantize(x=P + 2) == ALIGN and quantize(scales=P + 2) == ALIGN
    assert quantize(M=0) == 0


def test_matmul_refusals(lib, m):
    def call(d=None, xt=1, x=P, ld=128, sx=0, M=2, bias=0, yt=1, y=P):
        d = m._Desc(P, 64, 128) if d is None else d
        return lib.qmm_q8c_matmul(ctypes.addressof(d), xt, x, ld, sx, M, bias, yt, y, 0, 0, 0)
    assert lib.qmm_q8c_matmul(0, 1, P, 128, 0, 2, 0, 1, P, 0, 0, 0) == NULL
    assert call(xt=3) == TYPE and call(yt=3) == TYPE and call(xt=9, sx=P, yt=-1) == TYPE
    assert call(ld=127) == SHAPE and call(M=-1) == SHAPE and call(M=1 << 31) == SHAPE and call(m._Desc(P, 64, 0)) == SHAPE
    assert call(x=0) == NULL and call(y=0) == NULL and call(m._Desc(0, 64, 128)) == NULL
    assert call(x=P + 1) == ALIGN and call(y=P + 1) == ALIGN and call(sx=P + 2) == ALIGN and call(bias=P + 1) == ALIGN and call(m._Desc(P + 8, 64, 128)) == ALIGN
    assert call(M=0) == 0 and call(m._Desc(P, 0, 128)) == 0


def test_norm_refusals(lib, m):
    def call(T=2, K=64, **k):
        a = dict(y=P, weight=P, h=P, ldy=64, ldr=64, ldg=64, ldro=64, ldh=64)
        a.update(k)
        n = m._Norm(**a)
        return lib.qmm_block_norm(ctypes.addressof(n), T, K, 0)
    assert lib.qmm_block_norm(0, 2, 64, 0) == NULL
    assert call(type=3) == TYPE and call(weight_type=-1) == TYPE
    assert call(T=-1) == SHAPE and call(K=0) == SHAPE and call(K=32769, ldy=32769, ldh=32769) == SHAPE and call(ldy=63) == SHAPE and call(ldh=63) == SHAPE
    assert call(residual=P, ldr=63) == SHAPE and call(gate=P, ldg=63) == SHAPE and call(residual_out=P, ldro=1) == SHAPE
    assert call(y=0) == NULL and call(weight=0) == NULL and call(h=0) == NULL and call(codes=P, scales=P) == NULL and call(h=0, codes=P) == NULL
    assert call(y=P + 2) == ALIGN and call(weight=P + 2) == ALIGN and call(residual=P + 1) == ALIGN and call(h=0, codes=P, scales=P + 2) == ALIGN
    assert call(T=0) == 0


def laid_out(m, N=40, K=192):
    return m.Q8CWeights(torch.randint(0, 256, (m._lib().qmm_q8c_bytes(N, K),), dtype=torch.uint8), N, K)


def test_weights_can_be_copied_and_saved(m, tmp_path):
    w = laid_out(m)
    for c in (copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert torch.equal(c.data, w.data) and (c.N, c.K) == (40, 192) and c.data.data_ptr() != w.data.data_ptr() and c._ptr != w._ptr
    torch.save(w, tmp_path / "w.pt")
    with torch.serialization.safe_globals([m.Q8CWeights]):
        assert torch.equal(torch.load(tmp_path / "w.pt", weights_only=True).data, w.data)


def test_weights_follow_their_data_and_refuse_other(m, monkeypatch):
    w = laid_out(m)
    n = w.data.numel()
    for bad in (torch.zeros(n - 1, dtype=torch.uint8), torch.zeros(n, dtype=torch.int8), torch.zeros((n, 2), dtype=torch.uint8)[:, 0], torch.zeros(n + 8, dtype=torch.uint8)[8:]):
        with pytest.raises(ValueError):
            w.data = bad
    with pytest.raises(ValueError):
        m.Q8CWeights(w.data, 40, 0)
    with pytest.raises(AttributeError):
        w.N = 3
    assert w.device == -1
    with pytest.raises(ValueError):
        m.q8c_dequantize(w)  # not on a GPU
    monkeypatch.setattr(m, "_need", lambda ok, text: None)  # the data is on the CPU here
    seen = lambda: m._Desc.from_address(w._descriptor()).data  # noqa: E731
    w.data = w.data.clone()
    assert seen() == w.data.data_ptr()

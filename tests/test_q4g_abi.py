"""Argument errors and sizes of the 4-bit group-scale and mixture-of-experts
entry points (no GPU needed: every call here returns before touching the device)."""
import ctypes

import pytest

NULL, SHAPE, TYPE, ALIGN, WORKSPACE = 1, 2, 3, 4, 5
P = 0x10000  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    import gguf_block_quantized_qmatmul_gb300 as q
    return q._lib()


@pytest.fixture(scope="module")
def m():
    from gguf_block_quantized_qmatmul_gb300 import q4g
    return q4g


def test_bytes(lib):
    # 16-row blocks of 128-K segments of 1024 + 64 (128 / group) bytes, and a power of two per row
    assert lib.qmm_q4g_bytes(1, 16, 128, 128, 0) == 1088 + 64
    assert lib.qmm_q4g_bytes(1, 17, 160, 32, 0) == 2 * 2 * 1280 + 128
    assert lib.qmm_q4g_bytes(3, 40, 256, 64, 1) == 3 * (3 * 2 * 1152 + 192)
    assert lib.qmm_q4g_bytes(1, 28672, 8192, 256, 0) == 1792 * 64 * 1088 + 4 * 28672
    for bad in ((0, 16, 128, 128, 0), (1, 16, 128, 48, 0), (1, 16, 160, 64, 0), (1, 17, 128, 64, 1), (1, 16, -128, 64, 0), (70000, 16, 128, 64, 0)):
        assert lib.qmm_q4g_bytes(*bad) == 0


def test_pack_refusals(lib):
    ok = [P, P, 1, P, 1, 16, 128, 64, 0, P, 0]

    def call(**k):
        a = list(ok)
        for i, v in k.items():
            a[int(i[1:])] = v
        return lib.qmm_q4g_pack(*a)
    assert call(_2=0) == TYPE and call(_2=3) == TYPE
    assert call(_7=48) == SHAPE and call(_6=96) == SHAPE and call(_4=0) == SHAPE and call(_5=17, _8=1) == SHAPE
    assert call(_0=0) == NULL and call(_1=0) == NULL and call(_9=0) == NULL
    assert call(_9=P + 8) == ALIGN and call(_1=P + 1) == ALIGN
    assert call(_5=0) == 0  # no rows
    assert lib.qmm_q4g_pack_q4_0(P, 1, 16, 48, 0, P, 0) == SHAPE
    assert lib.qmm_q4g_pack_q4_0(P + 2, 1, 16, 64, 0, P, 0) == ALIGN


def desc(m, **k):
    a = dict(data=P, experts=1, N=64, K=128, group=64, paired=0)
    a.update(k)
    return m._Desc(**a)


def test_matmul_refusals(lib, m):
    def call(d=None, xt=1, x=P, ld=128, M=2, y=P):
        d = desc(m) if d is None else d
        return lib.qmm_q4g_matmul(ctypes.addressof(d), xt, x, ld, M, y, 0, 0, 0)
    assert lib.qmm_q4g_matmul(0, 1, P, 128, 2, P, 0, 0, 0) == NULL
    assert call(xt=3) == TYPE
    assert call(ld=120) == SHAPE and call(M=-1) == SHAPE and call(M=1 << 31) == SHAPE
    assert call(desc(m, experts=2)) == SHAPE and call(desc(m, paired=1)) == SHAPE and call(desc(m, group=48)) == SHAPE and call(desc(m, K=96, group=64)) == SHAPE
    assert call(x=0) == NULL and call(y=0) == NULL and call(desc(m, data=0)) == NULL
    assert call(x=P + 8) == ALIGN and call(ld=132) == ALIGN and call(y=P + 1) == ALIGN and call(desc(m, data=P + 4)) == ALIGN
    assert call(M=0) == 0 and call(desc(m, N=0)) == 0


def test_route_refusals(lib, m):
    def call(type=0, ldl=64, T=4, E=64, logits=P, ids=P, weights=P, offsets=P, order=P, **k):
        c = dict(score=0, top_k=4, groups=1, top_groups=1, group_score=0, renorm=1, scale=1.0)
        c.update(k)
        cfg = m._RouteConfig(**c)
        return lib.qmm_moe_route(ctypes.addressof(cfg), type, logits, ldl, T, E, 0, ids, weights, offsets, order, 0, 0, 0)
    assert lib.qmm_moe_route(0, 0, P, 64, 4, 64, 0, P, P, P, P, 0, 0, 0) == NULL
    assert call(type=5) == TYPE and call(score=2) == TYPE and call(group_score=2) == TYPE
    assert call(ldl=63) == SHAPE and call(T=-1) == SHAPE and call(E=513, ldl=513) == SHAPE and call(E=0) == SHAPE
    assert call(top_k=0) == SHAPE and call(top_k=33) == SHAPE and call(top_k=65) == SHAPE
    assert call(groups=5) == SHAPE and call(groups=64) == SHAPE and call(groups=8, top_groups=0) == SHAPE and call(groups=8, top_groups=9) == SHAPE
    assert call(groups=32, top_groups=1, top_k=4) == SHAPE  # two experts a group
    assert call(logits=0) == NULL and call(ids=0) == NULL and call(weights=0) == NULL and call(order=0) == NULL and call(offsets=0) == NULL
    assert call(logits=P + 2) == ALIGN and call(ids=P + 2) == ALIGN
    assert call(T=1000) == WORKSPACE


def test_expert_refusals(lib, m):
    def call(f="qmm_moe_down", d=None, xt=1, x=P, ld=128, T=4, k=2, y=P, **r):
        d = desc(m, experts=8, paired=1 if f == "qmm_moe_gate_up" else 0) if d is None else d
        a = dict(ids=P, weights=P, offsets=P, order=P, T=T, top_k=k)
        a.update(r)
        ro = m._Routing(**a)
        return getattr(lib, f)(ctypes.addressof(d), xt, x, ld, ctypes.addressof(ro), y, 0, 0, 0)
    for f in ("qmm_moe_gate_up", "qmm_moe_down"):
        assert call(f, xt=-1) == TYPE
        assert call(f, k=0) == SHAPE and call(f, k=33) == SHAPE and call(f, T=-1) == SHAPE and call(f, ld=64) == SHAPE and call(f, T=1 << 30) == SHAPE
        assert call(f, desc(m, experts=600, paired=int(f == "qmm_moe_gate_up"))) == SHAPE
        assert call(f, x=0) == NULL and call(f, y=0) == NULL and call(f, ids=0) == NULL and call(f, order=0) == NULL and call(f, offsets=0) == NULL
        assert call(f, x=P + 8) == ALIGN and call(f, ids=P + 1) == ALIGN and call(f, ld=129) == ALIGN
        assert call(f, T=0) == 0
    assert call("qmm_moe_gate_up", desc(m, experts=8)) == SHAPE and call("qmm_moe_down", desc(m, experts=8, paired=1)) == SHAPE
    assert call("qmm_moe_down", weights=0) == NULL

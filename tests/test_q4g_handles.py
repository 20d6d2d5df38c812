"""The Python side of the 4-bit and expert calls without a GPU: which device
and stream a call is made on.  The library, torch's device and stream contexts
and CUDA tensors are stand-ins."""
import contextlib
import copy
import pickle

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    from gguf_block_quantized_qmatmul_gb300 import q4g
    return q4g


class OnDevice:
    """A CPU tensor that says that it is on CUDA device `index`."""
    is_cuda = True

    def __init__(self, t, index):
        self.t, self.index = t, index
        self.shape, self.dtype, self.device = t.shape, t.dtype, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index

    def unsqueeze(self, d):
        return OnDevice(self.t.unsqueeze(d), self.index)

    def contiguous(self):
        return OnDevice(self.t.contiguous(), self.index)


class FakeStream:
    def __init__(self, handle, device):
        self.cuda_stream = handle
        self.device = torch.device("cuda", device)


class World:
    """The current device, its streams, and what was called where."""

    def __init__(self):
        self.device, self.streams, self.calls = 0, {}, []

    @contextlib.contextmanager
    def on_device(self, index):
        was, self.device = self.device, index if index >= 0 else self.device
        yield
        self.device = was

    @contextlib.contextmanager
    def on_stream(self, s):
        was = self.device, dict(self.streams)
        self.device = s.device.index
        self.streams[self.device] = s.cuda_stream
        yield
        self.device, self.streams = was

    def __getattr__(self, name):  # an entry point of the library
        def call(*args):
            if name != "qmm_q4g_bytes":  # arithmetic, wherever it is made
                self.calls.append((name, self.device, args[-1]))
            return 4096 if name.endswith("bytes") or name.endswith("workspace") else 0
        return call

    def product(self, *args):  # one of the extension: it sets the tensors' device itself and takes its current stream
        self.calls.append(("product", self.device, self.streams.get(self.device, 0)))
        return OnDevice(torch.empty(0), 1)


@pytest.fixture
def world(m, monkeypatch):
    w = World()
    monkeypatch.setattr(m, "_lib", lambda: w)
    monkeypatch.setattr(m, "_raw_stream", lambda device: w.streams.get(device, 0))
    monkeypatch.setattr(m, "_binding", type("B", (), dict.fromkeys(("matmul", "gate_up", "down"), staticmethod(w.product)))())
    monkeypatch.setattr(m, "_laid_out", lambda E, N, K, group, gate_up, device: OnDevice(torch.empty(4096, dtype=torch.uint8), device.index))
    monkeypatch.setattr(torch.cuda, "device", w.on_device)
    monkeypatch.setattr(torch.cuda, "stream", w.on_stream)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle, w.device if device is None else device))
    return w


def packed(m, world, **kw):
    codes, scales = torch.zeros((32, 64), dtype=torch.uint8), torch.ones((32, 2), dtype=torch.float16)
    return m.q4g_pack(OnDevice(codes, 1), OnDevice(scales, 1), **kw)


def test_launches_are_made_on_the_tensors_device(m, world):
    w = packed(m, world)
    m.q4g_pack_q4_0(OnDevice(torch.zeros((32, 36), dtype=torch.uint8), 1), 64)
    m.q4g_dequantize(w, out=OnDevice(torch.empty((1, 32, 128)), 1))
    assert [c for c in world.calls if c[0] != "qmm_q4g_bytes"] == [("qmm_q4g_pack", 1, 0), ("qmm_q4g_pack_q4_0", 1, 0), ("qmm_q4g_dequantize", 1, 0)]
    assert world.device == 0


def test_a_workspace_is_sized_for_the_weights_device(m, world):
    w = packed(m, world)
    assert m.q4g_matmul_workspace(w, torch.float16, 100) == 4096
    assert world.calls[-1][:2] == ("qmm_q4g_matmul_workspace", 1)


@pytest.mark.parametrize("stream", [77, FakeStream(77, 1)])
def test_a_stream_is_one_of_the_tensors_device(m, world, stream):
    w = packed(m, world, stream=stream)
    assert world.calls[-1] == ("qmm_q4g_pack", 1, 77)
    m.q4g_dequantize(w, out=OnDevice(torch.empty((1, 32, 128)), 1), stream=stream)
    assert world.calls[-1] == ("qmm_q4g_dequantize", 1, 77)
    x = OnDevice(torch.zeros((2, 128), dtype=torch.float16), 1)
    r = m.Route(None, None)
    for f in (lambda: m.q4g_matmul(w, x, stream=stream), lambda: m.moe_gate_up(w, x, r, stream=stream), lambda: m.moe_down(w, x, r, stream=stream)):
        f()
        assert world.calls[-1] == ("product", 1, 77)
    assert world.device == 0 and world.streams == {}


def test_another_devices_stream_is_refused(m, world):
    w = packed(m, world)
    n = len(world.calls)
    for f in (lambda s: packed(m, world, stream=s), lambda s: m.q4g_dequantize(w, stream=s),
              lambda s: m.q4g_matmul(w, OnDevice(torch.zeros((2, 128)), 1), stream=s)):
        with pytest.raises(ValueError):
            f(FakeStream(5, 0))
    assert len(world.calls) == n


# ------------------------------------------------------------------ laid-out weights as an object


def laid_out(m, E=2, N=40, K=192, group=64, gate_up=True):
    n = m._lib().qmm_q4g_bytes(E, N, K, group, int(gate_up))
    return m.Q4GWeights(torch.randint(0, 256, (n,), dtype=torch.uint8), E, N, K, group, gate_up)


def same(a, b):
    return torch.equal(a.data, b.data) and all(getattr(a, f) == getattr(b, f) for f in ("experts", "N", "K", "group", "gate_up"))


def test_weights_can_be_copied_and_saved(m, tmp_path):
    w = laid_out(m)
    holder = torch.nn.Module()
    holder.w = w
    for c in (copy.deepcopy(w), pickle.loads(pickle.dumps(w)), copy.deepcopy(holder).w):
        assert same(c, w) and c.data.data_ptr() != w.data.data_ptr() and c._ptr != w._ptr
    assert copy.copy(w).data is w.data
    torch.save({"w": w}, tmp_path / "w.pt")
    assert same(torch.load(tmp_path / "w.pt", weights_only=False)["w"], w)
    with torch.serialization.safe_globals([m.Q4GWeights]):
        assert same(torch.load(tmp_path / "w.pt", weights_only=True)["w"], w)


def test_weights_follow_their_data(m, monkeypatch):
    """The descriptor that a call gets holds where the data is at that call."""
    w = laid_out(m)
    monkeypatch.setattr(m, "_need", lambda ok, text: None)  # the data is on the CPU here
    seen = lambda: m._Desc.from_address(w._descriptor()).data  # noqa: E731
    assert seen() == w.data.data_ptr()
    w.data = w.data.clone()
    assert seen() == w.data.data_ptr()
    other = w.data.clone()
    w.data.data = other  # as torch.nn.Module.to moves a parameter
    assert seen() == other.data_ptr()


def test_weights_refuse_other_data(m):
    w = laid_out(m)
    n = w.data.numel()
    for bad in (torch.zeros(n - 1, dtype=torch.uint8), torch.zeros(n + 1, dtype=torch.uint8), torch.zeros(n, dtype=torch.int8),
                torch.zeros((n, 2), dtype=torch.uint8)[:, 0], torch.zeros(n + 8, dtype=torch.uint8)[8:]):
        with pytest.raises(ValueError):
            w.data = bad
        with pytest.raises(ValueError):
            m.Q4GWeights(bad, 2, 40, 192, 64, True)
    with pytest.raises(ValueError):
        m.Q4GWeights(w.data, 2, 40, 192, 48, True)  # no such group
    for name in ("experts", "N", "K", "group", "gate_up", "device"):
        with pytest.raises(AttributeError):
            setattr(w, name, 1)
    assert w.device == -1
    with pytest.raises(ValueError):
        m.q4g_dequantize(w)  # not on a GPU

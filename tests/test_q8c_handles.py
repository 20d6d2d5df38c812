"""The Python side of the 8-bit calls without a GPU: which device and stream a
call is made on.  The library, torch's device and stream contexts and CUDA
tensors are stand-ins, those of test_q4g_handles.py."""
import pytest

torch = pytest.importorskip("torch")

from test_q4g_handles import FakeStream, OnDevice, World  # noqa: E402


@pytest.fixture(scope="module")
def modules():
    from gguf_block_quantized_qmatmul_gb300 import build
    build.build()
    from gguf_block_quantized_qmatmul_gb300 import q4g, q8c
    return q4g, q8c


class Tensor(OnDevice):
    def reshape(self, *a):
        return Tensor(self.t.reshape(*a), self.index)

    def float(self):
        return Tensor(self.t.float(), self.index)

    def contiguous(self):
        return Tensor(self.t.contiguous(), self.index)


@pytest.fixture
def world(modules, monkeypatch):
    q4g, m = modules
    w = World()
    product = staticmethod(w.product)
    for module in (q4g, m):
        monkeypatch.setattr(module, "_lib", lambda: w)
        monkeypatch.setattr(module, "_raw_stream", lambda device: w.streams.get(device, 0))
        monkeypatch.setattr(module, "_binding", type("B", (), dict.fromkeys(("matmul8", "norm", "layer"), product))())
    monkeypatch.setattr(torch.cuda, "device", w.on_device)
    monkeypatch.setattr(torch.cuda, "stream", w.on_stream)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle, w.device if device is None else device))
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, dtype=None, device=None: Tensor(real(*a, dtype=dtype), torch.device(device).index if device else 0))
    monkeypatch.setattr(Tensor, "__getitem__", lambda self, i: Tensor(self.t[i], self.index), raising=False)
    return w


def test_launches_are_made_on_the_tensors_device_and_stream(modules, world):
    q4g, m = modules
    codes, scales, x = Tensor(torch.zeros((32, 64), dtype=torch.int8), 1), Tensor(torch.ones(32), 1), Tensor(torch.zeros((2, 64)), 1)
    for stream, handle in ((None, 0), (77, 77), (FakeStream(77, 1), 77)):
        del world.calls[:]
        m.q8c_quantize(x, stream=stream)
        w = m.Q8CWeights.__new__(m.Q8CWeights)
        w._desc, w._bytes, w._data = m._Desc(0, 32, 64), 4096, Tensor(torch.zeros(4096, dtype=torch.uint8), 1)
        w._ptr = 1
        m.q8c_dequantize(w, out=Tensor(torch.zeros((32, 64)), 1), stream=stream)
        m.q8c_matmul(w, x, stream=stream)
        m.block_norm(x, scales, stream=stream)
        names = [c[0] for c in world.calls]
        assert names == ["qmm_q8c_quantize", "qmm_q8c_dequantize", "product", "product"]
        assert all(c[2] == handle for c in world.calls)
        assert all(c[1] == 1 for c in world.calls if c[0] != "product" or stream is not None)  # the extension sets the device itself
        assert world.device == 0 and world.streams == {}


def test_another_devices_stream_is_refused(modules, world):
    _, m = modules
    x = Tensor(torch.zeros((2, 64)), 1)
    for f in (lambda s: m.q8c_quantize(x, stream=s), lambda s: m.block_norm(x, x, stream=s)):
        with pytest.raises(ValueError):
            f(FakeStream(5, 0))
    assert not [c for c in world.calls if not c[0].endswith("bytes")]

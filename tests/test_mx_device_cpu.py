"""CPU: the binding of the microscaled operators launches on the tensors' GPU and its
current stream, whichever GPU is current, and leaves the current one as it was.

The tensors say that they lie on GPU 1; the library's functions are recorded, not
called."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import bit_quantized_amd as w4  # noqa: E402
from bit_quantized_amd import _lib  # noqa: E402


class Second(torch.Tensor):
    """A tensor of GPU 1, as far as the binding asks."""

    def get_device(self):
        return 1


def second(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Second)


@pytest.fixture(params=[0, 1], ids=["another_current", "same_current"])
def calls(request, monkeypatch):
    """(function, current GPU, stream) of each launch; GPU i's stream is 100 + i."""
    now, out = [request.param], []

    @contextlib.contextmanager
    def device(index):
        before, now[0] = now[0], index
        try:
            yield
        finally:
            now[0] = before

    def recorded(name):
        def call(*args):
            out.append((name, now[0], args[-1].value))
            return 0
        return call

    names = ["quant", "dequant", "pack_weights", "unpack_weights", "linear", "grouped_linear"]
    real = _lib.load()
    fake = types.SimpleNamespace(**{f"w4a8_mx_{n}": recorded(n) for n in names},
                                 **{f"w4a8_mx_{n}": getattr(real, f"w4a8_mx_{n}") for n in
                                    ("weight_bytes", "linear_workspace_bytes", "grouped_linear_workspace_bytes")})
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(_lib, "_gpus", 0, raising=False)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    yield out
    assert now[0] == request.param


def test_launches_are_on_the_tensors_gpu(calls):
    x = second(2, 64, dtype=torch.float32)
    t = w4.mx_quant(x)
    w4.mx_dequant(w4.MxTensor(second(2, 32), second(2, 2), "fp4"))
    w = w4.mx_pack_weights(second(32, 32), second(32, 2))
    w4.mx_unpack_weights(w)
    w4.mx_linear(x, w)
    w4.mx_grouped_linear(x, w4.MxWeight(w.buf, 2, 16, 64), second(3, dtype=torch.int32))
    assert t.format == "fp4"
    assert [c[0] for c in calls] == ["quant", "dequant", "pack_weights", "unpack_weights", "linear", "grouped_linear"]
    assert all(c[1:] == (1, 101) for c in calls), calls


def test_a_refusal_leaves_the_current_gpu(calls, monkeypatch):
    monkeypatch.setattr(_lib.load(), "w4a8_mx_quant", lambda *a: -1, raising=False)
    monkeypatch.setattr(_lib.load(), "w4a8_last_error", lambda: b"refused", raising=False)
    with pytest.raises(_lib.W4A8Error):
        w4.mx_quant(second(2, 64, dtype=torch.float32))

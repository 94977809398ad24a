"""Calls at the edges of what the operators take: which GPU they run on (with
stand-ins for tensors of several GPUs, on the CPU)."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu


class Tensor:
    """A contiguous tensor of GPU `device` as the binding sees it."""

    def __init__(self, shape, dtype=torch.bfloat16, device=1, strides=None):
        self.shape, self.dtype, self.number, self.is_cuda = torch.Size(shape), dtype, device, device >= 0
        self.device, self.requires_grad = device, False
        self.strides = strides or torch.empty(shape, device="meta").stride()

    def get_device(self):
        return self.number

    def stride(self, dim=None):
        return self.strides if dim is None else self.strides[dim]

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        pass


class Machine:
    """Two GPUs, of which `current` is current; calls are noted as (operator,
    current GPU, stream's handle)."""

    def __init__(self, stmat, current=0):
        self.current, self.calls = current, []
        names = ("BF16", "F16", "F32", "F8_E4M3", "F8_E5M2")
        self.codes = {stmat.torch_dtype(n): stmat.DTYPES.index(n) for n in names}
        self.dsts = {n: (stmat.torch_dtype(n), stmat.DTYPES.index(n)) for n in names}
        self.torch = types.SimpleNamespace(
            float32=torch.float32, uint8=torch.uint8, bfloat16=torch.bfloat16, is_grad_enabled=lambda: True,
            cuda=types.SimpleNamespace(device=self.on, stream=lambda s: self.on(s.device_index), ExternalStream=Stream))
        for op in ("rms_norm", "gated_act", "linear"):
            setattr(self, op, lambda args, stream, op=op: self.calls.append((op, self.current, stream)) or 0)

    @contextlib.contextmanager
    def on(self, number):
        before, self.current = self.current, number
        try:
            yield
        finally:
            self.current = before

    def device(self):
        return self.current

    def stream(self, number):
        return 100 + number

    def empty(self, shape, dtype, device):
        return Tensor(tuple(shape) if not isinstance(shape, int) else (shape,), dtype, device)

    def empty_like(self, like, dtype):
        return Tensor(like.shape, dtype, like.device)


class Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device_index = handle, device


@pytest.fixture
def machine(stmat, monkeypatch):
    m = Machine(stmat)
    monkeypatch.setattr(stmat, "_OPS", m)
    return m


def test_a_call_runs_on_its_operands_gpu(stmat, machine):
    """Its kernels, outputs and stream belong to that GPU, whichever is
    current, and that one is current again afterwards."""
    x, w = Tensor((4, 16)), Tensor((8, 16))
    for current in (0, 1):
        machine.current = current
        for call in (lambda **k: stmat.rms_norm(x, dst="F8_E4M3", **k), lambda **k: stmat.gated_act(x, x, **k),
                     lambda **k: stmat.linear(x, w, **k)):
            for kw in ({}, {"stream": 101}, {"stream": Stream(101, 1)}):
                machine.calls.clear()
                got = call(**kw)
                assert [c[1:] for c in machine.calls] == [(1, 101)] and machine.current == current
                assert all(t is None or t.device == 1 for t in (got if isinstance(got, tuple) else (got,)))


def test_operands_of_several_gpus_are_refused(stmat, machine):
    def on(device, *shape, dtype=torch.bfloat16):
        return Tensor(shape, dtype, device)

    x, w, vec, one = on(1, 4, 16), on(1, 8, 16), on(1, 16), on(1, 1, dtype=torch.float32)
    for far in (0, -1):
        calls = [
            lambda **k: stmat.rms_norm(x, on(far, 16), **k), lambda **k: stmat.rms_norm(x, vec, residual=on(far, 4, 16), **k),
            lambda **k: stmat.rms_norm(x, vec, dst="F8_E4M3", scale=on(far, 1, dtype=torch.float32), **k),
            lambda **k: stmat.rms_norm(on(far, 4, 16), vec, **k) if far < 0 else stmat.rms_norm(on(far, 4, 16), vec),
            lambda **k: stmat.gated_act(x, on(far, 4, 16), **k),
            lambda **k: stmat.gated_act(x, x, dst="F8_E4M3", scale=on(far, 1, dtype=torch.float32), **k),
            lambda **k: stmat.linear(x, on(far, 8, 16), **k), lambda **k: stmat.linear(x, w, bias=on(far, 8), **k),
            lambda **k: stmat.linear(x, w, x_scale=on(far, 4, dtype=torch.float32), **k),
            lambda **k: stmat.linear(x, w, x_scale=one, w_scale=on(far, 1, dtype=torch.float32), **k),
            lambda **k: stmat.linear(x, w, residual=on(far, 4, 8), **k), lambda **k: stmat.linear(x, w, out=on(far, 4, 8), **k),
        ]
        for current in (0, 1):
            machine.current = current
            for i, call in enumerate(calls):
                for kw in ({}, {"stream": Stream(101, 1)}):
                    with pytest.raises(stmat.StmatError) as e:
                        call(**kw)
                    assert e.value.status == "ST_E_INVAL" and "GPU" in str(e.value), i
    assert machine.calls == []


def test_a_stream_of_another_gpu_is_refused(stmat, machine):
    x, w = Tensor((4, 16)), Tensor((8, 16))
    for call in (lambda s: stmat.rms_norm(x, stream=s), lambda s: stmat.gated_act(x, stream=s),
                 lambda s: stmat.linear(x, w, stream=s)):
        with pytest.raises(stmat.StmatError) as e:
            call(Stream(100, 0))
        assert e.value.status == "ST_E_INVAL" and "GPU" in str(e.value)
    assert machine.calls == []

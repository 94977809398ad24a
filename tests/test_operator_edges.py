"""Calls at the edges of what the operators take: which GPU they run on (with
stand-ins for tensors of several GPUs, on the CPU), operands that overlap."""
import contextlib
import ctypes as C
import random
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


# ------------------------------------------------------ overlapping operands

X, W, Y = 1 << 20, 2 << 20, 3 << 20


def linear_args(stmat, **kw):
    """A BF16 product of 8 tokens of 16 with a 16 x 16 weight."""
    a = stmat.LinearArgs(m=8, n=16, k=16, act=0, x_dtype=10, w_dtype=10, y_dtype=10, bias_dtype=10, x=X, ldx=16, w=W,
                         ldw=16, y=Y, ldy=16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


# y over x (all of it, its last row, from its middle, a strided one), over the
# weight, the vectors, and over a part of the residual.
OVERLAPS = [
    dict(y=X), dict(y=X + 7 * 32), dict(y=X - 7 * 32), dict(y=X + 16), dict(y=X, ldy=24), dict(y=X - 100 * 2, ldy=40),
    dict(y=X + 2, ldx=40, ldy=40), dict(y=X + 15 * 2, ldx=40, ldy=40), dict(y=X - 15 * 2, ldx=40, ldy=40),
    dict(y=X + 40 * 2 * 7 + 15 * 2, ldx=40, ldy=40), dict(y=X, m=1, ldy=0), dict(y=X, ldx=0), dict(y=X - 7 * 32, ldx=0),
    dict(y=W), dict(y=W + 15 * 32), dict(y=W, m=16), dict(y=W - 8 * 32 + 2), dict(y=W, w_dtype=13, x_dtype=13, y_dtype=11),
    dict(x_scale=Y, x_scale_count=1), dict(x_scale=Y + 252, x_scale_count=1), dict(w_scale=Y - 60, w_scale_count=16),
    dict(bias=Y + 128), dict(bias=Y - 30), dict(bias=Y + 16 * 2, ldy=20, n=18),
    dict(residual=Y + 2, ldr=16), dict(residual=Y, ldr=18), dict(residual=Y, ldr=0), dict(residual=Y - 32, ldr=16),
]
# Neighbours, columns of one buffer between one another, operands of length 0,
# and the residual itself.
APART = [
    dict(y=X + 8 * 32), dict(y=X - 8 * 32), dict(y=W + 16 * 32), dict(y=X + 32, ldx=32, ldy=32),
    dict(y=X + 16 * 2, ldx=40, ldy=40), dict(y=X + 24 * 2, ldx=40, ldy=40), dict(y=X - 16 * 2, ldx=40, ldy=40),
    dict(y=X + 32, ldx=32, ldy=64), dict(y=X, k=0), dict(y=X + 32, ldx=0), dict(bias=Y + 8 * 32), dict(bias=Y - 32),
    dict(bias=Y + 16 * 2, ldy=32), dict(x_scale=Y + 8 * 32, x_scale_count=8), dict(w_scale=Y - 64, w_scale_count=16),
    dict(residual=Y, ldr=16), dict(residual=Y, ldr=99, m=1), dict(residual=Y + 32, ldr=32, ldy=32),
]


@pytest.mark.parametrize("kw", OVERLAPS, ids=range(len(OVERLAPS)))
def test_linear_refuses_y_over_another_operand(stmat, kw):
    """Tiles that are written would change what other tiles still read.  (On
    the host, before anything is queued: the addresses are made up.)"""
    a, need = linear_args(stmat, **kw), C.c_uint64()
    for code in (stmat.lib().st_linear(C.byref(a), None), stmat.lib().st_linear_workspace(C.byref(a), C.byref(need))):
        assert stmat.STATUS[code] == "ST_E_INVAL"
        assert "overlaps" in stmat.lib().st_last_error().decode()


@pytest.mark.parametrize("kw", APART, ids=range(len(APART)))
def test_linear_takes_neighbours_and_the_residual(stmat, kw):
    need = C.c_uint64()
    assert stmat.STATUS[stmat.lib().st_linear_workspace(C.byref(linear_args(stmat, **kw)), C.byref(need))] == "ST_OK"


def test_linear_overlaps_against_every_byte(stmat):
    """Random placements of y and x against the sets of their bytes."""
    rng, need, seen = random.Random(3), C.c_uint64(), set()
    for _ in range(4000):
        m, n, k = rng.randint(1, 6), rng.randint(1, 9), rng.randint(1, 9)
        ldx, ldy = k + rng.choice([0, 0, 1, 5, 12]), n + rng.choice([0, 0, 1, 5, 12])
        if rng.random() < 0.3:
            ldx = ldy = max(ldx, ldy)
        y = X + 2 * rng.randint(-130, 130)
        got = stmat.lib().st_linear_workspace(C.byref(linear_args(stmat, m=m, n=n, k=k, ldx=ldx, ldw=k, y=y, ldy=ldy)),
                                              C.byref(need))
        meet = {X + 2 * (i * ldx + j) for i in range(m) for j in range(k)} & {
            y + 2 * (i * ldy + j) for i in range(m) for j in range(n)}
        assert stmat.STATUS[got] == ("ST_E_INVAL" if meet else "ST_OK"), (m, n, k, ldx, ldy, y - X)
        seen.add(bool(meet))
    assert seen == {True, False}


def test_linear_refuses_a_workspace_over_an_operand(stmat):
    base = dict(ldx=17, ldw=17, ldy=16, residual=4 << 20, ldr=16)
    a, need = linear_args(stmat, **base), C.c_uint64()
    stmat._check(stmat.lib().st_linear_workspace(C.byref(a), C.byref(need)))
    for at in (X, X + 256, W, W + 512, Y - 16, (4 << 20) + 240):
        a = linear_args(stmat, workspace=at, workspace_bytes=need.value, **base)
        assert stmat.STATUS[stmat.lib().st_linear(C.byref(a), None)] == "ST_E_INVAL"
        assert "workspace" in stmat.lib().st_last_error().decode()


@gpu
def test_linear_binding_refuses_out_over_x_and_weight(stmat):
    buf = torch.zeros(64, 96, dtype=torch.bfloat16, device="cuda")
    x, w = buf[:, :32], torch.eye(32, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(64 * 32).view(64, 32) % 250)
    sq = torch.zeros(32, 32, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: stmat.linear(x, w, out=x), lambda: stmat.linear(x, w, out=buf[:, 31:63]),
                 lambda: stmat.linear(sq, w, out=w), lambda: stmat.linear(sq, w, out=sq)):
        with pytest.raises(stmat.StmatError) as e:
            call()
        assert e.value.status == "ST_E_INVAL"
    # columns of one buffer
    assert torch.equal(stmat.linear(x, w, out=buf[:, 32:64]), x)

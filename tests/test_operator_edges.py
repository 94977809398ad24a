"""Calls at the edges of what the operators take: which GPU they run on (with
stand-ins for tensors of several GPUs, on the CPU), operands that overlap,
activations far out, rows without columns, batches without rows, the smallest
scales, sums of more stages than any wait's polls."""
import contextlib
import ctypes as C
import math
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


# -------------------------------------------------------------- activations

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
ACTS = ["silu", "gelu", "gelu_tanh"]


def act64(v, act):
    """(act(v), |e|): the value in 64 bits and the size of its exponential's
    argument."""
    if act == "gelu":
        # erfc: torch's ndtr is 1 + erf, which keeps no digits far below 0
        return v * torch.special.erfc(-v * math.sqrt(0.5)) / 2, v * v / 2
    e = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    return v * torch.special.expit(e), e.abs()


def act_error(v, act, dtype):
    """(act(v), bound of the error), from the header's: relative to the value,
    then its rounding to dtype.  Below binary32's normal range the bound is
    absolute: an exponential there is off by half a unit of 2^-149 and the
    gate's at most 2^7 of them (F32), or 0 from 2^-126 on."""
    want, e = act64(v, act)
    far = 2.0 ** -142 if dtype == torch.float32 else 2.0 ** -126 * v.abs()
    if dtype != torch.float32:
        own = 2 * e + 6
    else:
        own = {"silu": 4, "gelu": 7}.get(act, 2 * e + 4)
    own = own * 2.0 ** -23 * want.abs()
    return want, own + U[dtype] * (want.abs() + own) + far + TINY[dtype]


def far_and_near():
    """Arguments of either sign from 2^-30 to 120, dense where the activations
    bend."""
    v = torch.cat([torch.linspace(-14, 14, 1 << 19), torch.linspace(-120, 120, 1 << 16),
                   torch.logspace(-30, 0, 1 << 15, base=2.0), -torch.logspace(-30, 0, 1 << 15, base=2.0)])
    return v[torch.randperm(v.numel(), generator=torch.Generator().manual_seed(1))].cuda().view(-1, 1024)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dst", ["F32", "BF16", "F16"])
def test_activations_relative_to_their_value(stmat, act, dst):
    v = far_and_near()
    y, _ = stmat.gated_act(v, act=act, dst=dst)
    want, tol = act_error(v.double(), act, y.dtype)
    off = (y.double() - want).abs() / tol
    assert (off <= 1).all(), (off.max().item(), v.flatten()[off.argmax()].item())
    # halves of an odd length, with up
    both = v.reshape(-1)[:1022 * 400].view(400, 1022)
    gate, up = both[:, :511], both[:, 511:]
    y, _ = stmat.gated_act(gate, up, act=act, dst=dst)
    want, tol = act_error(gate.double(), act, torch.float32 if dst == "F32" else torch.bfloat16)
    want, tol = want * up.double(), tol * up.double().abs() + (U[y.dtype] + 2.0 ** -24) * (want * up.double()).abs() + TINY[y.dtype]
    keep = want.abs() < 65000
    assert ((y.double() - want).abs() <= tol)[keep].all()


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_activations_of_rows_far_out_in_eight_bits(stmat, act):
    """Rows whose values all lie in one tail: their scale and codes hold the
    values' own digits."""
    for lo, hi in ((-4, -3), (-6, -5), (-7.5, -6.5), (-9, -8.5)):
        v = torch.linspace(lo, hi, 3 * 512).cuda().view(3, 512)
        y, scales = stmat.gated_act(v, act=act, dst="F8_E4M3")
        want, e = act64(v.double(), act)
        own = (2 * e.max() + 8) * 2.0 ** -23
        top = want.abs().amax(1) / 448
        assert ((scales.double() - top).abs() <= own * top).all()
        q = want / scales.double()[:, None]
        assert ((y.double() - q).abs() <= torch.clamp(q.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 16 * own) + 2 * own * q.abs()).all()


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dst", ["F32", "BF16"])
@pytest.mark.parametrize("m,n,k", [(3, 500, 4096), (40, 1201, 4096), (600, 512, 64), (600, 510, 64), (256, 1024, 4096)])
def test_product_activations_relative_to_their_value(stmat, act, dst, m, n, k):
    """Sums that are exact (one term each), so that the activation's error is
    all there is."""
    x, w = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    at = k - 5
    x[:, at] = torch.linspace(-9, 9, m, device="cuda")
    w[:, at] = torch.linspace(0.25, 1.4, n, device="cuda")
    x, w = x.bfloat16(), w.bfloat16()
    y = stmat.linear(x, w, act=act, dst=dst)
    want, tol = act_error(x[:, at].double()[:, None] * w[:, at].double()[None], act, y.dtype)
    off = (y.double() - want).abs() / tol
    assert (off <= 1).all(), off.max().item()


@gpu
@pytest.mark.parametrize("dst", ["F32", "BF16"])
def test_activations_of_infinities(stmat, dst):
    v = torch.tensor([[math.inf, -math.inf, math.nan, 3e38, -3e38, 0.0, -0.0, 1e-45]], device="cuda")
    x = v.clone().bfloat16().view(8, 1)
    w = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda")
    for act in ACTS:
        for y in (stmat.gated_act(v, act=act, dst=dst)[0][0], stmat.linear(x, w, act=act, dst=dst)[:, 0]):
            assert y[0] == math.inf and torch.isnan(y[1:3]).all() and y[3] > 2.9e38
            assert (y[4:7] == 0).all() and 0 <= y[7] <= 1e-44


# -------------------------------------------------------------- empty sizes

@gpu
@pytest.mark.parametrize("shape", [(3, 0), (2, 5, 0), (0, 0), (2500, 0), (0,)])
def test_rows_without_columns_have_the_smallest_scale(stmat, shape):
    """The largest magnitude of no value is 0."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        torch.full((1 << 16,), math.nan, device="cuda")  # what new scales would hold
        for y, scales in (stmat.rms_norm(x, residual=x, dst="F8_E4M3")[:2], stmat.gated_act(x, x, dst="F8_E4M3")):
            assert y.shape == shape and scales.shape == shape[:-1] and (scales == 2.0 ** -126).all()
        assert stmat.rms_norm(x)[0].shape == shape


@pytest.mark.parametrize("op,cls", [("st_rms_norm", "RmsNormArgs"), ("st_gated_act", "GatedActArgs")])
def test_no_rows_need_no_scales(stmat, op, cls):
    """An array of no entries has no address."""
    a = getattr(stmat, cls)(rows=0, cols=96, x_dtype=10, y_dtype=13)
    call = getattr(stmat.lib(), op)
    assert stmat.STATUS[call(C.byref(a), None)] == "ST_OK"
    a.scale = a.scales = X
    assert stmat.STATUS[call(C.byref(a), None)] == "ST_E_INVAL"
    a.scale, a.y_dtype = None, 10
    assert stmat.STATUS[call(C.byref(a), None)] == "ST_E_INVAL"


@gpu
def test_no_rows_in_eight_bits(stmat):
    x = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    for y, scales in (stmat.rms_norm(x, residual=x, dst="F8_E4M3")[:2], stmat.gated_act(x, x, dst="F8_E4M3")):
        assert y.shape == (0, 96) and scales.shape == (0,)


@pytest.mark.parametrize("shape", [(2, 0, 96), (0, 3, 96), (2, 0, 5, 96), (2, 3, 0, 96), (4, 0), (0, 0, 0), (1, 0, 1, 7)])
def test_batches_without_rows_are_no_stride_error(stmat, machine, shape):
    """Whatever strides such a tensor has: it has no row."""
    n = shape[-1]
    for x in (Tensor(shape), Tensor(shape, strides=tuple(range(41, 40 + len(shape))) + (1,))):
        machine.calls.clear()
        y, scales, h = stmat.rms_norm(x, residual=x, dst="F8_E4M3")
        assert y.shape == h.shape == shape and scales.shape == shape[:-1]
        assert stmat.gated_act(x, x)[0].shape == shape
        assert stmat.linear(x, Tensor((8, n))).shape == shape[:-1] + (8,)
        assert [c[0] for c in machine.calls] == ["rms_norm", "gated_act", "linear"]


@gpu
@pytest.mark.parametrize("shape", [(2, 0, 96), (0, 3, 96), (2, 3, 0, 96)])
def test_batches_without_rows(stmat, shape):
    x, w = torch.empty(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 96, dtype=torch.bfloat16, device="cuda")
    assert stmat.rms_norm(x, w[0], residual=x, dst="F8_E4M3")[0].shape == shape
    assert stmat.gated_act(x, x)[0].shape == shape
    assert stmat.linear(x, w, residual=None).shape == shape[:-1] + (8,)
    big = torch.zeros(2, 4, 96, dtype=torch.bfloat16, device="cuda")
    assert stmat.rms_norm(big[:, :0])[0].shape == (2, 0, 96) and stmat.linear(big[:, 4:], w).shape == (2, 0, 8)


# ----------------------------------------------------------- smallest scales

@gpu
@pytest.mark.parametrize("exponent", [-149, -146, -140, -129, -128, -127, -126, -120, -20])
@pytest.mark.parametrize("c", [40, 43, 20000])
def test_given_scales_of_any_size(stmat, exponent, c):
    """Codes are the clamped quotients, whether or not 1 / scale is a binary32
    number.  The values are whole multiples of 2^-149 (or of the scale's
    2^-5), so that the quotients have no error of their own."""
    scale = torch.tensor([2.0 ** exponent], device="cuda")
    unit = 2.0 ** max(-149, exponent - 5)
    g = torch.Generator().manual_seed(c)
    k = torch.randint(-20000, 20001, (3, c), generator=g).float()
    k[:, 1] = 0
    v = (k.double() * unit).float().cuda()
    v[0, 0], v[1, 0], v[2, 0] = 3e38, -1e-10, math.nan
    want = (v.double() / 2.0 ** exponent).clamp(-448, 448)

    def same(y):
        y = y.double()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        tol = torch.clamp(want.abs() * 2.0 ** -4, min=2.0 ** -10)
        assert torch.nan_to_num((y - want).abs() - tol, nan=0.0).max() <= 0

    same(stmat.gated_act(v, act="none", dst="F8_E4M3", scale=scale)[0])
    same(stmat.gated_act(v, torch.ones_like(v), act="none", dst="F8_E4M3", scale=scale)[0])
    # rows of ones: y is the weight (rstd is 1 to 2^-23)
    for row in range(3):
        y = stmat.rms_norm(torch.ones(1, c, device="cuda"), v[row], eps=0.0, dst="F8_E4M3", scale=scale)[0].double()
        q = want[row:row + 1]
        assert torch.equal(torch.isnan(y), torch.isnan(q))
        tol = torch.clamp(q.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 2.0 ** -18) + q.abs() * 2.0 ** -22 + unit / scale.double() / 2
        assert torch.nan_to_num((y - q).abs() - tol, nan=0.0).max() <= 0


@gpu
def test_a_given_scale_of_zero(stmat):
    v = torch.tensor([[0.0, 1.0, -1e-40, math.nan]], device="cuda")
    y = stmat.gated_act(v, act="none", dst="F8_E4M3", scale=torch.zeros(1, device="cuda"))[0].float()
    assert torch.isnan(y[0, 0]) and y[0, 1] == 448 and y[0, 2] == -448 and torch.isnan(y[0, 3])


# ----------------------------------------------------------------- long sums

@gpu
def test_a_sum_that_takes_longer_than_a_stages_wait(stmat):
    """2^29 terms: a quarter of a second between a readout's first poll and its
    last, in which a wait that allows for one stage can run out."""
    k = 1 << 29
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of device memory")
    x, w = torch.zeros(1, k, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, k, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 63, 64, k // 8 - 1, k // 8, k // 2 + 77, k - 65, k - 1], device="cuda")
    x[0, at] = torch.arange(1, 9, device="cuda").bfloat16()
    w[0, at], w[1, at[[0, 2, 4, 6]]] = 3, 5
    y = stmat.linear(x, w, dst="F32")
    assert y.tolist() == [[3.0 * 36, 5.0 * (1 + 3 + 5 + 7)]] and stmat.static_check() == 0


@gpu
def test_no_gradient_passes_through(stmat):
    """As their documentation says."""
    x, w = (torch.ones(4, 16, device="cuda", dtype=torch.bfloat16, requires_grad=True) for _ in range(2))
    for op, got in ((stmat.rms_norm, stmat.rms_norm(x, w[0].detach(), residual=x)), (stmat.gated_act, stmat.gated_act(x, x)),
                    (stmat.linear, (stmat.linear(x, w),))):
        assert all(t is None or not t.requires_grad for t in got) and "No gradient" in op.__doc__

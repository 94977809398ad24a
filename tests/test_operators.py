"""The operators on materialized tensors (st_rms_norm, st_gated_act,
st_linear): refusals on the CPU, results on the GPU against the formulas in
64 bits.

Tolerances, from the formats and the formulas:
  - a value rounded to BF16, F16 or F32 is off by at most u |y|, u = 2^-8,
    2^-11 or 2^-24 (half a unit of 8, 11 or 24 significant bits; F16: and 2^-25
    below its normal range);
  - an E4M3 code by 2^-4 |code| or half its subnormal step, 2^-10, times the
    scale;
  - binary32 work of a row operator: the sum of squares has positive terms, so
    its relative error is at most the depth of the sum (64 terms in a thread
    and 10 levels, halved by the root) and a handful of single roundings:
    48 * 2^-24 of the value, plus what exp, erf and tanh add (a few ulp of
    their result, magnified by no more than |argument| <= 32): 2^-18; where
    1 + erf or 1 + tanh cancels, a few ulp of 1 times the argument: 2^-21 |g|;
  - a product: every addition to a binary32 sum, rounded or truncated, is off
    by at most 2^-23 of what has been summed: k 2^-23 sum |x w|, times the
    scales and the activation's largest slope (1.13).
Integer inputs whose sums stay under 2^24 have exact products and are compared
bit for bit.
"""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
TYPES = {"BF16": torch.bfloat16, "F16": torch.float16, "F32": torch.float32, "F8_E4M3": torch.float8_e4m3fn,
         "F8_E5M2": torch.float8_e5m2}
ROW = 48 * 2.0 ** -24 + 2.0 ** -18
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def act64(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def normal(seed, *shape, dtype=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(dtype).cuda()


def padded(t, extra, offset=0):
    """t as a view with `extra` unused columns between rows, starting `offset`
    elements into its buffer (the rest holds a guard value)."""
    m, c = t.shape
    buf = torch.full((offset + m * (c + extra) + 64,), 77.0, device="cuda").to(t.dtype)
    v = buf[offset:offset + m * (c + extra)].view(m, c + extra)[:, :c] if m else buf[:0].view(0, c)
    v.copy_(t)
    return v


def check_values(got, want, extra=0.0, slack=ROW):
    """got (16 or 32 bits) against want (64 bits)."""
    assert got.shape == want.shape
    u = U[got.dtype]
    tol = (u * (1 + slack) + slack) * want.abs() + TINY[got.dtype] + extra
    bad = ((got.double() - want).abs() > tol).sum().item()
    assert bad == 0, f"{bad} of {want.numel()} off, worst {((got.double() - want).abs() / tol).max().item():.3g} of the tolerance"


def check_codes(codes, scale, want, slack=ROW):
    """8-bit codes times their scale(s) against want (64 bits)."""
    s = scale.double().reshape(-1, 1) if scale.numel() > 1 else scale.double().reshape(1, 1)
    q = (want / s).clamp(-448, 448)
    tol = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) * (1 + 2 * slack) + 2 * slack * q.abs()
    off = (codes.double() - q).abs()
    assert (off <= tol).all(), f"worst {(off / tol).max().item():.3g} of the tolerance"


def check_scales(scales, want):
    top = (want.abs().amax(-1) / 448).clamp_min(2.0 ** -126)
    assert ((scales.double() - top).abs() <= 2 * ROW * top).all()


# --------------------------------------------------------------- refusals

def norm_args(stmat, **kw):
    a = stmat.RmsNormArgs(rows=2, cols=8, eps=1e-5, x_dtype=10, w_dtype=10, y_dtype=10, x=1 << 20, ldx=8,
                          weight=2 << 20, y=3 << 20, ldy=8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def act_args(stmat, **kw):
    a = stmat.GatedActArgs(rows=2, cols=8, act=2, x_dtype=10, y_dtype=10, gate=1 << 20, ldg=8, up=2 << 20, ldu=8,
                           y=3 << 20, ldy=8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def linear_args(stmat, **kw):
    a = stmat.LinearArgs(m=2, n=8, k=16, act=0, x_dtype=10, w_dtype=10, y_dtype=10, bias_dtype=11, x=1 << 20, ldx=16,
                         w=2 << 20, ldw=16, y=3 << 20, ldy=8)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


OPS = {"st_rms_norm": norm_args, "st_gated_act": act_args, "st_linear": linear_args}
REFUSED = [
    ("st_rms_norm", dict(x=None), "ST_E_INVAL"), ("st_rms_norm", dict(y=None), "ST_E_INVAL"),
    ("st_rms_norm", dict(rows=-1), "ST_E_INVAL"), ("st_rms_norm", dict(cols=1 << 31), "ST_E_INVAL"),
    ("st_rms_norm", dict(ldx=7), "ST_E_INVAL"), ("st_rms_norm", dict(ldy=0), "ST_E_INVAL"),
    ("st_rms_norm", dict(ldx=-8), "ST_E_INVAL"), ("st_rms_norm", dict(ldx=1 << 62), "ST_E_INVAL"),
    ("st_rms_norm", dict(x=(1 << 20) + 1), "ST_E_ALIGN"), ("st_rms_norm", dict(weight=(2 << 20) + 1), "ST_E_ALIGN"),
    ("st_rms_norm", dict(x_dtype=13), "ST_E_DTYPE"), ("st_rms_norm", dict(w_dtype=13), "ST_E_DTYPE"),
    ("st_rms_norm", dict(y_dtype=14), "ST_E_DTYPE"), ("st_rms_norm", dict(eps=-1.0), "ST_E_INVAL"),
    ("st_rms_norm", dict(eps=math.nan), "ST_E_INVAL"), ("st_rms_norm", dict(h=4 << 20, ldh=8), "ST_E_INVAL"),
    ("st_rms_norm", dict(residual=4 << 20, ldr=3), "ST_E_INVAL"),
    ("st_rms_norm", dict(y_dtype=13), "ST_E_INVAL"), ("st_rms_norm", dict(scales=4 << 20), "ST_E_INVAL"),
    ("st_rms_norm", dict(y_dtype=13, scale=4 << 20, scales=5 << 20), "ST_E_INVAL"),
    ("st_rms_norm", dict(y_dtype=13, scales=(4 << 20) + 2), "ST_E_ALIGN"),
    ("st_gated_act", dict(gate=None), "ST_E_INVAL"), ("st_gated_act", dict(y=None), "ST_E_INVAL"),
    ("st_gated_act", dict(act=5), "ST_E_INVAL"), ("st_gated_act", dict(act=-1), "ST_E_INVAL"),
    ("st_gated_act", dict(ldu=7), "ST_E_INVAL"), ("st_gated_act", dict(x_dtype=0), "ST_E_DTYPE"),
    ("st_gated_act", dict(y_dtype=99), "ST_E_DTYPE"), ("st_gated_act", dict(up=(2 << 20) + 1), "ST_E_ALIGN"),
    ("st_linear", dict(x=None), "ST_E_INVAL"), ("st_linear", dict(w=None), "ST_E_INVAL"),
    ("st_linear", dict(y=None), "ST_E_INVAL"), ("st_linear", dict(m=-1), "ST_E_INVAL"),
    ("st_linear", dict(k=-1), "ST_E_INVAL"), ("st_linear", dict(n=1 << 31), "ST_E_INVAL"),
    ("st_linear", dict(ldx=15), "ST_E_INVAL"), ("st_linear", dict(ldw=15), "ST_E_INVAL"),
    ("st_linear", dict(ldy=7), "ST_E_INVAL"), ("st_linear", dict(act=9), "ST_E_INVAL"),
    ("st_linear", dict(x_dtype=9), "ST_E_DTYPE"), ("st_linear", dict(x_dtype=11, w_dtype=11), "ST_E_DTYPE"),
    ("st_linear", dict(x_dtype=14, w_dtype=14), "ST_E_DTYPE"), ("st_linear", dict(x_dtype=10, w_dtype=13), "ST_E_DTYPE"),
    ("st_linear", dict(y_dtype=13), "ST_E_DTYPE"), ("st_linear", dict(bias=4 << 20, bias_dtype=13), "ST_E_DTYPE"),
    ("st_linear", dict(x_scale=4 << 20, x_scale_count=3), "ST_E_INVAL"),
    ("st_linear", dict(w_scale=4 << 20, w_scale_count=2), "ST_E_INVAL"),
    ("st_linear", dict(w_scale=(4 << 20) + 2, w_scale_count=1), "ST_E_ALIGN"),
    ("st_linear", dict(residual=4 << 20, ldr=7), "ST_E_INVAL"), ("st_linear", dict(y=(3 << 20) + 1), "ST_E_ALIGN"),
]


@pytest.mark.parametrize("op,kw,status", REFUSED, ids=[f"{o[3:]}-{'-'.join(k)}-{i}" for i, (o, k, _) in enumerate(REFUSED)])
def test_refusals_queue_nothing(stmat, op, kw, status):
    """Every check runs on the host before anything is queued (there is no GPU
    here, and the addresses are made up)."""
    a = OPS[op](stmat, **kw)
    assert stmat.STATUS[getattr(stmat.lib(), op)(C.byref(a), None)] == status
    assert op in stmat.lib().st_last_error().decode()


@pytest.mark.parametrize("op", OPS)
def test_null_arguments_and_empty_sizes(stmat, op):
    call = getattr(stmat.lib(), op)
    assert stmat.STATUS[call(None, None)] == "ST_E_INVAL"
    rows, cols = ("m", "n") if op == "st_linear" else ("rows", "cols")
    for kw in ({rows: 0}, {cols: 0}, {rows: 0, "y": None}):
        assert stmat.STATUS[call(C.byref(OPS[op](stmat, **kw)), None)] == "ST_OK"


def test_linear_workspace_size_and_refusals(stmat):
    """Room for an aligned copy of what does not lie on 16-byte boundaries."""
    call, need = stmat.lib().st_linear_workspace, C.c_uint64()
    for kw, want in ((dict(), 0), (dict(ldx=17), 2 * 32), (dict(x=(1 << 20) + 2), 2 * 32), (dict(ldw=18), 8 * 32),
                     (dict(k=13), 0), (dict(k=13, ldx=13, ldw=13), 10 * 32), (dict(m=1, ldx=17), 0), (dict(ldw=0), 8 * 32),
                     (dict(k=0, ldx=1), 0), (dict(m=0, ldx=17), 0),
                     (dict(x_dtype=13, w_dtype=13, ldw=24), 8 * 16)):
        a = linear_args(stmat, **kw)
        assert stmat.STATUS[call(C.byref(a), C.byref(need))] == "ST_OK"
        assert need.value == want, kw
    a = linear_args(stmat, ldx=17)
    for kw, status in ((dict(), "ST_E_INVAL"), (dict(workspace=5 << 20, workspace_bytes=63), "ST_E_INVAL"),
                       (dict(workspace=(5 << 20) + 8, workspace_bytes=64), "ST_E_ALIGN")):
        for k, v in kw.items():
            setattr(a, k, v)
        assert stmat.STATUS[stmat.lib().st_linear(C.byref(a), None)] == status
    assert stmat.STATUS[call(None, C.byref(need))] == "ST_E_INVAL"
    assert stmat.STATUS[call(C.byref(a), None)] == "ST_E_INVAL"
    assert stmat.STATUS[call(C.byref(linear_args(stmat, k=-1)), C.byref(need))] == "ST_E_INVAL"


def test_packed_arguments_have_the_structs_layout(stmat):
    for packed, cls in ((stmat._NORM_ARGS, stmat.RmsNormArgs), (stmat._ACT_ARGS, stmat.GatedActArgs),
                        (stmat._LINEAR_ARGS, stmat.LinearArgs)):
        n = len(cls._fields_)
        got = cls.from_buffer_copy(packed.pack(*range(1, n + 1)))
        assert packed.size == C.sizeof(cls)
        assert [getattr(got, f) for f, _ in cls._fields_] == list(range(1, n + 1))


def test_binding_refuses_host_tensors_and_unknown_names(stmat):
    x = torch.zeros(2, 8)
    for call in (lambda: stmat.rms_norm(x), lambda: stmat.gated_act(x), lambda: stmat.linear(x, x)):
        with pytest.raises(stmat.StmatError) as e:
            call()
        assert e.value.status == "ST_E_INVAL"


@gpu
def test_binding_refusals(stmat):
    x, w = normal(1, 4, 16, dtype=torch.bfloat16), normal(2, 8, 16, dtype=torch.bfloat16)
    vec = normal(3, 16)
    bad = [
        (lambda: stmat.rms_norm(x.t()), "ST_E_INVAL"),
        (lambda: stmat.rms_norm(x, vec[:8]), "ST_E_INVAL"),
        (lambda: stmat.rms_norm(x, vec, residual=x[:2]), "ST_E_INVAL"),
        (lambda: stmat.rms_norm(x, vec, residual=x.float()), "ST_E_INVAL"),
        (lambda: stmat.rms_norm(x, vec, dst="F8_E5M2"), "ST_E_DTYPE"),
        (lambda: stmat.rms_norm(x, vec, dst="I8"), "ST_E_DTYPE"),
        (lambda: stmat.rms_norm(x, vec, scale=vec[:1]), "ST_E_INVAL"),
        (lambda: stmat.rms_norm(x.double(), vec), "ST_E_DTYPE"),
        (lambda: stmat.rms_norm(x[None].expand(3, 4, 16).transpose(0, 1), vec), "ST_E_INVAL"),
        (lambda: stmat.gated_act(x, x[:, :8]), "ST_E_INVAL"),
        (lambda: stmat.gated_act(x, x, act="swish"), "ST_E_INVAL"),
        (lambda: stmat.linear(x, w[:, :8]), "ST_E_INVAL"),
        (lambda: stmat.linear(x, w.half()), "ST_E_DTYPE"),
        (lambda: stmat.linear(x, w, bias=vec), "ST_E_INVAL"),
        (lambda: stmat.linear(x, w, x_scale=vec[:3]), "ST_E_INVAL"),
        (lambda: stmat.linear(x, w, w_scale=vec[:8].half()), "ST_E_DTYPE"),
        (lambda: stmat.linear(x, w, residual=x), "ST_E_INVAL"),
        (lambda: stmat.linear(x, w, out=x), "ST_E_INVAL"),
        (lambda: stmat.linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), dst="F8_E4M3"), "ST_E_DTYPE"),
    ]
    for i, (call, status) in enumerate(bad):
        with pytest.raises(stmat.StmatError) as e:
            call()
        assert e.value.status == status, (i, e.value)


# ------------------------------------------------------------------- norm

# (rows, cols): one element, warp rows, block rows of each register depth,
# scalar rows, rows longer than registers hold.
NORM_SIZES = [(1, 1), (3, 7), (9, 8), (17, 64), (5, 256), (33, 264), (1, 4096), (2, 5120), (7, 1111), (3, 12288),
              (2, 16381), (2, 32768), (1, 32776), (2, 17000)]


def norm64(x, r, w, eps):
    h = x.double() if r is None else x.double() + r.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return h, y if w is None else y * w.double()


@gpu
@pytest.mark.parametrize("m,c", NORM_SIZES)
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
def test_norm_values(stmat, m, c, dtype):
    dt = TYPES[dtype]
    x, r, w = normal(m + c, m, c, dtype=dt), normal(m + c + 1, m, c, dtype=dt), normal(3, c, dtype=dt)
    for residual, weight, dst in ((r, w, dtype), (None, w, "F32"), (r, None, "BF16"), (None, w.float(), "F16")):
        y, scales, h = stmat.rms_norm(x, weight, eps=1e-5, residual=residual, dst=dst)
        h64, y64 = norm64(x, residual, weight, 1e-5)
        assert scales is None and (h is None) == (residual is None)
        check_values(y, y64)
        if h is not None:
            check_values(h, h64, slack=2.0 ** -23)


@gpu
@pytest.mark.parametrize("m,c", NORM_SIZES)
@pytest.mark.parametrize("static", [False, True])
def test_norm_codes(stmat, m, c, static):
    x, r, w = (normal(m + c + i, *s, dtype=torch.bfloat16) for i, s in enumerate([(m, c), (m, c), (c,)]))
    given = torch.tensor([0.004], device="cuda") if static else None
    y, scales, h = stmat.rms_norm(x, w, residual=r, dst="F8_E4M3", scale=given)
    h64, y64 = norm64(x, r, w, 1e-5)
    assert y.dtype == torch.float8_e4m3fn and (scales is None) == static
    if not static:
        check_scales(scales, y64)
        assert (y.float().abs().amax(1) == 448).all()
    check_codes(y, given if static else scales, y64)
    check_values(h, h64, slack=2.0 ** -23)


@gpu
@pytest.mark.parametrize("extra,offset", [(0, 1), (1, 0), (8, 0), (8, 8), (3, 5)])
@pytest.mark.parametrize("dst", ["BF16", "F8_E4M3"])
def test_norm_strides_and_offsets(stmat, extra, offset, dst):
    """Rows apart and off 16-byte boundaries; nothing is written outside."""
    m, c = 5, 520
    x, r = normal(1, m, c, dtype=torch.bfloat16), normal(2, m, c, dtype=torch.bfloat16)
    w = normal(3, c + 1, dtype=torch.bfloat16)[1:]
    a = stmat.RmsNormArgs(rows=m, cols=c, eps=1e-6, x_dtype=10, w_dtype=10, y_dtype=stmat.DTYPES.index(dst))
    xv, rv = padded(x, extra, offset), padded(r, extra + 1, offset + 1)
    yv, hv = padded(torch.zeros_like(x).to(TYPES[dst]), extra, offset), padded(torch.zeros_like(x), extra, offset)
    scales = torch.full((m + 1,), 5.0, device="cuda")
    a.x, a.ldx, a.residual, a.ldr = xv.data_ptr(), c + extra, rv.data_ptr(), c + extra + 1
    a.y, a.ldy, a.h, a.ldh, a.weight = yv.data_ptr(), c + extra, hv.data_ptr(), c + extra, w.data_ptr()
    if dst == "F8_E4M3":
        a.scales = scales.data_ptr()
    stmat._check(stmat.lib().st_rms_norm(a, torch.cuda.current_stream().cuda_stream))
    h64, y64 = norm64(x, r, w, 1e-6)
    check_values(hv, h64, slack=2.0 ** -23)
    if dst == "F8_E4M3":
        check_codes(yv, scales[:m], y64)
    else:
        check_values(yv, y64)
    assert scales[m] == 5.0
    for v in (yv, hv):
        base = v._base if v._base is not None else v
        flat = base.reshape(-1).float()
        inside = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
        inside[offset:offset + m * (c + extra)].view(m, c + extra)[:, :c] = True
        guard = torch.tensor(77.0).to(v.dtype).float().item()
        assert (flat[~inside] == guard).all()


@gpu
@pytest.mark.parametrize("m,c", [(3, 5), (9, 77), (4, 1111), (300, 2405), (2, 9001)])
@pytest.mark.parametrize("extra,offset", [(0, 3), (2, 0), (5, 7), (8, 1)])
@pytest.mark.parametrize("dtype", ["BF16", "F32"])
@pytest.mark.parametrize("dst", ["BF16", "F32", "F8_E4M3"])
def test_norm_rows_off_the_same_boundary(stmat, m, c, extra, offset, dtype, dst):
    """Every matrix with the same stride and offset: accesses around the rows,
    of whose elements outside the row none is changed (or read into a sum: the
    buffers hold 77 there)."""
    dt = TYPES[dtype]
    x, r, w = normal(1, m, c, dtype=dt), normal(2, m, c, dtype=dt), normal(3, c + 1, dtype=dt)[1:]
    a = stmat.RmsNormArgs(rows=m, cols=c, eps=1e-6, x_dtype=stmat.DTYPES.index(dtype), w_dtype=stmat.DTYPES.index(dtype),
                          y_dtype=stmat.DTYPES.index(dst))
    xv, rv, yv, hv = (padded(t, extra, offset) for t in (x, r, torch.zeros_like(x).to(TYPES[dst]), torch.zeros_like(x)))
    scales = torch.zeros(m, device="cuda")
    for field, v in (("x", xv), ("residual", rv), ("h", hv), ("y", yv), ("weight", w)):
        setattr(a, field, v.data_ptr())
    a.ldx = a.ldr = a.ldh = a.ldy = c + extra
    if dst == "F8_E4M3":
        a.scales = scales.data_ptr()
    stmat._check(stmat.lib().st_rms_norm(a, torch.cuda.current_stream().cuda_stream))
    h64, y64 = norm64(x, r, w, 1e-6)
    check_values(hv, h64, slack=2.0 ** -23)
    if dst == "F8_E4M3":
        check_scales(scales, y64)
        check_codes(yv, scales, y64)
    else:
        check_values(yv, y64)
    for v in (yv, hv):
        flat = v._base.reshape(-1).float()
        inside = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
        inside[offset:offset + m * (c + extra)].view(m, c + extra)[:, :c] = True
        assert (flat[~inside] == torch.tensor(77.0).to(v.dtype).float().item()).all()


@gpu
def test_norm_special_rows(stmat):
    """Zero rows, rows of the smallest numbers, and NaN and infinities, which
    stay in their own rows."""
    c = 512
    x = normal(5, 6, c, dtype=torch.bfloat16)
    x[0] = 0
    x[1] = 2.0 ** -130
    x[2, 17] = math.nan
    x[3, 5] = math.inf
    x[4, 400] = -math.inf
    w = torch.ones(c, dtype=torch.bfloat16, device="cuda")
    y, scales, _ = stmat.rms_norm(x, w, dst="F8_E4M3")
    y16, _, _ = stmat.rms_norm(x, w)
    want = norm64(x, None, w, 1e-5)[1]
    assert (y[0].float() == 0).all() and scales[0] == 2.0 ** -126 and (y16[0] == 0).all()
    check_codes(y[1:2], scales[1:2], want[1:2])
    assert torch.isnan(scales[2:5]).all()
    assert torch.isnan(y[2:5].float()).all()
    assert torch.isnan(y16[2]).all()
    for row, at in ((3, 5), (4, 400)):
        assert torch.isnan(y16[row, at])
        assert (torch.cat([y16[row, :at], y16[row, at + 1:]]) == 0).all()
    check_codes(y[5:], scales[5:], want[5:])
    # eps 0 and a zero row: 0 / 0
    assert torch.isnan(stmat.rms_norm(x[:1], w, eps=0.0)[0]).all()


@gpu
def test_norm_shapes(stmat):
    """A vector, leading dimensions, an expanded residual, no rows."""
    w = normal(1, 96)
    x = normal(2, 2, 3, 96)
    y, scales, h = stmat.rms_norm(x, w, residual=x[0, 0].expand(2, 3, 96), dst="F8_E4M3")
    assert y.shape == x.shape == h.shape and scales.shape == (2, 3)
    want = norm64(x, x[0, 0].expand(2, 3, 96), w, 1e-5)[1]
    check_codes(y.reshape(6, 96), scales.reshape(6), want.reshape(6, 96))
    y, scales, _ = stmat.rms_norm(x[0, 0], w)
    assert y.shape == (96,) and scales is None
    check_values(y, norm64(x[0, 0], None, w, 1e-5)[1])
    assert stmat.rms_norm(x[:0], w)[0].shape == (0, 3, 96)
    assert stmat.rms_norm(x[..., :0])[0].shape == (2, 3, 0)


@gpu
def test_norm_in_place(stmat):
    """h over x and y over the residual, as a serving loop keeps its stream."""
    for c in (768, 771, 33000):
        x, r, w = (normal(i, *s, dtype=torch.bfloat16) for i, s in enumerate([(9, c), (9, c), (c,)]))
        h64, y64 = norm64(x, r, w, 1e-5)
        a = stmat.RmsNormArgs(rows=9, cols=c, eps=1e-5, x_dtype=10, w_dtype=10, y_dtype=10, x=x.data_ptr(), ldx=c,
                              residual=r.data_ptr(), ldr=c, weight=w.data_ptr(), h=x.data_ptr(), ldh=c,
                              y=r.data_ptr(), ldy=c)
        stmat._check(stmat.lib().st_rms_norm(a, torch.cuda.current_stream().cuda_stream))
        check_values(x, h64, slack=2.0 ** -23)
        check_values(r, y64)


# ------------------------------------------------------------- activation

@gpu
@pytest.mark.parametrize("m,c", [(1, 1), (4, 9), (3, 64), (2, 777), (1, 14336), (5, 2048), (2, 20001), (1, 40000)])
@pytest.mark.parametrize("act", ACTS)
def test_gated_act_values(stmat, m, c, act):
    for dt, dst in ((torch.bfloat16, "BF16"), (torch.float16, "F32"), (torch.float32, "F16")):
        both = normal(m + c, m, 2 * c, dtype=dt, spread=4.0)
        gate, up = both[:, :c], both[:, c:]
        y, scales = stmat.gated_act(gate, up, act=act, dst=dst)
        assert scales is None
        cancel = 2.0 ** -21 * gate.double().abs()
        check_values(y, act64(gate.double(), act) * up.double(), extra=cancel * up.double().abs())
        y, _ = stmat.gated_act(gate, act=act, dst=dst)
        check_values(y, act64(gate.double(), act), extra=cancel)


@gpu
@pytest.mark.parametrize("m,c", [(1, 1), (4, 9), (3, 64), (2, 777), (1, 14336), (6, 2048), (1, 40000)])
@pytest.mark.parametrize("static", [False, True])
def test_gated_act_codes(stmat, m, c, static):
    gate, up = normal(m, m, c, dtype=torch.bfloat16), normal(c, m, c, dtype=torch.bfloat16)
    given = torch.tensor([0.003], device="cuda") if static else None
    y, scales = stmat.gated_act(gate, up, dst="F8_E4M3", scale=given)
    want = act64(gate.double(), "silu") * up.double()
    if not static:
        check_scales(scales, want)
    check_codes(y, given if static else scales, want)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_gated_act_special_values(stmat, act):
    """Arguments far out on both sides, zeros, and a NaN's row."""
    v = torch.tensor([[-100.0, -30.0, -1e-30, 0.0, 1e-30, 30.0, 100.0, 1e4]] * 2, device="cuda")
    up = torch.full_like(v, 0.5)
    v[1, 3] = math.nan
    y, _ = stmat.gated_act(v, up, act=act)
    want = act64(v.double(), act) * 0.5
    check_values(y[:1], want[:1], extra=2.0 ** -20)
    y, scales = stmat.gated_act(v, up, act=act, dst="F8_E4M3")
    assert torch.isfinite(scales[0]) and torch.isnan(scales[1]) and torch.isnan(y[1].float()).all()


# ----------------------------------------------------------------- linear

def linear64(x, w, xs=None, ws=None, b=None, act="none", r=None):
    """(y, bound of the sum's error) in 64 bits."""
    s = x.double() @ w.double().t()
    top = x.double().abs() @ w.double().abs().t() * (x.shape[-1] * 2.0 ** -23)
    for f in ([] if xs is None else [xs.double().reshape(-1, 1)]) + ([] if ws is None else [ws.double().reshape(1, -1)]):
        s, top = s * f, top * f.abs()
    if b is not None:
        s = s + b.double()
    y = act64(s, act)
    slack = 1.13 * top + 2.0 ** -20 * s.abs() * (act != "none")
    return (y if r is None else y + r.double()), slack


def check_linear(got, want, slack):
    check_values(got, want, extra=slack, slack=2.0 ** -21)


# One element; one token; fewer rows than a tile; ragged in every dimension;
# more than a tile; long sums; single columns.
LINEAR_SIZES = [(1, 1, 1), (1, 8, 16), (1, 300, 257), (3, 128, 64), (2, 1, 512), (16, 129, 40), (17, 256, 1000),
                (33, 1111, 72), (65, 64, 2048), (100, 391, 333), (129, 257, 130), (200, 512, 4096), (300, 96, 8),
                (257, 640, 768), (520, 1000, 520), (1, 2048, 8192), (7, 4104, 1544), (768, 512, 128), (513, 257, 1040),
                (1111, 2000, 80), (600, 33, 4096), (2560, 2592, 272), (777, 1, 16)]
PAIRS = [("BF16", "BF16"), ("F16", "F16"), ("F8_E4M3", "F8_E4M3"), ("F8_E4M3", "F8_E5M2")]


def operands(m, n, k, xt, wt, seed=0):
    return normal(seed + m, m, k, dtype=TYPES[xt]), normal(seed + n + 1, n, k, dtype=TYPES[wt], spread=0.5)


@gpu
@pytest.mark.parametrize("m,n,k", LINEAR_SIZES)
@pytest.mark.parametrize("xt,wt", PAIRS)
def test_linear_values(stmat, m, n, k, xt, wt):
    x, w = operands(m, n, k, xt, wt)
    y = stmat.linear(x, w, dst="F32")
    want, slack = linear64(x, w)
    check_linear(y, want, slack)
    assert torch.equal(y, stmat.linear(x, w, dst="F32"))    # the same bits again
    y = stmat.linear(x, w)
    assert y.dtype == (torch.float16 if xt == "F16" else torch.bfloat16)
    check_linear(y, want, slack)


@gpu
@pytest.mark.parametrize("m,n,k", LINEAR_SIZES)
@pytest.mark.parametrize("xt,wt", PAIRS)
def test_linear_of_integers_is_exact(stmat, m, n, k, xt, wt):
    """Small integers: every partial sum is exact, so any order gives the same
    bits; a wrong, missing or repeated element shows."""
    g = torch.Generator().manual_seed(m * n + k)
    x = torch.randint(-3, 4, (m, k), generator=g).float()
    w = torch.randint(-3, 4, (n, k), generator=g).float()
    y = stmat.linear(x.to(TYPES[xt]).cuda(), w.to(TYPES[wt]).cuda(), dst="F32")
    assert torch.equal(y.cpu().double(), x.double() @ w.double().t())


@gpu
@pytest.mark.parametrize("m,n,k", [(100003, 17, 40), (70000, 300, 48), (3, 100001, 64), (17, 30000, 64), (3, 5, 200000),
                                   (5, 7, 100001), (700, 700, 20000)])
@pytest.mark.parametrize("xt", ["BF16", "F8_E4M3"])
def test_linear_of_integers_far_out(stmat, m, n, k, xt):
    """Many tokens, many weight rows, long sums, compared on the GPU: integers
    of magnitude 2, whose sums a binary32 product holds exactly too."""
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = torch.randint(-2, 3, (m, k), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (n, k), generator=g, device="cuda").float()
    y = stmat.linear(x.to(TYPES[xt]), w.to(TYPES[xt]), dst="F32")
    assert torch.equal(y, x @ w.t())


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 200, 136), (5, 328, 64), (40, 130, 96), (150, 391, 300), (300, 520, 128), (600, 544, 256),
                                   (530, 391, 64)])
def test_linear_epilogue(stmat, m, n, k, act):
    """Scales per row and single, bias in each type, residual, activation."""
    for xt, wt, dst, bt, rows, cols in (("F8_E4M3", "F8_E4M3", "BF16", "BF16", m, 1),
                                        ("F8_E4M3", "F8_E5M2", "F16", "F32", 1, n),
                                        ("BF16", "BF16", "F32", "F16", m, n), ("F16", "F16", "F16", "F16", 0, 0)):
        x, w = operands(m, n, k, xt, wt, seed=7)
        xs = normal(8, rows).abs() * 0.1 + 0.01 if rows else None
        ws = normal(9, cols).abs() * 0.1 + 0.01 if cols else None
        b, r = normal(10, n, dtype=TYPES[bt]), normal(11, m, n, dtype=TYPES[dst])
        for bias, residual in ((b, r), (b, None), (None, r)):
            y = stmat.linear(x, w, xs, ws, bias, act, residual, dst)
            want, slack = linear64(x, w, xs, ws, bias, act, residual)
            scale = 2.0 ** -21 * (want - (residual.double() if residual is not None else 0)).abs()
            check_linear(y, want, slack + scale + 2.0 ** -22 * (bias.double().abs() if bias is not None else 0))


@gpu
@pytest.mark.parametrize("m,n,k", [(1, 72, 64), (6, 200, 128), (130, 264, 256), (300, 300, 100), (515, 304, 192)])
@pytest.mark.parametrize("xt", ["BF16", "F8_E4M3"])
@pytest.mark.parametrize("extra,offset", [(16, 0), (16, 16), (1, 0), (0, 1), (7, 3)])
def test_linear_strides_and_offsets(stmat, m, n, k, xt, extra, offset):
    """Row strides, addresses off 16-byte boundaries, and no write outside y."""
    x, w = operands(m, n, k, xt, xt)
    r = normal(5, m, n, dtype=torch.bfloat16)
    xv, wv, rv = padded(x, extra, offset), padded(w, extra, offset), padded(r, extra + 1, offset + 1)
    yv = padded(torch.zeros_like(r), extra, offset)
    stmat.linear(xv, wv, residual=rv, out=yv)
    want, slack = linear64(x, w, r=r)
    check_linear(yv, want, slack)
    flat = yv._base.reshape(-1).float()
    inside = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
    inside[offset:offset + m * (n + extra)].view(m, n + extra)[:, :n] = True
    assert (flat[~inside] == torch.tensor(77.0).bfloat16().float().item()).all()


@gpu
def test_linear_empty_sum_and_sizes(stmat):
    for xt in ("BF16", "F8_E4M3"):
        x, w = (torch.zeros(s, 0, device="cuda").to(TYPES[xt]) for s in (5, 40))
        b, r = normal(1, 40, dtype=torch.bfloat16), normal(2, 5, 40, dtype=torch.bfloat16)
        y = stmat.linear(x, w, bias=b, act="silu", residual=r, dst="BF16")
        check_values(y, act64(b.double(), "silu") + r.double(), extra=2.0 ** -20)
        assert (stmat.linear(x, w, dst="F32") == 0).all()
    x, w = normal(3, 4, 32, dtype=torch.float16), normal(4, 24, 32, dtype=torch.float16)
    assert stmat.linear(x[:0], w).shape == (0, 24) and stmat.linear(x, w[:0]).shape == (4, 0)
    assert stmat.linear(x[0], w).shape == (24,)
    assert stmat.linear(x.view(2, 2, 32), w).shape == (2, 2, 24)
    # one row for every token
    y = stmat.linear(x[0].expand(4, 32), w, dst="F32")
    want, slack = linear64(x[0].expand(4, 32), w)
    check_linear(y, want, slack)


@gpu
@pytest.mark.parametrize("m", [1, 20, 200, 700])
def test_linear_residual_in_place(stmat, m):
    x, w = operands(m, 1024, 512, "BF16", "BF16")
    r = normal(3, m, 1024, dtype=torch.bfloat16)
    want, slack = linear64(x, w, r=r)
    y = stmat.linear(x, w, residual=r, out=r)
    assert y.data_ptr() == r.data_ptr()
    check_linear(r, want, slack)


@gpu
@pytest.mark.parametrize("xt", ["BF16", "F8_E4M3"])
@pytest.mark.parametrize("m,n,k", [(40, 150, 200), (600, 150, 208)])
def test_linear_nan_and_infinity(stmat, m, n, k, xt):
    """They stay in their row and column; a tile's other rows are untouched."""
    x, w = operands(m, n, k, xt, xt)
    x[3, 7] = math.nan
    if xt == "BF16":
        x[9, 100] = math.inf
        w[11, 199] = -math.inf
    y = stmat.linear(x, w, dst="F32")
    want = x.double() @ w.double().t()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(y.double()[inf], want[inf])
    clean = torch.isfinite(want)
    x2, w2 = torch.nan_to_num(x.float(), 0, 0, 0), torch.nan_to_num(w.float(), 0, 0, 0)
    slack = x2.double().abs() @ w2.double().abs().t() * (k * 2.0 ** -23)
    assert ((y.double() - want).abs()[clean] <= (slack + 2.0 ** -20 * want.abs())[clean]).all()


@gpu
def test_linear_offsets_beyond_32_bits(stmat):
    """A weight whose last rows start more than 2^32 elements in (a slice of a
    larger buffer), and an output of the same kind."""
    k, ld = 64, 1 << 25
    rows = 130
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    buf = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
    w = buf.view(rows, ld)[:, :k]
    x, src = operands(3, rows, k, "BF16", "BF16")
    w.copy_(src)
    want, slack = linear64(x, src)
    check_linear(stmat.linear(x, w, dst="F32"), want, slack)
    want, slack = linear64(src, x)
    out = buf.view(rows, ld)[:, 1024:1027]
    stmat.linear(src, x, out=out)
    check_linear(out, want, slack)


# ------------------------------------------------------- streams and graphs

@gpu
def test_operators_on_another_stream_and_in_a_graph(stmat):
    side = torch.cuda.Stream()
    x, r, w = normal(1, 8, 1024, dtype=torch.bfloat16), normal(2, 8, 1024, dtype=torch.bfloat16), normal(3, 1024)
    weight = normal(4, 512, 1024).to(torch.float8_e4m3fn)
    torch.cuda.synchronize()

    def chain(stream=None):
        y, s, h = stmat.rms_norm(x, w, residual=r, dst="F8_E4M3", stream=stream)
        z = stmat.linear(y, weight, x_scale=s, dst="BF16", stream=stream)
        return stmat.gated_act(z[:, :256], z[:, 256:], dst="F8_E4M3", stream=stream)

    want = chain()
    for stream in (side, side.cuda_stream):
        got = chain(stream)
        side.synchronize()
        assert torch.equal(got[0].float(), want[0].float()) and torch.equal(got[1], want[1])
    # captured after a copy on the same stream, and after work of another one
    graph, source = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        x.copy_(source)
        got = chain()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = chain()
        torch.cuda.current_stream().wait_stream(side)
        y, s, _ = stmat.rms_norm(again[0].bfloat16(), dst="F8_E4M3")
    source.copy_(normal(9, 8, 1024, dtype=torch.bfloat16))
    x.copy_(source)
    want = chain()
    last = stmat.rms_norm(want[0].bfloat16(), dst="F8_E4M3")
    x.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((got, want), (again, want), ((y, s), last)):
        assert torch.equal(a[0].float(), b[0].float()) and torch.equal(a[1], b[1])


@gpu
def test_row_offsets_beyond_32_bits(stmat):
    """Rows that start more than 2^32 elements in, read and written."""
    rows, c, ld = 67, 520, 1 << 26
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    buf = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)
    x, w = normal(1, rows, c, dtype=torch.bfloat16), normal(2, c)
    for at in (0, 3):
        buf[:, at:at + c] = x
        want = norm64(x, None, w, 1e-5)[1]
        check_values(stmat.rms_norm(buf[:, at:at + c], w)[0], want)
        out = buf[:, 4096 + at:4096 + at + c]
        a = stmat.GatedActArgs(rows=rows, cols=c, act=1, x_dtype=10, y_dtype=10, gate=buf[:, at:].data_ptr(), ldg=ld,
                               y=out.data_ptr(), ldy=ld)
        stmat._check(stmat.lib().st_gated_act(a, torch.cuda.current_stream().cuda_stream))
        assert torch.equal(out, x.clamp_min(0))


# --------------------------------------------------------------- the example

@gpu
def test_scaled_fp8_mlp_example():
    """A checkpoint's MLP through the loader and the operators.  The 8-bit
    rounding moves a value by at most 2^-4 of itself, in the norm's rows (so in
    gate and up) and in the activation's: (1 + 2^-4)^3 - 1 of the result, and
    the BF16 roundings of z, the residual and the output next to it."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "scaled_fp8_mlp.py")
    spec = importlib.util.spec_from_file_location("scaled_fp8_mlp", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(hidden=1024, inter=2752, tokens=(1, 37, 700))
    assert set(found) == {1, 37, 700} and all(0 < v < (1 + 2.0 ** -4) ** 3 - 1 for v in found.values()), found


@gpu
def test_no_wait_gave_up(stmat):
    """After every other test of this file: the error word is clear."""
    assert stmat.static_check() == 0

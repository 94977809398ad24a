"""The operators on block-scaled FP8 (st_rms_norm_blocks, st_gated_act_blocks,
st_block_linear): refusals on the CPU, results on the GPU against the formulas
in 64 bits.

Tolerances are those of test_operators.py; a product's sum adds one
multiplication and one addition per block of 128 to the tensor core's, each
off by at most 2^-24 of the block's part or of the sum so far, and the product
of the two scales 2^-24 of it: (k + 3) 2^-23 sum |x' w'| covers them, with x'
and w' the scaled operands.  Integer inputs with scales of powers of two whose
sums stay under 2^24 units are exact and are compared bit for bit.
"""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

from test_operators import (ACTS, ROW, TYPES, act64, check_linear, check_values, norm64, normal, padded)  # noqa: E402

gpu = pytest.mark.gpu
BLOCK = 128


def blocks_of(n):
    return -(-n // BLOCK)


def spread(scales, *size):
    """Block scales for every element they stand for."""
    for d, n in zip((-2, -1), size):
        scales = scales.repeat_interleave(BLOCK, d).narrow(d, 0, n)
    return scales


def check_block_codes(codes, scales, want, slack=ROW):
    """8-bit codes and their scales against the values in 64 bits."""
    m, c = want.shape
    assert codes.shape == want.shape and scales.shape == (m, blocks_of(c))
    pad = torch.nn.functional.pad(want, (0, blocks_of(c) * BLOCK - c)).reshape(m, -1, BLOCK)
    top = (pad.abs().amax(2) / 448).clamp_min(2.0 ** -126)
    assert ((scales.double() - top).abs() <= 2 * slack * top).all()
    q = (want / scales.double().repeat_interleave(BLOCK, 1)[:, :c]).clamp(-448, 448)
    tol = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10)) * (1 + 2 * slack) + 2 * slack * q.abs()
    off = (codes.double() - q).abs()
    assert (off <= tol).all(), f"worst {(off / tol).max().item():.3g} of the tolerance"


# --------------------------------------------------------------- refusals

def norm_args(stmat, **kw):
    a = stmat.RmsNormArgs(rows=2, cols=200, eps=1e-5, x_dtype=10, w_dtype=10, y_dtype=13, x=1 << 20, ldx=200,
                          weight=2 << 20, y=3 << 20, ldy=200, scales=4 << 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def act_args(stmat, **kw):
    a = stmat.GatedActArgs(rows=2, cols=200, act=2, x_dtype=10, y_dtype=13, gate=1 << 20, ldg=200, up=2 << 20, ldu=200,
                           y=3 << 20, ldy=200, scales=4 << 20)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def linear_args(stmat, **kw):
    a = stmat.BlockLinearArgs(m=2, n=200, k=300, act=0, x_dtype=13, w_dtype=13, y_dtype=10, bias_dtype=11, x=1 << 20,
                              ldx=304, w=2 << 20, ldw=304, x_scale=4 << 20, ldxs=3, w_scale=5 << 20, ldws=3, y=3 << 20,
                              ldy=200)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


OPS = {"st_rms_norm_blocks": norm_args, "st_gated_act_blocks": act_args, "st_block_linear": linear_args}
REFUSED = [
    ("st_rms_norm_blocks", dict(y_dtype=10), "ST_E_DTYPE"), ("st_rms_norm_blocks", dict(y_dtype=14), "ST_E_DTYPE"),
    ("st_rms_norm_blocks", dict(scales=None), "ST_E_INVAL"), ("st_rms_norm_blocks", dict(scale=5 << 20), "ST_E_INVAL"),
    ("st_rms_norm_blocks", dict(scales=(4 << 20) + 2), "ST_E_ALIGN"), ("st_rms_norm_blocks", dict(x=None), "ST_E_INVAL"),
    ("st_rms_norm_blocks", dict(x_dtype=13), "ST_E_DTYPE"), ("st_rms_norm_blocks", dict(eps=-1.0), "ST_E_INVAL"),
    ("st_rms_norm_blocks", dict(h=5 << 20, ldh=200), "ST_E_INVAL"), ("st_rms_norm_blocks", dict(ldx=199), "ST_E_INVAL"),
    ("st_rms_norm_blocks", dict(cols=(1 << 27) + 1, ldx=1 << 28, ldy=1 << 28), "ST_E_INVAL"),
    ("st_gated_act_blocks", dict(act=5), "ST_E_INVAL"), ("st_gated_act_blocks", dict(y=None), "ST_E_INVAL"),
    ("st_gated_act_blocks", dict(scales=None), "ST_E_INVAL"), ("st_gated_act_blocks", dict(y_dtype=11), "ST_E_DTYPE"),
    ("st_gated_act_blocks", dict(ldu=199), "ST_E_INVAL"), ("st_gated_act_blocks", dict(up=(2 << 20) + 1), "ST_E_ALIGN"),
    ("st_block_linear", dict(x=None), "ST_E_INVAL"), ("st_block_linear", dict(w=None), "ST_E_INVAL"),
    ("st_block_linear", dict(y=None), "ST_E_INVAL"), ("st_block_linear", dict(x_scale=None), "ST_E_INVAL"),
    ("st_block_linear", dict(w_scale=None), "ST_E_INVAL"), ("st_block_linear", dict(ldxs=2), "ST_E_INVAL"),
    ("st_block_linear", dict(ldws=2), "ST_E_INVAL"), ("st_block_linear", dict(w_scale=(5 << 20) + 2), "ST_E_ALIGN"),
    ("st_block_linear", dict(x_dtype=14), "ST_E_DTYPE"), ("st_block_linear", dict(w_dtype=10), "ST_E_DTYPE"),
    ("st_block_linear", dict(x_dtype=10, w_dtype=10), "ST_E_DTYPE"), ("st_block_linear", dict(y_dtype=13), "ST_E_DTYPE"),
    ("st_block_linear", dict(m=-1), "ST_E_INVAL"), ("st_block_linear", dict(k=1 << 31), "ST_E_INVAL"),
    ("st_block_linear", dict(act=9), "ST_E_INVAL"), ("st_block_linear", dict(ldx=299), "ST_E_INVAL"),
    ("st_block_linear", dict(residual=6 << 20, ldr=199), "ST_E_INVAL"),
    ("st_block_linear", dict(bias=6 << 20, bias_dtype=13), "ST_E_DTYPE"),
    ("st_block_linear", dict(y=1 << 20), "ST_E_INVAL"), ("st_block_linear", dict(y=4 << 20), "ST_E_INVAL"),
    ("st_block_linear", dict(y=5 << 20), "ST_E_INVAL"), ("st_block_linear", dict(residual=(3 << 20) + 400, ldr=200), "ST_E_INVAL"),
    ("st_block_linear", dict(ldx=301), "ST_E_INVAL"),
    ("st_block_linear", dict(ldx=301, workspace=(6 << 20) + 8, workspace_bytes=4096), "ST_E_ALIGN"),
    ("st_block_linear", dict(ldx=301, workspace=4 << 20, workspace_bytes=4096), "ST_E_INVAL"),
]


@pytest.mark.parametrize("op,kw,status", REFUSED, ids=[f"{o[3:]}-{'-'.join(k)}-{i}" for i, (o, k, _) in enumerate(REFUSED)])
def test_refusals_queue_nothing(stmat, op, kw, status):
    a = OPS[op](stmat, **kw)
    assert stmat.STATUS[getattr(stmat.lib(), op)(C.byref(a), None)] == status
    assert op in stmat.lib().st_last_error().decode()


@pytest.mark.parametrize("op", OPS)
def test_null_arguments_and_empty_sizes(stmat, op):
    call = getattr(stmat.lib(), op)
    assert stmat.STATUS[call(None, None)] == "ST_E_INVAL"
    rows, cols = ("m", "n") if op == "st_block_linear" else ("rows", "cols")
    for kw in ({rows: 0}, {cols: 0}, {rows: 0, "y": None}):
        assert stmat.STATUS[call(C.byref(OPS[op](stmat, **kw)), None)] == "ST_OK"


def test_block_linear_workspace(stmat):
    call, need = stmat.lib().st_block_linear_workspace, C.c_uint64()
    for kw, want in ((dict(), 0), (dict(ldx=301), 2 * 304), (dict(ldw=301), 200 * 304), (dict(x=(1 << 20) + 1), 2 * 304),
                     (dict(m=1, ldx=301), 0), (dict(k=0), 0), (dict(n=0), 0)):
        a = linear_args(stmat, **kw)
        assert stmat.STATUS[call(C.byref(a), C.byref(need))] == "ST_OK"
        assert need.value == want, kw
    assert stmat.STATUS[call(None, C.byref(need))] == "ST_E_INVAL"
    assert stmat.STATUS[call(C.byref(a), None)] == "ST_E_INVAL"


def test_block_linear_forms(stmat):
    """Every choice is a form that exists; others are refused."""
    L = stmat.lib()
    for m in (1, 16, 17, 64, 65, 128, 129, 1000, 8192):
        for n, k in ((1, 1), (64, 4096), (14336, 4096), (4096, 14336), (100, 129)):
            kernel, width, splits = stmat.block_linear_choice(m, n, k)
            a = linear_args(stmat, m=m, n=n, k=k, ldx=16 * 1024, ldw=16 * 1024, ldxs=128, ldws=128, ldy=16 * 1024,
                            x=1 << 33, w=1 << 34, y=1 << 35, residual=1, ldr=16 * 1024)
            # A misaligned residual is refused before a form that exists is
            # looked at again, and one that does not exist after it.
            form = stmat.LinearForm(stmat.LINEAR_KERNELS.index(kernel), width, splits)
            assert stmat.STATUS[L.st_block_linear_as(C.byref(a), C.byref(form), None)] == "ST_E_ALIGN"
            assert splits <= max(1, blocks_of(k)) and (kernel == "split" or splits == 1)
    for form in ((0, 48, 1), (0, 16, 3), (0, 16, 16), (1, 32, 1), (1, 256, 2), (1, 320, 1), (2, 64, 1), (0, 16, 4), (0, 16, 0)):
        a = linear_args(stmat)
        assert stmat.STATUS[L.st_block_linear_as(C.byref(a), C.byref(stmat.LinearForm(*form)), None)] == "ST_E_INVAL", form
    assert stmat.STATUS[L.st_block_linear_as(C.byref(a), None, None)] == "ST_E_INVAL"
    out = stmat.LinearForm()
    for bad in ((None, 152, out), (a, 1, out), (linear_args(stmat, m=0), 152, out)):
        args = C.byref(bad[0]) if bad[0] is not None else None
        assert stmat.STATUS[L.st_block_linear_choose(args, bad[1], C.byref(bad[2]))] == "ST_E_INVAL"


def test_packed_arguments_have_the_structs_layout(stmat):
    n = len(stmat.BlockLinearArgs._fields_)
    got = stmat.BlockLinearArgs.from_buffer_copy(stmat._LINEAR_ARGS.pack(*range(1, n + 1)))
    assert [getattr(got, f) for f, _ in stmat.BlockLinearArgs._fields_] == list(range(1, n + 1))


@gpu
def test_binding_refusals(stmat):
    x, up = normal(1, 4, 256, dtype=torch.bfloat16), normal(2, 4, 256, dtype=torch.bfloat16)
    x8, w8 = x.to(torch.float8_e4m3fn), normal(3, 136, 256).to(torch.float8_e4m3fn)
    xs, ws = torch.ones(4, 2, device="cuda"), torch.ones(2, 2, device="cuda")
    for call, status in (
            (lambda: stmat.rms_norm(x, block=64, dst="F8_E4M3"), "ST_E_INVAL"),
            (lambda: stmat.rms_norm(x, block=128), "ST_E_INVAL"),
            (lambda: stmat.rms_norm(x, block=128, dst="F8_E4M3", scale=xs[0, :1]), "ST_E_INVAL"),
            (lambda: stmat.gated_act(x, up, block=128, dst="BF16"), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x8, w8, xs[:, :1], ws), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x8, w8, xs[:3], ws), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x8, w8, None, ws), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x8, w8, xs, None), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x8, w8, xs, ws[:1]), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x8, w8, xs.half(), ws), "ST_E_DTYPE"),
            (lambda: stmat.block_linear(x8, w8, xs.cpu(), ws), "ST_E_INVAL"),
            (lambda: stmat.block_linear(x, w8, xs, ws), "ST_E_DTYPE"),
            (lambda: stmat.block_linear(x8, w8, xs, ws, form=("dense", 256, 2)), "ST_E_INVAL")):
        with pytest.raises(stmat.StmatError) as e:
            call()
        assert e.value.status == status, e.value


# -------------------------------------------------------------------- rows

ROW_SIZES = [(1, 1), (3, 7), (9, 8), (17, 64), (5, 128), (4, 130), (300, 256), (33, 264), (1, 4096), (2, 5120), (7, 1111),
             (400, 1111), (300, 1000), (3, 12288), (2, 16381), (2, 16384), (1, 16392), (2, 17001), (1, 33000)]


@gpu
@pytest.mark.parametrize("m,c", ROW_SIZES)
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
def test_norm_blocks(stmat, m, c, dtype):
    dt = TYPES[dtype]
    x, r, w = normal(m + c, m, c, dtype=dt), normal(m + c + 1, m, c, dtype=dt), normal(3, c, dtype=dt)
    for residual, weight in ((r, w), (None, w), (r, None), (None, w.float())):
        y, scales, h = stmat.rms_norm(x, weight, eps=1e-5, residual=residual, dst="F8_E4M3", block=128)
        h64, y64 = norm64(x, residual, weight, 1e-5)
        check_block_codes(y, scales, y64)
        assert (h is None) == (residual is None)
        if h is not None:
            check_values(h, h64, slack=2.0 ** -23)


@gpu
@pytest.mark.parametrize("m", [2048, 2049])
@pytest.mark.parametrize("c", [1000, 1032, 2048, 2056, 4104])
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
def test_norm_blocks_of_many_rows(stmat, m, c, dtype):
    """To both sides of the number of rows from which a row has fewer threads."""
    x, w = normal(m + c, m, c, dtype=TYPES[dtype]), normal(3, c, dtype=TYPES[dtype])
    for residual in (None, x):
        y, scales, _ = stmat.rms_norm(x, w, residual=residual, dst="F8_E4M3", block=128)
        check_block_codes(y, scales, norm64(x, residual, w, 1e-5)[1])


@gpu
@pytest.mark.parametrize("m,c", ROW_SIZES)
@pytest.mark.parametrize("dtype", ["BF16", "F16", "F32"])
def test_gated_act_blocks(stmat, m, c, dtype):
    """Halves of one product's columns, whose rows start at odd places where
    the number of columns is odd."""
    both = normal(m + c, m, 2 * c, dtype=TYPES[dtype], spread=4.0)
    for act in ACTS if c in (8, 1111, 5120) else ("silu",):
        y, scales = stmat.gated_act(both[:, :c], both[:, c:], act=act, dst="F8_E4M3", block=128)
        check_block_codes(y, scales, act64(both[:, :c].double(), act) * both[:, c:].double(), slack=80 * 2.0 ** -23)
    y, scales = stmat.gated_act(both[:, :c], act="relu", dst="F8_E4M3", block=128)
    check_block_codes(y, scales, act64(both[:, :c].double(), "relu"))


@gpu
@pytest.mark.parametrize("m,c", [(3, 5), (9, 77), (4, 1111), (300, 2405), (2, 9001), (5, 520), (2, 20000), (300, 136)])
@pytest.mark.parametrize("extra,offset", [(0, 3), (2, 0), (5, 7), (8, 1), (8, 8)])
@pytest.mark.parametrize("dtype", ["BF16", "F32"])
def test_rows_anywhere(stmat, m, c, extra, offset, dtype):
    """Strides and addresses off every boundary, each matrix at its own; what
    lies outside the rows is neither written nor read into a value."""
    dt, code = TYPES[dtype], stmat.DTYPES.index(dtype)
    x, r, w = normal(1, m, c, dtype=dt), normal(2, m, c, dtype=dt), normal(3, c + 1, dtype=dt)[1:]
    xv, rv = padded(x, extra, offset), padded(r, extra + 1, offset + 2)
    yv = padded(torch.zeros_like(x).to(torch.float8_e4m3fn), extra + 2, offset + 1)
    hv = padded(torch.zeros_like(x), extra + 3, offset)
    scales = torch.full((m * blocks_of(c) + 1,), 5.0, device="cuda")
    a = stmat.RmsNormArgs(rows=m, cols=c, eps=1e-6, x_dtype=code, w_dtype=code, y_dtype=13, x=xv.data_ptr(), ldx=c + extra,
                          residual=rv.data_ptr(), ldr=c + extra + 1, weight=w.data_ptr(), h=hv.data_ptr(), ldh=c + extra + 3,
                          y=yv.data_ptr(), ldy=c + extra + 2, scales=scales.data_ptr())
    stmat._check(stmat.lib().st_rms_norm_blocks(a, torch.cuda.current_stream().cuda_stream))
    h64, y64 = norm64(x, r, w, 1e-6)
    check_values(hv, h64, slack=2.0 ** -23)
    check_block_codes(yv, scales[:-1].view(m, -1), y64)
    y2 = padded(torch.zeros_like(x).to(torch.float8_e4m3fn), extra + 2, offset + 1)
    b = stmat.GatedActArgs(rows=m, cols=c, act=0, x_dtype=code, y_dtype=13, gate=xv.data_ptr(), ldg=c + extra,
                           up=rv.data_ptr(), ldu=c + extra + 1, y=y2.data_ptr(), ldy=c + extra + 2, scales=scales.data_ptr())
    stmat._check(stmat.lib().st_gated_act_blocks(b, torch.cuda.current_stream().cuda_stream))
    check_block_codes(y2, scales[:-1].view(m, -1), x.double() * r.double())
    assert scales[-1] == 5.0
    for v, e, o in ((yv, extra + 2, offset + 1), (y2, extra + 2, offset + 1), (hv, extra + 3, offset)):
        flat = v._base.reshape(-1).float()
        inside = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
        inside[o:o + m * (c + e)].view(m, c + e)[:, :c] = True
        assert (flat[~inside] == torch.tensor(77.0).to(v.dtype).float().item()).all()


@gpu
def test_special_rows(stmat):
    """Zero blocks, the smallest numbers, NaN and infinities, which stay in
    their row (norm) or block (activation)."""
    c = 512
    x = normal(5, 6, c, dtype=torch.bfloat16)
    x[0] = 0
    x[1, :128] = 2.0 ** -130
    x[2, 17] = math.nan
    x[3, 5] = math.inf
    x[4, 400] = -math.inf
    y, scales = stmat.gated_act(x, act="none", dst="F8_E4M3", block=128)
    assert (y[0].float() == 0).all() and (scales[0] == 2.0 ** -126).all()
    assert scales[1, 0] == 2.0 ** -126
    check_block_codes(y[1:2], scales[1:2], x[1:2].double())
    for row, at in ((2, 17), (3, 5), (4, 400)):
        b = at // 128
        keep = [i for i in range(4) if i != b]
        assert not torch.isfinite(scales[row, b]) and torch.isnan(y[row, at].float())
        cols = torch.cat([torch.arange(128 * i, 128 * i + 128) for i in keep]).cuda()
        check_block_codes(y[row:row + 1, cols], scales[row:row + 1, keep], x[row:row + 1, cols].double())
    w = torch.ones(c, dtype=torch.bfloat16, device="cuda")
    y, scales, _ = stmat.rms_norm(x, w, dst="F8_E4M3", block=128)
    assert (y[0].float() == 0).all() and (scales[0] == 2.0 ** -126).all()
    assert torch.isnan(scales[2]).all() and torch.isnan(y[2].float()).all()
    assert torch.isnan(y[3, 5].float()) and (y[3, 128:].float() == 0).all() and (scales[3, 1:] == 2.0 ** -126).all()
    check_block_codes(y[5:], scales[5:], norm64(x, None, w, 1e-5)[1][5:])


@gpu
def test_row_shapes_and_in_place(stmat):
    x, w = normal(2, 2, 3, 200), normal(1, 200)
    y, scales, h = stmat.rms_norm(x, w, residual=x[0, 0].expand(2, 3, 200), dst="F8_E4M3", block=128)
    assert y.shape == x.shape == h.shape and scales.shape == (2, 3, 2)
    check_block_codes(y.view(6, 200), scales.view(6, 2), norm64(x, x[0, 0].expand(2, 3, 200), w, 1e-5)[1].view(6, 200))
    assert stmat.rms_norm(x[0, 0], w, dst="F8_E4M3", block=128)[1].shape == (2,)
    assert stmat.rms_norm(x[:0], w, dst="F8_E4M3", block=128)[1].shape == (0, 3, 2)
    assert stmat.gated_act(x[..., :0], dst="F8_E4M3", block=128)[1].shape == (2, 3, 0)
    for c in (768, 771, 33000, 33001):
        x, r, w = (normal(i, *s, dtype=torch.bfloat16) for i, s in enumerate([(300 if c < 999 else 9, c)] * 2 + [(c,)]))
        m = x.shape[0]
        h64, y64 = norm64(x, r, w, 1e-5)
        y = torch.empty(m, c, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(m, blocks_of(c), device="cuda")
        a = stmat.RmsNormArgs(rows=m, cols=c, eps=1e-5, x_dtype=10, w_dtype=10, y_dtype=13, x=x.data_ptr(), ldx=c,
                              residual=r.data_ptr(), ldr=c, weight=w.data_ptr(), h=r.data_ptr(), ldh=c,
                              y=y.data_ptr(), ldy=c, scales=scales.data_ptr())
        stmat._check(stmat.lib().st_rms_norm_blocks(a, torch.cuda.current_stream().cuda_stream))
        check_values(r, h64, slack=2.0 ** -23)
        check_block_codes(y, scales, y64)


# ----------------------------------------------------------------- product

def product64(x, w, xs, ws, bias=None, act="none", r=None):
    """(y in 64 bits, what the sum may be off by)."""
    xd = x.double() * xs.double().repeat_interleave(BLOCK, 1)[:, :x.shape[1]]
    wd = w.double() * spread(ws.double(), *w.shape)
    s = xd @ wd.t()
    slack = 1.13 * (xd.abs() @ wd.abs().t()) * ((x.shape[1] + 3) * 2.0 ** -23)
    if bias is not None:
        s = s + bias.double()
        slack = slack + 2.0 ** -22 * bias.double().abs()
    y = act64(s, act)
    slack = slack + (2.0 ** -20 * s.abs() if act != "none" else 0)
    return (y if r is None else y + r.double()), slack


def operands(m, n, k, wt="F8_E4M3", seed=0):
    x, w = normal(seed + m, m, k, dtype=torch.float8_e4m3fn), normal(seed + n + 1, n, k, dtype=TYPES[wt], spread=0.5)
    xs = normal(seed + 2, m, blocks_of(k)).abs() * 0.1 + 0.01
    ws = normal(seed + 3, blocks_of(n), blocks_of(k)).abs() * 0.1 + 0.01
    return x, w, xs, ws


SIZES = [(1, 1, 1), (1, 8, 16), (1, 300, 257), (3, 128, 64), (2, 1, 512), (16, 129, 40), (17, 256, 1000), (33, 1111, 72),
         (65, 64, 2048), (100, 391, 333), (128, 257, 384), (129, 257, 130), (200, 512, 4096), (300, 96, 8), (257, 640, 768),
         (520, 1000, 520), (1, 2048, 8192), (7, 4104, 1544), (768, 512, 128), (513, 257, 1040), (1111, 2000, 80),
         (600, 33, 4096), (2560, 2592, 272), (777, 1, 16)]
FORMS = [("split", w, s) for w in (16, 32, 64, 128) for s in (1, 2, 8)] + [("dense", w, 1) for w in (64, 128, 192, 256)]


@gpu
@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("wt", ["F8_E4M3", "F8_E5M2"])
def test_block_linear_values(stmat, m, n, k, wt):
    x, w, xs, ws = operands(m, n, k, wt)
    y = stmat.block_linear(x, w, xs, ws, dst="F32")
    want, slack = product64(x, w, xs, ws)
    check_linear(y, want, slack)
    assert torch.equal(y, stmat.block_linear(x, w, xs, ws, dst="F32"))    # the same bits again
    y = stmat.block_linear(x, w, xs, ws)
    assert y.dtype == torch.bfloat16
    check_linear(y, want, slack)


def integers(seed, m, n, k):
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randint(-3, 4, (m, k), generator=g).float(), torch.randint(-3, 4, (n, k), generator=g).float()
    xs = 2.0 ** torch.randint(-1, 2, (m, blocks_of(k)), generator=g).float()
    ws = 2.0 ** torch.randint(-1, 2, (blocks_of(n), blocks_of(k)), generator=g).float()
    y = (x.double() * xs.double().repeat_interleave(BLOCK, 1)[:, :k]) @ (w.double() * spread(ws.double(), n, k)).t()
    return x.to(torch.float8_e4m3fn).cuda(), w.to(torch.float8_e4m3fn).cuda(), xs.cuda(), ws.cuda(), y


@gpu
@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(map(str, f)))
def test_every_form_is_exact(stmat, form):
    """Ragged and whole tiles, several rounds of tiles, in every form: integers
    and scales of powers of two, so that any order gives the same bits."""
    for m, n, k in ((1, 130, 1024), (37, 300, 1030), (130, 391, 2000), (300, 520, 1153), (1500, 4100, 1024)):
        if form[0] == "split" and m > 300:
            continue
        x, w, xs, ws, want = integers(m + n + k, m, n, k)
        y = stmat.block_linear(x, w, xs, ws, dst="F32", form=form)
        assert torch.equal(y.cpu().double(), want), (m, n, k)


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(1, 200, 136), (5, 328, 64), (40, 130, 96), (128, 391, 300), (150, 391, 300), (300, 520, 128),
                                   (600, 544, 256), (530, 391, 64)])
def test_block_linear_epilogue(stmat, m, n, k, act):
    for wt, dst, bt in (("F8_E4M3", "BF16", "BF16"), ("F8_E5M2", "F16", "F32"), ("F8_E4M3", "F32", "F16")):
        x, w, xs, ws = operands(m, n, k, wt, seed=7)
        b, r = normal(10, n, dtype=TYPES[bt]), normal(11, m, n, dtype=TYPES[dst])
        for bias, residual in ((b, r), (b, None), (None, r)):
            y = stmat.block_linear(x, w, xs, ws, bias, act, residual, dst)
            want, slack = product64(x, w, xs, ws, bias, act, residual)
            check_linear(y, want, slack + 2.0 ** -20 * (want - (residual.double() if residual is not None else 0)).abs())


@gpu
@pytest.mark.parametrize("m,n,k", [(1, 72, 64), (6, 200, 128), (130, 264, 256), (300, 300, 100), (515, 304, 192)])
@pytest.mark.parametrize("extra,offset", [(16, 0), (16, 16), (1, 0), (0, 1), (7, 3)])
def test_block_linear_strides(stmat, m, n, k, extra, offset):
    """Row strides of every operand, addresses off 16-byte boundaries, and no
    write outside y."""
    x, w, xs, ws = operands(m, n, k)
    r = normal(5, m, n, dtype=torch.bfloat16)
    xv, wv, rv = padded(x, extra, offset), padded(w, extra, offset), padded(r, extra + 1, offset + 1)
    yv = padded(torch.zeros_like(r), extra, offset)
    stmat.block_linear(xv, wv, padded(xs, 3, 1), padded(ws, 2, 5), residual=rv, out=yv)
    want, slack = product64(x, w, xs, ws, r=r)
    check_linear(yv, want, slack)
    flat = yv._base.reshape(-1).float()
    inside = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
    inside[offset:offset + m * (n + extra)].view(m, n + extra)[:, :n] = True
    assert (flat[~inside] == torch.tensor(77.0).bfloat16().float().item()).all()


@gpu
def test_block_linear_sizes_of_zero_and_shapes(stmat):
    x, w, xs, ws = operands(6, 200, 256)
    b = normal(4, 200)
    y = stmat.block_linear(x[:, :0], w[:, :0], xs[:, :0], ws[:, :0], bias=b, dst="F32")
    assert torch.equal(y, b.expand(6, 200))
    assert stmat.block_linear(x[:0], w, xs[:0], ws).shape == (0, 200)
    assert stmat.block_linear(x, w[:0], xs, ws[:0]).shape == (6, 0)
    y = stmat.block_linear(x.view(2, 3, 256), w, xs.view(2, 3, 2), ws, dst="F32")
    assert torch.equal(y.view(6, 200), stmat.block_linear(x, w, xs, ws, dst="F32"))
    one = torch.full((1, 1), 0.25, device="cuda")
    y = stmat.block_linear(x, w, one.expand(6, 2), one.expand(2, 2), dst="F32")
    want, slack = product64(x, w, one.expand(6, 2), one.expand(2, 2))
    check_linear(y, want, slack)
    y = stmat.block_linear(x, w, xs[:1].expand(6, 2), ws[:1].expand(2, 2), dst="F32")
    want, slack = product64(x, w, xs[:1].expand(6, 2), ws[:1].expand(2, 2))
    check_linear(y, want, slack)


@gpu
@pytest.mark.parametrize("m", [1, 20, 100, 300])
def test_block_linear_residual_in_place(stmat, m):
    x, w, xs, ws = operands(m, 1000, 512)
    r = normal(5, m, 1000, dtype=torch.bfloat16)
    want = stmat.block_linear(x, w, xs, ws, residual=r)
    stmat.block_linear(x, w, xs, ws, residual=r, out=r)
    assert torch.equal(r, want)


@gpu
@pytest.mark.parametrize("m,n,k", [(5, 300, 400), (300, 520, 640)])
def test_block_linear_nan_and_infinity(stmat, m, n, k):
    """A NaN code, a NaN or infinite scale: in the products they enter alone."""
    x, w, xs, ws = operands(m, n, k)
    clean = stmat.block_linear(x, w, xs, ws, dst="F32")
    x[2, 129], xs[3, 1], ws[1, 0] = math.nan, math.inf, math.nan
    y = stmat.block_linear(x, w, xs, ws, dst="F32")
    hit = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    hit[2], hit[3], hit[:, 128:256] = True, True, True
    assert torch.equal(y[~hit], clean[~hit])
    assert not torch.isfinite(y[hit]).any() and torch.isnan(y[2]).all() and torch.isnan(y[:, 128:256]).all()


@gpu
def test_a_block_scaled_mlp_on_another_stream_and_in_a_graph(stmat):
    """The operators in a row, as a layer runs them, eagerly, on a stream of
    their own and replayed with new inputs; against 64 bits with the same
    roundings of the rows."""
    m, c, i = 37, 512, 1100
    w1, s1 = operands(1, 2 * i, c)[1::2]
    w2, s2 = operands(1, c, i)[1::2]
    norm = normal(4, c, dtype=torch.bfloat16)

    def layer(x, r):
        y8, s, h = stmat.rms_norm(x, norm, residual=r, dst="F8_E4M3", block=128)
        z = stmat.block_linear(y8, w1, s, s1)
        a8, t = stmat.gated_act(z[:, :i], z[:, i:], act="silu", dst="F8_E4M3", block=128)
        return y8, s, h, z, a8, t, stmat.block_linear(a8, w2, t, s2, residual=h)

    x, r = normal(5, m, c, dtype=torch.bfloat16), normal(6, m, c, dtype=torch.bfloat16)
    y8, s, h, z, a8, t, out = layer(x, r)
    check_block_codes(y8, s, norm64(x, r, norm, 1e-5)[1])
    want, slack = product64(y8, w1, s, s1)
    check_linear(z, want, slack)
    check_block_codes(a8, t, act64(z[:, :i].double(), "silu") * z[:, i:].double(), slack=80 * 2.0 ** -23)
    want, slack = product64(a8, w2, t, s2, r=h)
    check_linear(out, want, slack)
    eager = [v.clone() for v in (y8, s, h, z, a8, t, out)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(x, r)
    side.synchronize()
    for a, b in zip(got, eager):
        assert torch.equal(a.float(), b.float())
    x2, r2 = normal(7, m, c, dtype=torch.bfloat16), normal(8, m, c, dtype=torch.bfloat16)
    after = [v.clone() for v in layer(x2, r2)]
    gx, gr = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(gx, gr)
    for source, want in (((x, r), eager), ((x2, r2), after), ((x, r), eager)):
        gx.copy_(source[0])
        gr.copy_(source[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.float(), b.float())


@gpu
def test_no_wait_gave_up(stmat):
    torch.cuda.synchronize()
    assert stmat.static_check() == 0

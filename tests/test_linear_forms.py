"""Every form of a product (st_linear_form: kernel, width of a tile, parts of
the sum) on purpose, with the whole epilogue, and which form st_linear takes.

Integers whose sums stay under 2^24, scales that are powers of two: every step
of the sum and of the epilogue up to its rounding is exact in binary32, whatever
the order, so results are compared bit for bit.  Activations are compared with
64 bits within the header's bound, (2 |e| + 6) 2^-23 of the value, e the
exponential's argument, and the rounding of the output."""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu
TYPES = {"BF16": torch.bfloat16, "F16": torch.float16, "F32": torch.float32, "F8_E4M3": torch.float8_e4m3fn,
         "F8_E5M2": torch.float8_e5m2}
U = {"BF16": 2.0 ** -8, "F16": 2.0 ** -11, "F32": 2.0 ** -24}
PAIRS = [("BF16", "BF16"), ("F16", "F16"), ("F8_E4M3", "F8_E4M3"), ("F8_E4M3", "F8_E5M2")]
FORMS = [("split", w, s) for w in (16, 32, 64, 128) for s in (1, 2, 4, 8)]
FORMS += [("dense", w, s) for s in (1, 2, 4) for w in range(32, 257, 32) if w % (32 * s) == 0]
ids = ["-".join(map(str, f)) for f in FORMS]


# ------------------------------------------------------------- on the host

# (m, n, k, dtype of the weight) and the form on a GB300.
CHOSEN = [
    ((1, 14336, 4096, "F8_E4M3"), ("split", 16, 2)), ((8, 4096, 14336, "BF16"), ("split", 16, 8)),
    ((1, 300, 1024, "BF16"), ("split", 16, 4)), ((17, 300, 2048, "BF16"), ("split", 32, 8)),
    ((40, 14336, 4096, "BF16"), ("split", 64, 2)), ((65, 64, 4096, "BF16"), ("split", 128, 8)),
    ((65, 8192, 8192, "BF16"), ("split", 128, 4)), ((256, 4096, 4096, "F8_E4M3"), ("dense", 64, 1)),
    ((200, 512, 4096, "F8_E4M3"), ("dense", 64, 2)), ((600, 512, 4096, "BF16"), ("dense", 128, 4)),
    ((256, 4096, 14336, "BF16"), ("dense", 128, 2)), ((600, 2048, 4096, "BF16"), ("dense", 192, 2)),
    ((600, 1024, 8192, "BF16"), ("dense", 256, 4)), ((200, 8192, 8192, "BF16"), ("dense", 256, 2)),
    ((8192, 14336, 4096, "F8_E4M3"), ("dense", 256, 1)), ((4096, 4096, 14336, "BF16"), ("dense", 224, 1)),
    ((600, 2048, 64, "BF16"), ("dense", 96, 1)), ((8192, 300, 64, "BF16"), ("dense", 160, 1)),
    ((1, 300, 257, "BF16"), ("split", 16, 1)), ((16, 304, 256, "BF16"), ("dense", 32, 1)), ((5, 7, 0, "BF16"), ("split", 16, 1)),
]


@pytest.mark.parametrize("size,form", CHOSEN, ids=["x".join(map(str, s)) for s, _ in CHOSEN])
def test_the_form_taken_on_a_gb300(stmat, size, form):
    assert stmat.linear_choice(*size) == form
    assert form in FORMS


def test_a_few_tokens_take_the_kernel_for_them(stmat):
    """However short the sum, and however many weight rows."""
    for m in (1, 2, 5, 8):
        for n in (1, 64, 300, 1024, 4096, 14336, 28672, 100000):
            for k in (1, 64, 100, 256, 512, 1000, 4096, 14336):
                for dtype in ("BF16", "F8_E4M3"):
                    assert stmat.linear_choice(m, n, k, dtype)[:2] == ("split", 16), (m, n, k, dtype)


def test_the_form_fits_any_device(stmat):
    """Whatever the device, a form that exists; no shared sum without room for
    its clusters."""
    for sms, clusters in ((2, (0, 0)), (132, (30, 12)), (152, (0, 0)), (152, (36, 15)), (160, (40, 20))):
        for m in (1, 16, 33, 64, 100, 257, 700, 5000):
            for n in (1, 100, 1000, 4096, 30000):
                for k in (1, 64, 700, 4096, 20000):
                    for dtype in ("BF16", "F8_E5M2"):
                        form = stmat.linear_choice(m, n, k, dtype, sms, clusters)
                        assert form in FORMS
                        if form[0] == "dense" and form[2] > 1:
                            tiles = -(-m // 256) * -(-n // form[1])
                            assert tiles <= clusters[form[2] == 4]


@pytest.mark.parametrize("form", [(0, 24, 1), (0, 256, 1), (0, 0, 1), (0, 16, 3), (0, 16, 16), (0, 16, 0), (1, 16, 1),
                                  (1, 288, 1), (1, 48, 1), (1, 32, 2), (1, 96, 2), (1, 96, 4), (1, 256, 8), (1, 128, 3),
                                  (2, 32, 1), (-1, 32, 1), (0, 16, 8), (1, 256, 4)])
def test_forms_that_do_not_exist_are_refused(stmat, form):
    """(The last two: a sum of two runs of 128 bytes in more parts.)"""
    at = 1 << 20
    a = stmat.LinearArgs(m=2, n=8, k=128, x_dtype=10, w_dtype=10, y_dtype=10, x=at, ldx=128, w=2 * at, ldw=128, y=3 * at, ldy=8)
    L = stmat.lib()
    assert stmat.STATUS[L.st_linear_as(C.byref(a), C.byref(stmat.LinearForm(*form)), None)] == "ST_E_INVAL"


def test_form_entry_points_refuse_what_st_linear_does(stmat):
    at = 1 << 20
    a = stmat.LinearArgs(m=2, n=8, k=128, x_dtype=10, w_dtype=10, y_dtype=10, x=at, ldx=128, w=2 * at, ldw=128, y=3 * at, ldy=8)
    L, form = stmat.lib(), stmat.LinearForm(0, 16, 1)

    def as_(args, f):
        return stmat.STATUS[L.st_linear_as(args and C.byref(args), f and C.byref(f), None)]

    def choose(args, f, *device):
        return stmat.STATUS[L.st_linear_choose(args and C.byref(args), *device, f and C.byref(f))]

    assert choose(a, form, 152, 36, 15) == "ST_OK" and as_(a, None) == as_(None, form) == "ST_E_INVAL"
    assert choose(None, form, 152, 36, 15) == choose(a, None, 152, 36, 15) == choose(a, form, 1, 0, 0) == "ST_E_INVAL"
    a.ldx = 5
    assert as_(a, form) == choose(a, form, 152, 36, 15) == "ST_E_INVAL"
    a.ldx, a.k = 128, 0
    assert as_(a, stmat.LinearForm(1, 32, 1)) == "ST_E_INVAL"  # the dense kernel has no empty sums
    a.m = 0
    assert as_(a, form) == "ST_OK" and choose(a, form, 152, 36, 15) == "ST_E_INVAL"


# ------------------------------------------------------------- on the GPU

def sizes(form):
    """Fewer rows and columns than a tile, several tiles and a ragged rest."""
    kernel, width, _ = form
    if kernel == "split":
        return [(max(1, width - 3), 133), (2 * width + 1, 300), (width, 256)]
    return [(269, 2 * width + 7), (512, width), (100, width - 9)]


def integers(seed, m, n, k, xt, wt):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-3, 4, (m, k), generator=g, device="cuda").float()
    w = torch.randint(-3, 4, (n, k), generator=g, device="cuda").float()
    b = torch.randint(-50, 51, (n,), generator=g, device="cuda").float()
    r = torch.randint(-100, 101, (m, n), generator=g, device="cuda").float()
    xs = 2.0 ** torch.randint(-3, 2, (m,), generator=g, device="cuda").float()
    ws = 2.0 ** torch.randint(-3, 2, (n,), generator=g, device="cuda").float()
    return x, w, b, r, xs, ws


def placed(t, extra, offset):
    """t in a larger buffer of 77s: `extra` columns between rows, `offset`
    elements before the first."""
    m, c = t.shape
    buf = torch.full((offset + m * (c + extra) + 64,), 77.0, device="cuda").to(t.dtype)
    v = buf[offset:offset + m * (c + extra)].view(m, c + extra)[:, :c]
    v.copy_(t)
    return v


def untouched(v, extra, offset):
    m, c = v.shape
    flat = v._base.reshape(-1).float()
    outside = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    outside[offset:offset + m * (c + extra)].view(m, c + extra)[:, :c] = False
    return bool((flat[outside] == 77).all())


@gpu
@pytest.mark.parametrize("xt,wt", PAIRS)
@pytest.mark.parametrize("form", FORMS, ids=ids)
def test_every_form_is_exact(stmat, form, xt, wt):
    """Scales, bias and residual of each kind, rows on and off boundaries of 32
    bytes, y in place of the residual; nothing outside y is written."""
    item = TYPES[xt].itemsize
    for i, (m, n) in enumerate(sizes(form)):
        # 9 runs of 128 bytes and some; rows off 16 bytes are copied first
        k = (9 * 128 + (16, 48, 0)[i]) // item + (0, 5 if item == 1 else 3, 0)[i]
        x, w, b, r, xs, ws = integers(m + n, m, n, k, xt, wt)
        total = (x @ w.t()).double()
        xd, wd = x.to(TYPES[xt]), w.to(TYPES[wt])
        dst = ("F32", "BF16", "F16")[i]
        y = stmat.linear(xd, wd, dst="F32", form=form)
        assert torch.equal(y.double(), total)
        for extra, offset, act in ((0, 0, "none"), (9, 1, "relu"), (32, 32, "none"), (0, 3, "relu")):
            for scales, bt in (((xs, ws), "F32"), ((xs[:1], ws), dst), ((xs, ws[:1]), "BF16"), ((None, None), None)):
                sx, sw = scales
                want = total if sx is None else total * sx.double()[:, None] * sw.double()[None]
                if bt:
                    want = want + b.double()
                if act == "relu":
                    want = want.clamp_min(0)
                want = (want + r.double()).float().to(TYPES[dst])
                rv = placed(r.to(TYPES[dst]), extra, offset)
                got = stmat.linear(xd, wd, x_scale=sx, w_scale=sw, bias=b.to(TYPES[bt]) if bt else None, act=act,
                                   residual=rv, out=rv, form=form)
                assert got is rv and torch.equal(rv, want), (m, n, k, extra, offset, bt)
                assert untouched(rv, extra, offset)
        # a residual of its own, and one row for all
        yv = placed(torch.zeros_like(r).to(TYPES[dst]), 5, 7)
        for res in (placed(r.to(TYPES[dst]), 2, 4), r[:1].to(TYPES[dst]).expand(m, n)):
            stmat.linear(xd, wd, residual=res, out=yv, form=form)
            assert torch.equal(yv, (total + res.double()).float().to(TYPES[dst])) and untouched(yv, 5, 7)


@gpu
@pytest.mark.parametrize("m", [700, 2600])
@pytest.mark.parametrize("width", range(32, 257, 32))
def test_dense_tiles_in_several_rounds(stmat, width, m):
    """More tiles than pairs of CTAs: each pair takes two or more in turn, in
    alternating halves of TMEM."""
    n = (27 if m == 700 else 17) * width + 13
    for xt, wt, k in (("BF16", "BF16", 264), ("F8_E4M3", "F8_E5M2", 400)):
        x, w, b, r, xs, ws = integers(m + width, m, n, k, xt, wt)
        want = ((x @ w.t()).double() * xs.double()[:, None] * ws.double() + b.double() + r.double()).float()
        for dst in ("BF16", "F32"):
            y = stmat.linear(x.to(TYPES[xt]), w.to(TYPES[wt]), xs, ws, b.bfloat16(), "none", r.to(TYPES[dst]), dst,
                             form=("dense", width, 1))
            assert torch.equal(y, want.to(TYPES[dst]))


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("form", FORMS, ids=ids)
def test_every_form_activates(stmat, form, act):
    """Sums between -9 and 9 that are exact: the activation's error and the
    output's rounding are all there is."""
    for i, (m, n) in enumerate(sizes(form)):
        for xt, dst in (("F8_E4M3", "BF16"), ("BF16", "F32"), ("F16", "F16")):
            k = 9 * 128 // TYPES[xt].itemsize
            x, w, b, r, xs, ws = integers(i, m, n, k, xt, xt)
            xs, ws = xs * 2.0 ** -5, ws * 2.0 ** -2
            v = ((x @ w.t()).double() * xs.double()[:, None] * ws.double() + b.double() / 16).clamp(-1e3, 1e3)
            if act == "gelu":
                value, e = v * torch.special.erfc(-v * math.sqrt(0.5)) / 2, v * v / 2
            else:
                e = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
                value, e = v * torch.special.expit(e), e.abs()
            own = (2 * e + 7) * 2.0 ** -23 * value.abs() + 2.0 ** -126 * v.abs()
            for residual in (None, r.to(TYPES[dst])):
                want = value if residual is None else value + residual.double()
                y = stmat.linear(x.to(TYPES[xt]), w.to(TYPES[xt]), xs, ws, b / 16, act, residual, dst, form=form)
                tol = own + (U[dst] + 2.0 ** -23) * (want.abs() + own) + (2.0 ** -25 if dst == "F16" else 0)
                assert ((y.double() - want).abs() <= tol).all(), (m, n, xt)


@gpu
@pytest.mark.parametrize("form", FORMS, ids=ids)
def test_every_form_keeps_nan_and_infinity_apart(stmat, form):
    """They stay in their row and column, in every part of the sum."""
    for m, n in sizes(form)[:2]:
        k = 9 * 64 + 8
        x, w, *_ = integers(7, m, n, k, "BF16", "BF16")
        x[m // 2, k - 1] = math.nan
        x[0, 3] = math.inf
        w[n // 3, k // 2] = -math.inf
        w[:, 3] = 1
        x[:, k // 2] = 1
        y = stmat.linear(x.bfloat16(), w.bfloat16(), dst="F32", form=form)
        want = x.double() @ w.double().t()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(y.double(), nan=0.0, posinf=1e9, neginf=-1e9),
                           torch.nan_to_num(want, nan=0.0, posinf=1e9, neginf=-1e9))


@gpu
@pytest.mark.parametrize("form", FORMS, ids=ids)
def test_forms_on_a_busy_gpu_and_in_a_graph(stmat, form):
    """A chain of products (each starts while the one before it ends), beside
    work on another stream, captured and replayed."""
    m = sizes(form)[1][0]
    x = torch.eye(m, 640, device="cuda").bfloat16()
    w = torch.roll(torch.eye(640, device="cuda"), 1, 0).bfloat16()
    x[:, 5] += 3
    want = torch.roll(x, 4, 1)
    side, noise = torch.cuda.Stream(), torch.zeros(1 << 24, device="cuda")

    def chain(y):
        for _ in range(4):
            y = stmat.linear(y, w, form=form)
        return y

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            noise.add_(1)
    assert torch.equal(chain(x), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(x)
    for _ in range(3):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@gpu
def test_no_wait_gave_up_in_any_form(stmat):
    assert stmat.static_check() == 0

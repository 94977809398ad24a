"""The mixture-of-experts layer (st_moe): refusals on the CPU, results on the
GPU against the formulas in 64 bits.

Tolerances.  With A = sum |x w| and B = sum over runs of 128 of (largest |x| of
the run) sum |w|: a product's sum is off by (k + 3) 2^-23 A (test_operators.py,
and one addition a block), and by 2^-21 B where its operand goes in columns of
eight bits; h's columns hold 2^-12 of a value.  The activation, its product with
up and with p, which is within 64 2^-24 (expf's ulps, |l - largest l| 2^-24 of
its argument, a sum and a division), add 2^-17 of h.  These go through the
formulas with the activation's largest slope (1.13), then into down's sum.
"""
import ctypes as C
import math

import pytest

torch = pytest.importorskip("torch")

from test_block_operators import blocks_of, spread  # noqa: E402
from test_operators import TYPES, act64, check_values, normal, padded  # noqa: E402

gpu = pytest.mark.gpu
P = 64 * 2.0 ** -24


# --------------------------------------------------------------- refusals

def moe_args(stmat, **kw):
    E, H, I, T, K = 8, 256, 384, 5, 2
    w = stmat.MoeWeight
    a = stmat.MoeArgs(tokens=T, hidden=H, inter=I, experts=E, top_k=K, act=2, score=0, normalize=1, factor=1.0, x_dtype=10,
                      router_dtype=10, w_dtype=13, y_dtype=10, x=1 << 20, ldx=H, router=2 << 20, ld_router=H,
                      gate=w(16 << 20, I * H, H, 3 << 20, 6, 2, 1), up=w(32 << 20, I * H, H, (3 << 20) + 4096, 6, 2, 1),
                      down=w(48 << 20, I * H, I, (3 << 20) + 8192, 6, 3, 1), y=4 << 20, ldy=H, chosen=5 << 20,
                      weights=6 << 20, workspace=64 << 20, workspace_bytes=1 << 20)
    for k, v in kw.items():
        part, _, field = k.partition("__")
        setattr(getattr(a, part) if field else a, field or k, v)
    return a


REFUSED = [
    (dict(tokens=65), "ST_E_INVAL"), (dict(tokens=-1), "ST_E_INVAL"), (dict(hidden=0), "ST_E_INVAL"), (dict(inter=0), "ST_E_INVAL"),
    (dict(hidden=(1 << 24) + 1), "ST_E_INVAL"), (dict(experts=0), "ST_E_INVAL"), (dict(experts=1025), "ST_E_INVAL"),
    (dict(top_k=0), "ST_E_INVAL"), (dict(top_k=9), "ST_E_INVAL"), (dict(experts=40, top_k=33), "ST_E_INVAL"),
    (dict(act=7), "ST_E_INVAL"), (dict(score=2), "ST_E_INVAL"), (dict(x_dtype=11), "ST_E_DTYPE"), (dict(x_dtype=13), "ST_E_DTYPE"),
    (dict(router_dtype=13), "ST_E_DTYPE"), (dict(w_dtype=9), "ST_E_DTYPE"), (dict(w_dtype=11), "ST_E_DTYPE"),
    (dict(y_dtype=13), "ST_E_DTYPE"), (dict(x=None), "ST_E_INVAL"), (dict(router=None), "ST_E_INVAL"), (dict(y=None), "ST_E_INVAL"),
    (dict(ldx=255), "ST_E_INVAL"), (dict(ld_router=255), "ST_E_INVAL"), (dict(ldy=100), "ST_E_INVAL"),
    (dict(x=(1 << 20) + 1), "ST_E_ALIGN"), (dict(router_bias=(7 << 20) + 2), "ST_E_ALIGN"), (dict(chosen=(5 << 20) + 2), "ST_E_ALIGN"),
    (dict(gate__w=None), "ST_E_INVAL"), (dict(down__w=None), "ST_E_INVAL"), (dict(gate__scale=None), "ST_E_INVAL"),
    (dict(up__scale=None), "ST_E_INVAL"), (dict(down__scale=(3 << 20) + 2), "ST_E_ALIGN"), (dict(gate__w=(16 << 20) + 8), "ST_E_ALIGN"),
    (dict(gate__ld=264), "ST_E_INVAL"), (dict(gate__ld=264, gate__expert=264 * 384), "ST_E_ALIGN"), (dict(up__ld=255), "ST_E_INVAL"),
    (dict(down__expert=8), "ST_E_INVAL"), (dict(down__expert=384 * 256 + 8), "ST_E_ALIGN"), (dict(gate__scale_row=-1), "ST_E_INVAL"),
    (dict(w_dtype=10), "ST_E_INVAL"), (dict(residual=8 << 20, ldr=255), "ST_E_INVAL"),
    (dict(workspace=None), "ST_E_INVAL"), (dict(workspace_bytes=1000), "ST_E_INVAL"), (dict(workspace=(64 << 20) + 16), "ST_E_ALIGN"),
    (dict(y=1 << 20), "ST_E_INVAL"), (dict(y=(16 << 20) + 512), "ST_E_INVAL"), (dict(chosen=4 << 20), "ST_E_INVAL"),
    (dict(weights=3 << 20), "ST_E_INVAL"), (dict(workspace=16 << 20), "ST_E_INVAL"),
    (dict(residual=(4 << 20) + 2, ldr=256), "ST_E_INVAL"), (dict(weights=64 << 20), "ST_E_INVAL"),
]


@pytest.mark.parametrize("kw,status", REFUSED, ids=[f"{'-'.join(k)}-{i}" for i, (k, _) in enumerate(REFUSED)])
def test_refusals_queue_nothing(stmat, kw, status):
    assert stmat.STATUS[stmat.lib().st_moe(C.byref(moe_args(stmat, **kw)), None)] == status
    assert "st_moe" in stmat.lib().st_last_error().decode()


def test_null_arguments_no_tokens_and_the_workspace(stmat):
    L, need = stmat.lib(), C.c_uint64(7)
    assert stmat.STATUS[L.st_moe(None, None)] == "ST_E_INVAL"
    assert stmat.STATUS[L.st_moe_workspace(None, C.byref(need))] == "ST_E_INVAL"
    assert stmat.STATUS[L.st_moe(C.byref(moe_args(stmat, tokens=0, x=None)), None)] == "ST_OK"
    assert stmat.STATUS[L.st_moe_workspace(C.byref(moe_args(stmat, tokens=0)), C.byref(need))] == "ST_OK" and need.value == 0
    sizes = []
    for kw in (dict(), dict(tokens=6), dict(top_k=3), dict(x_dtype=9, router_dtype=9)):
        assert stmat.STATUS[L.st_moe_workspace(C.byref(moe_args(stmat, **kw)), C.byref(need))] == "ST_OK"
        sizes.append(need.value)
    assert min(sizes) == sizes[0] > 0 and sizes[0] % 256 == 0


def test_packed_arguments_have_the_structs_layout(stmat):
    assert stmat._MOE_ARGS.size == C.sizeof(stmat.MoeArgs)
    values = list(range(1, 48))
    got = stmat.MoeArgs.from_buffer_copy(stmat._MOE_ARGS.pack(*values))
    flat = []
    for f, _ in stmat.MoeArgs._fields_:
        v = getattr(got, f)
        flat += [getattr(v, g) for g, _ in v._fields_] if isinstance(v, C.Structure) else [v]
    assert flat == values


# ----------------------------------------------------------------- values

def experts(seed, e, n, k, kind, scale=0.05):
    """(weights [e, n, k] in rows at multiples of 16 bytes, block scales, what
    they stand for in 64 bits)."""
    dt = TYPES[kind]
    step = 16 // torch.empty((), dtype=dt).element_size()
    w = torch.zeros(e, n, -(-k // step) * step, dtype=dt, device="cuda")[..., :k]
    if kind.startswith("F8"):
        w.copy_(normal(seed, e, n, k, spread=40.0).to(dt))
        s = (normal(seed + 1, e, blocks_of(n), blocks_of(k)).abs() + 0.5) * (scale / 40)
        return w, s, w.double() * spread(s.double(), n, k)
    w.copy_(normal(seed, e, n, k, spread=scale).to(dt))
    return w, None, w.double()


def layer(seed, t, e, h, i, x_kind="BF16", w_kind="F8_E4M3", up=True):
    x = normal(seed, t, h, dtype=TYPES[x_kind])
    router = normal(seed + 1, e, h, dtype=TYPES[x_kind], spread=1.5 / math.sqrt(h))
    gate, gs, g64 = experts(seed + 2, e, i, h, w_kind)
    u, us, u64 = experts(seed + 4, e, i, h, w_kind) if up else (None, None, None)
    down, ds, d64 = experts(seed + 6, e, h, i, w_kind)
    return dict(x=x, router=router, gate=gate, up=u, down=down, gate_scale=gs, up_scale=us, down_scale=ds), (g64, u64, d64)


def choice64(x, router, top_k, score, normalize, factor, bias):
    l = x.double() @ router.double().t()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    key = s if bias is None else s + bias.double()
    chosen = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top_k]
    p = s.gather(1, chosen)
    return chosen, factor * (p / p.sum(1, keepdim=True) if normalize else p)


def runs_top(v):
    """The largest magnitude of each value's run of 128."""
    n = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, blocks_of(n) * 128 - n)).reshape(*v.shape[:-1], -1, 128)
    return b.abs().amax(-1, keepdim=True).expand_as(b).reshape(*v.shape[:-1], -1)[..., :n]


def experts64(x, weights, chosen, p, act, eight):
    """(y, what it may be off by) in 64 bits."""
    g64, u64, d64 = weights
    xd = x.double()
    y, off = torch.zeros_like(xd), torch.zeros_like(xd)
    hidden, inter = d64.shape[1:]
    column = 2.0 ** -21 if eight else 0.0
    for e in chosen.unique().tolist():
        tok, at = torch.nonzero(chosen == e, as_tuple=True)
        v, w = xd[tok], p[tok, at].unsqueeze(1)

        def product(m):
            return v @ m.t(), (hidden + 3) * 2.0 ** -23 * (v.abs() @ m.abs().t()) + column * (runs_top(v) @ m.abs().t())

        g, dg = product(g64[e])
        a, da = act64(g, act), 1.13 * dg
        u, du = product(u64[e]) if u64 is not None else (torch.ones_like(a), torch.zeros_like(a))
        h = a * u * w
        dh = (da * (u.abs() + du) + a.abs() * du) * w.abs() + (2.0 ** -17 + 2.0 ** -12 + 2.0 ** -20 * g.abs()) * h.abs() + column * runs_top(h)
        m = d64[e]
        y.index_add_(0, tok, h @ m.t())
        off.index_add_(0, tok, dh @ m.abs().t() + (inter + 3) * 2.0 ** -22 * (h.abs() @ m.abs().t()))
    return y, off


def check(stmat, args, weights, top_k, act="silu", score="softmax", normalize=True, factor=1.0, bias=None, residual=None,
          dst=None, out=None):
    y, chosen, p = stmat.moe(**args, top_k=top_k, act=act, score=score, normalize=normalize, factor=factor, router_bias=bias,
                             residual=residual, dst=dst, out=out)
    want, p64 = choice64(args["x"], args["router"], top_k, score, normalize, factor, bias)
    assert chosen.dtype == torch.int32 and torch.equal(chosen.long(), want)
    assert ((p.double() - p64).abs() <= P * p64.abs() + 2.0 ** -126).all()
    y64, off = experts64(args["x"], weights, want, p64, act, args["gate_scale"] is not None)
    assert torch.isfinite(y).all() and torch.isfinite(p).all()
    check_values(y, y64 if residual is None else y64 + residual.double(), extra=off, slack=2.0 ** -22)
    return y, chosen, p


SIZES = [(1, 1, 1, 16, 16), (1, 8, 2, 256, 128), (1, 64, 8, 512, 384), (2, 3, 3, 130, 70), (5, 16, 4, 384, 1100), (8, 128, 8, 256, 256),
         (9, 4, 2, 640, 129), (13, 60, 4, 1000, 500), (16, 300, 6, 128, 64), (17, 8, 1, 2048, 130), (32, 16, 5, 300, 260),
         (33, 8, 2, 512, 640), (47, 1024, 32, 64, 48), (64, 8, 8, 1024, 256), (64, 64, 6, 256, 384), (3, 2, 1, 8192, 1024)]


@gpu
@pytest.mark.parametrize("t,e,k,h,i", SIZES)
@pytest.mark.parametrize("x_kind,w_kind", [("BF16", "F8_E4M3"), ("F16", "F8_E4M3"), ("BF16", "F8_E5M2"), ("BF16", "BF16"), ("F16", "F16")])
def test_moe_values(stmat, t, e, k, h, i, x_kind, w_kind):
    args, weights = layer(t + h, t, e, h, i, x_kind, w_kind)
    y, chosen, p = check(stmat, args, weights, k, dst="F32")
    again = stmat.moe(**args, top_k=k, dst="F32")
    assert torch.equal(y, again[0]) and torch.equal(p, again[2])    # the same bits again
    y, _, _ = check(stmat, args, weights, k)
    assert y.dtype == TYPES[x_kind]


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("t,e", [(3, 20), (30, 200), (11, 500)])
def test_moe_choices(stmat, score, normalize, biased, t, e):
    args, weights = layer(t + e, t, e, 192, 96, "BF16", "BF16")
    bias = normal(99, e, spread=0.2) if biased else None
    check(stmat, args, weights, 6, score=score, normalize=normalize, factor=2.5, bias=bias)
    args["router"] = args["router"].float() * 1.01
    check(stmat, args, weights, 6, score=score, normalize=normalize, bias=bias)


@gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [1, 5, 20])
def test_chosen_scores_that_all_lie_below_binary32(stmat, score, t):
    """A bias chooses experts whose logits are 200 below the largest, and all
    of sigmoid's logits lie at -150: the chosen scores are 0 in binary32, their
    shares of their sum are not.  (Logits differ by under 30, so P holds.)"""
    args, weights = layer(t, t, 12, 256, 96, "BF16", "BF16")
    args["x"][:, 0] = 1.0
    bias = None
    if score == "softmax":
        args["router"][:, 0] = 200.0
        args["router"][:5, 0] = 0.0
        bias = torch.zeros(12, device="cuda")
        bias[:5] = torch.tensor([5.0, 7.0, 6.0, 3.0, 4.0], device="cuda")
    else:
        args["router"][:, 0] = -150.0
    check(stmat, args, weights, 4, score=score, bias=bias)


@gpu
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("up", [False, True])
@pytest.mark.parametrize("w_kind", ["F8_E4M3", "BF16"])
def test_moe_activations_and_residual(stmat, act, up, w_kind):
    args, weights = layer(3, 6, 12, 320, 200, "BF16", w_kind, up=up)
    r = normal(4, 6, 320, dtype=torch.bfloat16)
    check(stmat, args, weights, 3, act=act, residual=r)
    check(stmat, args, weights, 3, act=act, residual=r.half(), dst="F16")
    want = stmat.moe(**args, top_k=3, act=act, residual=r)[0]
    stmat.moe(**args, top_k=3, act=act, residual=r, out=r)
    assert torch.equal(r, want)


@gpu
@pytest.mark.parametrize("t", [1, 7, 8, 16, 31, 64])
@pytest.mark.parametrize("w_kind", ["F8_E4M3", "BF16"])
def test_every_token_chooses_the_same_experts(stmat, t, w_kind):
    """One expert with all tokens, and equal logits, of which the lowest
    indices are taken."""
    args, weights = layer(t, t, 10, 256, 300, "BF16", w_kind)
    bias = torch.zeros(10, device="cuda")
    bias[7], bias[2] = 50.0, 40.0
    chosen = check(stmat, args, weights, 2, bias=bias)[1]
    assert (chosen == torch.tensor([7, 2], device="cuda")).all()
    args["router"] = torch.zeros_like(args["router"])
    chosen = check(stmat, args, weights, 3, normalize=False)[1]
    assert (chosen == torch.arange(3, device="cuda")).all()
    args["router"][4:] = 1.0
    args["x"] = args["x"].abs()
    chosen = check(stmat, args, weights, 4)[1]
    assert (chosen == torch.arange(4, 8, device="cuda")).all()


@gpu
@pytest.mark.parametrize("seed", range(4))
def test_choices_that_turn_on_the_last_digits(stmat, seed):
    """Router rows that differ from one another by one unit of the last place
    of one entry: their logits' order takes more than binary32's digits of the
    sum, which large terms that cancel dominate."""
    t, e, h = 16, 32, 512
    args, weights = layer(seed, t, e, h, 64, "BF16", "BF16")
    x = args["x"]
    x[:, :128], x[:, 128:256] = 200.0, -200.0
    row = torch.ones(h, device="cuda")
    row[256:] = normal(seed + 50, 256, spread=0.01)
    router = row.bfloat16().expand(e, h).clone()
    g = torch.Generator().manual_seed(seed)
    bump = torch.randperm(e, generator=g).cuda()
    router[torch.arange(e, device="cuda"), 256 + bump] *= 1 + 2.0 ** -7
    args["router"] = router
    # (Exact in 64 bits: entries are multiples of 2^-20 or so; equal logits are
    # ties.  Neighbours are nearer than binary32's step at 25600, 2^-9.)
    l = x.double() @ router.double().t()
    assert l.sort(1).values.diff(dim=1).median() < 2.0 ** -10
    check(stmat, args, weights, 5, score="sigmoid")


@gpu
def test_large_and_small_values(stmat):
    """x over 2^40 and its runs' own scales, and tokens of zeros."""
    for w_kind in ("F8_E4M3", "BF16"):
        args, weights = layer(11, 5, 8, 512, 256, "BF16", w_kind)
        args["x"][0, :128] *= 2.0 ** 20
        args["x"][1] *= 2.0 ** -30
        args["x"][2] = 0
        args["x"][3, 128:256] = 0
        args["router"] *= 2.0 ** -18
        check(stmat, args, weights, 3, act="relu", dst="F32")


@gpu
def test_nan_and_infinity_stay_with_their_tokens(stmat):
    for w_kind in ("F8_E4M3", "BF16"):
        args, _ = layer(12, 6, 8, 384, 256, "BF16", w_kind)
        clean = stmat.moe(**args, top_k=2)
        args["x"][1, 200] = math.nan
        args["x"][4, 3] = math.inf
        y, chosen, p = stmat.moe(**args, top_k=2)
        keep = torch.tensor([0, 2, 3, 5], device="cuda")
        assert torch.equal(y[keep], clean[0][keep]) and torch.equal(chosen[keep], clean[1][keep]) and torch.equal(p[keep], clean[2][keep])
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[4]).any()
        assert ((chosen >= 0) & (chosen < 8)).all() and (chosen[1] == torch.tensor([0, 1], device="cuda")).all()
        args, _ = layer(12, 6, 8, 384, 256, "BF16", w_kind)
        args["router"][5, 7] = math.nan    # its expert is everyone's first
        y, chosen, p = stmat.moe(**args, top_k=2)
        assert (chosen[:, 0] == 5).all() and torch.isnan(y).all()


@gpu
def test_strides_scales_and_shapes(stmat):
    """Gate and up as halves of one tensor, one scale for all, matrices with
    rows apart; nothing is written outside y."""
    t, e, k, h, i = 7, 6, 2, 272, 144
    both, s, b64 = experts(1, e, 2 * i, h, "F8_E4M3")
    down, _, _ = experts(2, e, h, i, "F8_E4M3")
    one = torch.full((1, 1, 1), 2.0 ** -9, device="cuda")
    gs, ds = one.expand(e, blocks_of(i), blocks_of(h)), one.expand(e, blocks_of(h), blocks_of(i))
    x, router = normal(3, t, h, dtype=torch.bfloat16), normal(4, e, h, dtype=torch.bfloat16, spread=0.1)
    r = normal(5, t, h, dtype=torch.bfloat16)
    args = dict(x=padded(x, 3, 1), router=padded(router, 5, 3), gate=both[:, :i], up=both[:, i:], down=down, gate_scale=gs,
                up_scale=gs, down_scale=ds)
    weights = tuple(w.double() * 2.0 ** -9 for w in (both[:, :i], both[:, i:], down))
    yv = padded(torch.zeros_like(r), 9, 5)
    check(stmat, args, weights, k, residual=padded(r, 1, 2), out=yv)
    flat = yv._base.reshape(-1).float()
    inside = torch.zeros(flat.numel(), dtype=torch.bool, device="cuda")
    inside[5:5 + t * (h + 9)].view(t, h + 9)[:, :h] = True
    assert (flat[~inside] == torch.tensor(77.0).bfloat16().float().item()).all()
    args["x"] = x[:6].view(2, 3, h)
    y, chosen, p = stmat.moe(**args, top_k=k)
    assert y.shape == (2, 3, h) and chosen.shape == p.shape == (2, 3, k)
    args["x"] = x[:6]
    assert torch.equal(y.view(6, h), stmat.moe(**args, top_k=k)[0])
    args["x"] = x[0]
    assert stmat.moe(**args, top_k=k)[0].shape == (h,)
    args["x"] = x[:0]
    assert stmat.moe(**args, top_k=k)[0].shape == (0, h)


@gpu
def test_binding_refusals(stmat):
    args, _ = layer(1, 4, 8, 256, 128)

    def but(**kw):
        return lambda: stmat.moe(**{**args, "top_k": 2, **kw})

    for call, status in ((but(top_k=9), "ST_E_INVAL"), (but(x=args["x"].float()), "ST_E_DTYPE"), (but(act="swish"), "ST_E_INVAL"),
                         (but(score="max"), "ST_E_INVAL"), (but(router=args["router"][:, :8]), "ST_E_INVAL"),
                         (but(gate=args["gate"][:7]), "ST_E_INVAL"), (but(down=args["gate"]), "ST_E_INVAL"),
                         (but(up=args["up"].view(torch.float8_e5m2)), "ST_E_INVAL"), (but(gate_scale=None), "ST_E_INVAL"),
                         (but(down_scale=args["down_scale"].half()), "ST_E_DTYPE"), (but(gate_scale=args["gate_scale"][:, :, :1]), "ST_E_INVAL"),
                         (but(router_bias=torch.zeros(7, device="cuda")), "ST_E_INVAL"), (but(residual=args["x"].half()), "ST_E_INVAL"),
                         (but(x=args["x"].repeat(17, 1)), "ST_E_INVAL"), (but(x=args["x"].cpu()), "ST_E_INVAL"),
                         (but(out=args["x"]), "ST_E_INVAL"), (but(gate=args["gate"][:, :, :200], router=args["router"][:, :200],
                                                                  x=args["x"][:, :200]), "ST_E_INVAL")):
        with pytest.raises(stmat.StmatError) as e:
            call()
        assert e.value.status == status, e.value


@gpu
def test_graphs_streams_and_calls_side_by_side(stmat):
    """Replayed with new inputs, two graphs and an eager stream at once."""
    sets = [layer(21, 6, 16, 512, 256)[0], layer(22, 40, 16, 512, 256, "BF16", "BF16")[0]]
    others = [layer(31, 6, 16, 512, 256)[0]["x"], layer(32, 40, 16, 512, 256)[0]["x"]]
    first = [[v.clone() for v in stmat.moe(**s, top_k=4)] for s in sets]
    second = [[v.clone() for v in stmat.moe(**{**s, "x": o}, top_k=4)] for s, o in zip(sets, others)]
    xs = [s["x"].clone() for s in sets]
    graphs, outs = [], []
    for s, x in zip(sets, xs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(stmat.moe(**{**s, "x": x}, top_k=4))
        graphs.append(g)
    side = [torch.cuda.Stream() for _ in range(3)]
    for new in (True, False, True):
        for x, s, o in zip(xs, sets, others):
            x.copy_(o if new else s["x"])
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st in zip(graphs, side):
                with torch.cuda.stream(st):
                    g.replay()
            eager = [stmat.moe(**s, top_k=4, stream=side[2]) for s in sets]
        torch.cuda.synchronize()
        for got, want in zip(outs + eager, (second if new else first) + first):
            for a, b in zip(got, want):
                assert torch.equal(a, b)


@gpu
def test_no_wait_gave_up(stmat):
    torch.cuda.synchronize()
    assert stmat.static_check() == 0

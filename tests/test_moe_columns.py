"""What st_moe keeps of h, the values between its products, bit for bit.

One expert a token with the weight 1, act="none" and no up: h is gate x.  Gate's
rows pick two or three entries of x, each below the last one's digits, so that h
has 16 to 24 significant bits and is summed without rounding; down's rows pick an
entry of h each.  y is then h as down takes it: a power of two times two columns
of the experts' 16-bit type, or three of E4M3 codes, c0 + 2^-4 c1 + 2^-9 c2, each
the rounding error of those before it.  A rounding is off by half a unit of the
last place, relative 2^-8 (BF16), 2^-11 (F16) or 2^-4 (E4M3), so the columns
leave 2^-16, 2^-22 or 2^-12 of a value, and the smallest of a code's numbers
2^-39 (F16) or 2^-26 (E4M3) of the run's largest."""
import pytest

torch = pytest.importorskip("torch")

from test_block_operators import blocks_of, spread  # noqa: E402
from test_moe import runs_top  # noqa: E402
from test_operators import TYPES, normal  # noqa: E402

gpu = pytest.mark.gpu
# By the experts' type: significant bits that the columns' exponent leaves room
# for, and what the columns may lose of a value and of the run's largest.
FORMS = {"BF16": (2, 2.0 ** -16, 0.0), "F16": (15, 2.0 ** -22, 2.0 ** -39), "F8": (8, 2.0 ** -12, 2.0 ** -26)}


def rows16(e, n, k, kind):
    """Zeroed [e, n, k] weights in rows at multiples of 16 bytes."""
    dt = TYPES[kind]
    step = 16 // torch.empty((), dtype=dt).element_size()
    return torch.zeros(e, n, -(-k // step) * step, dtype=dt, device="cuda")[..., :k]


def powers(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return (2.0 ** torch.randint(-1, 2, shape, generator=g).float()).cuda()


def columns(h, kind, count):
    """The sum of h's first `count` columns, in binary32."""
    below = FORMS[kind[:2] if kind.startswith("F8") else kind][0]
    top = runs_top(h)
    s = torch.exp2(torch.floor(torch.log2(top)) - (below - 1))
    v = (h / s).float()
    if not kind.startswith("F8"):
        hi = v.to(TYPES[kind]).float()
        return (hi + (v - hi).to(TYPES[kind]).float() if count > 1 else hi).double() * s
    kept = torch.zeros_like(v)
    for up in (1.0, 16.0, 512.0)[:count]:
        c = (v * up).to(torch.float8_e4m3fn).float()
        v = v - c / up
        kept = kept + c / up
    return kept.double() * s


@gpu
@pytest.mark.parametrize("t,e,hidden,inter", [(1, 1, 48, 16), (5, 3, 300, 260), (9, 4, 640, 129), (17, 5, 1100, 384), (33, 2, 256, 300),
                                              (64, 1, 130, 500), (64, 40, 272, 144), (2, 2, 8192, 1024)])
@pytest.mark.parametrize("x_kind,w_kind", [("BF16", "BF16"), ("F16", "F16"), ("BF16", "F8_E4M3"), ("F16", "F8_E4M3"), ("BF16", "F8_E5M2")])
def test_every_column_of_h_reaches_y(stmat, t, e, hidden, inter, x_kind, w_kind):
    eight, half = w_kind.startswith("F8"), x_kind == "F16"
    g = torch.Generator().manual_seed(t + hidden)
    # Entries from 1 to 1.9 with all of their type's digits.
    one = 1024 if half else 128
    x = (torch.randint(one, int(1.9 * one), (t, hidden), generator=g).float() / one).to(TYPES[x_kind]).cuda()
    router = normal(1, e, hidden, dtype=TYPES[x_kind])
    gate, down = rows16(e, inter, hidden, w_kind), rows16(e, hidden, inter, w_kind)
    # (The third one's last digit is 2^-23: sums under 2 have 24 bits.)
    parts = (1.0, 2.0 ** -8) if eight else (1.0, 2.0 ** -11, 2.0 ** -13) if half else (1.0, 2.0 ** -8, 2.0 ** -16)
    third, n = hidden // 3, torch.arange(inter, device="cuda")
    for i, part in enumerate(parts):
        for j in range(e):
            gate[j].index_put_((n, i * third + (n * (2 * i + 1) + j) % third), torch.tensor(part, device="cuda").to(gate.dtype))
    m = torch.arange(hidden, device="cuda")
    pick = torch.stack([(5 * m + 1 + j) % inter for j in range(e)])
    for j in range(e):
        down[j].index_put_((m, pick[j]), torch.tensor(1.0, device="cuda").to(down.dtype))
    scales = dict(gate_scale=powers(2, e, blocks_of(inter), blocks_of(hidden)), down_scale=powers(3, e, blocks_of(hidden), blocks_of(inter))) if eight else {}
    y, chosen, p = stmat.moe(x, router, gate, None, down, 1, act="none", dst="F32", **scales)
    assert (p == 1).all()
    chosen = chosen.flatten().long()
    g64, d64 = gate.double(), down.double()
    if eight:
        g64, d64 = g64 * spread(scales["gate_scale"].double(), inter, hidden), d64 * spread(scales["down_scale"].double(), hidden, inter)
    h = torch.einsum("th,tih->ti", x.double(), g64[chosen])
    assert torch.equal(h.float().double(), h)    # no digit of h is beyond binary32

    def taken(v):
        return torch.einsum("ti,thi->th", v, d64[chosen])

    most = 3 if eight else 2
    assert torch.equal(y.double(), taken(columns(h, w_kind, most)))
    _, own, top = FORMS["F8" if eight else w_kind]
    bound = taken((own + 2.0 ** -24) * h.abs() + top * runs_top(h))
    want = taken(h)
    assert ((y.double() - want).abs() <= bound).all()
    # One column fewer would show.
    assert ((taken(columns(h, w_kind, most - 1)) - want).abs() > bound).any()

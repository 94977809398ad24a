"""Cases of the operators that follow a materialized checkpoint in a
transformer's MLP: the root-mean-square norm with the residual's addition and
an 8-bit output (stmat.rms_norm), the matrix product with scales, bias,
activation and residual in its epilogue (stmat.linear), and the gated
activation with an 8-bit output (stmat.gated_act).

Formulas (sums in 32 bits or more, one rounding at the end):
  rms_norm   h = x + r;  y = h * w / sqrt(mean(h^2) + eps)
  linear     y = act(xs[m] * ws * sum_k x[m, k] w[n, k] + b[n]) + r[m, n]
  gated_act  y = act(g) * u
  8 bits     scale[m] = max(max_c |y[m, c]| / 448, 2^-126), or one given scale;
             code = e4m3(clamp(y / scale, -448, 448))
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TYPES = {"BF16": torch.bfloat16, "F16": torch.float16, "F32": torch.float32, "F8_E4M3": torch.float8_e4m3fn}
SIZE = {"BF16": 2, "F16": 2, "F32": 4, "F8_E4M3": 1}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
EPS = 1e-5
# The largest listed product (8192 tokens through a 4096 -> 14336 weight), and
# the largest listed row operator, in elements.
MOST_MNK = 8192 * 14336 * 4096
MOST_ROWS = 8192 * 14336


def listed():
    return [
        # One new token's hidden state, residual added, 8 bits for the
        # scaled-FP8 projections: latency.
        {"name": "norm_1x4096_fp8", "op": "rms_norm", "m": 1, "c": 4096, "type": "BF16", "dst": "F8_E4M3",
         "residual": True, "static": False},
        # A prefill of 8192 tokens of the 8B LLM (hidden 4096).
        {"name": "norm_8192x4096_fp8", "op": "rms_norm", "m": 8192, "c": 4096, "type": "BF16", "dst": "F8_E4M3",
         "residual": True, "static": False},
        # A large hidden size of the scaled-FP8 transformer (12288), 16 bits out,
        # the checkpoint path without 8-bit weights.
        {"name": "norm_4096x12288_bf16", "op": "rms_norm", "m": 4096, "c": 12288, "type": "BF16", "dst": "BF16",
         "residual": True, "static": False},
        # Ragged: rows that start at odd byte offsets, one scale for the tensor.
        {"name": "norm_777x1111_static", "op": "rms_norm", "m": 777, "c": 1111, "type": "F16", "dst": "F8_E4M3",
         "residual": False, "static": True},
        # One token through the gate of an 8B LLM's MLP (14336), 8 bits out.
        {"name": "act_1x14336_fp8", "op": "gated_act", "m": 1, "c": 14336, "type": "BF16", "dst": "F8_E4M3",
         "act": "silu", "gated": True, "static": False},
        # The same for a prefill of 8192 tokens.
        {"name": "act_8192x14336_fp8", "op": "gated_act", "m": 8192, "c": 14336, "type": "BF16", "dst": "F8_E4M3",
         "act": "silu", "gated": True, "static": False},
        # One token through a scaled-FP8 up projection: the weight's bytes count.
        {"name": "lin_1_4096_14336_fp8", "op": "linear", "m": 1, "n": 14336, "k": 4096, "type": "F8_E4M3",
         "dst": "BF16", "act": "none", "bias": False, "residual": False},
        # A batch of 8 tokens through a BF16 down projection, residual added.
        {"name": "lin_8_14336_4096_bf16", "op": "linear", "m": 8, "n": 4096, "k": 14336, "type": "BF16",
         "dst": "BF16", "act": "none", "bias": False, "residual": True},
        # A batch of 256 tokens (continuous batching), 8 bits, attention output.
        {"name": "lin_256_4096_4096_fp8", "op": "linear", "m": 256, "n": 4096, "k": 4096, "type": "F8_E4M3",
         "dst": "BF16", "act": "none", "bias": True, "residual": True},
        # Ragged sizes in every dimension, rows at odd byte offsets (an
        # embedding head of a small text encoder).
        {"name": "lin_333_1111_777_f16", "op": "linear", "m": 333, "n": 1111, "k": 777, "type": "F16",
         "dst": "F16", "act": "gelu", "bias": True, "residual": False},
        # A prefill of 8192 tokens, scaled-FP8 up projection: the largest.
        {"name": "lin_8192_4096_14336_fp8", "op": "linear", "m": 8192, "n": 14336, "k": 4096, "type": "F8_E4M3",
         "dst": "BF16", "act": "silu", "bias": False, "residual": False},
        # A prefill of 4096 tokens, BF16 down projection with the residual.
        {"name": "lin_4096_14336_4096_bf16", "op": "linear", "m": 4096, "n": 4096, "k": 14336, "type": "BF16",
         "dst": "BF16", "act": "none", "bias": True, "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_norm", "gated_act", "linear", "linear"])
    if op == "linear":
        while True:
            m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
            # Half of the weights have the usual sizes, multiples of 64.
            if rng.random() < 0.5:
                n, k = -(-n // 64) * 64, -(-k // 64) * 64
            if m * n * k <= MOST_MNK:
                break
        kind = rng.choice(["BF16", "F16", "F8_E4M3", "F8_E4M3"])
        return {"op": op, "m": m, "n": n, "k": k, "type": kind, "dst": "BF16" if kind == "F8_E4M3" else kind,
                "act": rng.choice(ACTS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    while True:
        m, c = _log_int(rng, 1, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            c = -(-c // 64) * 64
        if m * c <= MOST_ROWS:
            break
    kind = rng.choice(["BF16", "BF16", "F16", "F32"])
    if kind == "F32" and 2 * m * c > MOST_ROWS:
        kind = "BF16"
    case = {"op": op, "m": m, "c": c, "type": kind, "dst": rng.choice([kind, "F8_E4M3", "F8_E4M3"]),
            "static": rng.random() < 0.3}
    if op == "rms_norm":
        case["residual"] = rng.random() < 0.5
    else:
        case["act"], case["gated"] = rng.choice(ACTS), rng.random() < 0.75
    return case


# --------------------------------------------------------------- inputs

def _inputs(case, seed):
    """What the caller holds: tensors on the GPU, made from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": dict(case)}
    dt = TYPES[case["type"]]
    m = case["m"]
    if case["op"] == "rms_norm":
        c = case["c"]
        # A residual stream: some channels carry far larger values than others.
        spread = torch.exp(0.7 * normal(c))
        s["x"] = (normal(m, c) * spread).to(dt)
        s["r"] = (0.5 * normal(m, c)).to(dt) if case["residual"] else None
        s["w"] = (1.0 + 0.2 * normal(c)).to(dt)
        s["scale"] = torch.full((1,), 0.02, device=dev) if case["static"] and case["dst"] == "F8_E4M3" else None
    elif case["op"] == "gated_act":
        c = case["c"]
        # Gate and up are the halves of one product's output, or one tensor.
        both = (1.5 * normal(m, 2 * c if case["gated"] else c)).to(dt)
        s["gate"] = both[:, :c]
        s["up"] = both[:, c:] if case["gated"] else None
        s["scale"] = torch.full((1,), 0.02, device=dev) if case["static"] and case["dst"] == "F8_E4M3" else None
    else:
        n, k = case["n"], case["k"]
        x, w = normal(m, k), 0.02 * normal(n, k)
        if case["type"] == "F8_E4M3":
            # Activations as a norm hands them over (a scale per token),
            # weights as a scaled-FP8 checkpoint holds them (one scale).
            s["xs"] = x.abs().amax(1) / E4M3_MAX
            s["ws"] = (w.abs().amax() / E4M3_MAX).reshape(1)
            x, w = x / s["xs"][:, None], w / s["ws"]
        else:
            s["xs"] = s["ws"] = None
        s["x"], s["w"] = x.to(dt), w.to(dt)
        out = TYPES[case["dst"]]
        s["b"] = (0.5 * normal(n)).to(out) if case["bias"] else None
        s["r"] = normal(m, n).to(out) if case["residual"] else None
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ----------------------------------------------------------- plain forms

def _act(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _eight_bits(y, scale):
    """(codes, scales): one scale per row, or the given one (scales None)."""
    if scale is not None:
        return (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), None
    scales = (y.abs().amax(1) / E4M3_MAX).clamp_min(2.0 ** -126)
    return (y / scales[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scales


def _plain(s):
    c = s["case"]
    dst = TYPES[c["dst"]]
    if c["op"] == "linear":
        y = torch.matmul(s["x"].float(), s["w"].float().t())
        if s["xs"] is not None:
            y = y * (s["xs"][:, None] * s["ws"])
        if s["b"] is not None:
            y = y + s["b"].float()
        y = _act(y, c["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return [y.to(dst)]
    if c["op"] == "rms_norm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
        kept = h.to(s["x"].dtype) if s["r"] is not None else None
    else:
        y = _act(s["gate"].float(), c["act"])
        if s["up"] is not None:
            y = y * s["up"].float()
        kept = None
    codes, scales = _eight_bits(y, s["scale"]) if c["dst"] == "F8_E4M3" else (y.to(dst), None)
    return [codes, scales, kept]


def run(state):
    if not own:
        return _plain(state)
    from safetensors_materialization_gb300 import stmat
    c = state["case"]
    if c["op"] == "linear":
        return [stmat.linear(state["x"], state["w"], x_scale=state["xs"], w_scale=state["ws"], bias=state["b"],
                             act=c["act"], residual=state["r"], dst=c["dst"])]
    if c["op"] == "rms_norm":
        y, scales, h = stmat.rms_norm(state["x"], state["w"], eps=EPS, residual=state["r"], dst=c["dst"],
                                      scale=state["scale"])
        return [y, scales, h]
    y, scales = stmat.gated_act(state["gate"], state["up"], act=c["act"], dst=c["dst"], scale=state["scale"])
    return [y, scales, None]


def work(case):
    m, size, out = case["m"], SIZE[case["type"]], SIZE[case["dst"]]
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        moved = size * (m * k + n * k) + out * m * n * (2 if case["residual"] else 1)
        moved += out * n if case["bias"] else 0
        moved += 4 * (m + 1) if case["type"] == "F8_E4M3" else 0
        return {"bytes": moved, "flops": 2 * m * n * k}
    c = case["c"]
    scales = 4 * m if case["dst"] == "F8_E4M3" and not case["static"] else 0
    if case["op"] == "rms_norm":
        return {"bytes": m * c * ((3 if case["residual"] else 1) * size + out) + c * size + scales, "flops": 6 * m * c}
    return {"bytes": m * c * ((2 if case["gated"] else 1) * size + out) + scales, "flops": 8 * m * c}


# ------------------------------------------- the definitions in 64 bits

def _exact_act(v, name):
    if name == "relu":
        return v.clamp_min(0.0)
    if name == "silu":
        return v * torch.special.expit(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    if name == "gelu_tanh":
        return v * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    """The formulas at the top in 64 bits, without the roundings at the end:
    an 8-bit output is compared with the quotient that its codes round."""
    s = _inputs(case, seed)
    rows = []
    if case["op"] == "linear":
        wt = s["w"].double().t()
        step = max(1, min(case["m"], (1 << 27) // max(case["n"], case["k"])))
        for a in range(0, case["m"], step):
            y = s["x"][a:a + step].double() @ wt
            if s["xs"] is not None:
                y *= s["xs"][a:a + step].double().unsqueeze(1)
                y *= s["ws"].double()
            if s["b"] is not None:
                y += s["b"].double()
            y = _exact_act(y, case["act"])
            if s["r"] is not None:
                y += s["r"][a:a + step].double()
            rows.append(y)
        return [torch.cat(rows)]
    kept = None
    if case["op"] == "rms_norm":
        h = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
        y = h / (h.square().sum(1, keepdim=True) / case["c"] + EPS).sqrt() * s["w"].double()
        kept = h if s["r"] is not None else None
    else:
        y = _exact_act(s["gate"].double(), case["act"])
        y = y if s["up"] is None else y * s["up"].double()
    if case["dst"] != "F8_E4M3":
        return [y, None, kept]
    if s["scale"] is not None:
        return [torch.clamp(y / s["scale"].double(), min=-E4M3_MAX, max=E4M3_MAX), None, kept]
    scales = torch.clamp(torch.max(torch.abs(y), dim=1).values / E4M3_MAX, min=2.0 ** -126)
    return [y / scales.unsqueeze(1), scales, kept]

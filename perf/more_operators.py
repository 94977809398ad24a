"""Cases of the operators that run a block-scaled FP8 checkpoint's layers on
its weights as stored: rows in 8 bits with a scale for every 128 columns
(stmat.rms_norm and stmat.gated_act with block=128), the product of such rows
with a weight that has a scale for every 128 x 128 block (stmat.block_linear),
and a whole mixture-of-experts layer for a few tokens, from its router to the
sum of its experts (stmat.moe), with block-scaled FP8 or 16-bit experts.

Formulas (one rounding at the end):
  rows          h = x + r;  v = h * w / sqrt(mean(h^2) + eps)   or   v = act(g) * u
                scale[m, b] = max(max over block b of |v[m, c]| / 448, 2^-126)
                code[m, c] = e4m3(v[m, c] / scale[m, c / 128])
  block_linear  y = act(sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] w[n, k] + bias[n]) + r[m, n]
  moe           l = x router^T;  s = softmax(l) or sigmoid(l)
                chosen: the top_k experts with the largest s + router_bias (ties: the lowest index)
                p = factor * s / (sum of the chosen s, or 1)
                y = sum over the chosen e of p_e down_e (act(gate_e x) * (up_e x)) + r
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TYPES = {"BF16": torch.bfloat16, "F16": torch.float16, "F32": torch.float32, "F8_E4M3": torch.float8_e4m3fn}
SIZE = {"BF16": 2, "F16": 2, "F32": 4, "F8_E4M3": 1}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
EPS = 1e-5
# The largest listed product, the largest listed row operator in elements, and
# for the layer: weights of all its experts, and weights times tokens' choices.
MOST_MNK = 8192 * 14336 * 4096
MOST_ROWS = 8192 * 14336
MOST_EXPERTS = 8 * 3 * 4096 * 14336
MOST_CHOICES = 64 * 6 * 3 * 4096 * 1408


def listed():
    return [
        # One new token's hidden state, residual added: latency.
        {"name": "norm_1x4096_blocks", "op": "norm", "m": 1, "c": 4096, "type": "BF16", "residual": True},
        # A prefill of 8192 tokens of the 8B LLM (hidden 4096).
        {"name": "norm_8192x4096_blocks", "op": "norm", "m": 8192, "c": 4096, "type": "BF16", "residual": True},
        # The same tokens through the gate of that model's MLP (14336).
        {"name": "act_8192x14336_blocks", "op": "act", "m": 8192, "c": 14336, "type": "BF16", "act": "silu", "gated": True},
        # Ragged: rows at odd byte offsets, a last block of 87 columns.
        {"name": "act_777x1111_blocks", "op": "act", "m": 777, "c": 1111, "type": "F16", "act": "gelu_tanh", "gated": True},
        # One token through an up projection: the weight's bytes count.
        {"name": "lin_1_4096_14336", "op": "linear", "m": 1, "n": 14336, "k": 4096, "dst": "BF16", "act": "none",
         "bias": False, "residual": False},
        # 64 sequences decoded together, down projection onto the residual.
        {"name": "lin_64_14336_4096", "op": "linear", "m": 64, "n": 4096, "k": 14336, "dst": "BF16", "act": "none",
         "bias": False, "residual": True},
        # Ragged sizes in every dimension, rows at odd byte offsets.
        {"name": "lin_333_1111_777", "op": "linear", "m": 333, "n": 1111, "k": 777, "dst": "F16", "act": "gelu",
         "bias": True, "residual": False},
        # A prefill of 8192 tokens, up projection: the largest.
        {"name": "lin_8192_4096_14336", "op": "linear", "m": 8192, "n": 14336, "k": 4096, "dst": "BF16", "act": "silu",
         "bias": False, "residual": False},
        # One token of a decode through a layer of many small experts.
        {"name": "moe_1_e128_k8", "op": "moe", "m": 1, "e": 128, "top": 8, "h": 2048, "i": 768, "type": "BF16",
         "weights": "F8_E4M3", "act": "silu", "score": "softmax", "normalize": True, "factor": 1.0, "bias": False,
         "residual": False},
        # Seven sequences through a layer of few large 16-bit experts.
        {"name": "moe_7_e8_k2", "op": "moe", "m": 7, "e": 8, "top": 2, "h": 4096, "i": 14336, "type": "BF16",
         "weights": "BF16", "act": "silu", "score": "softmax", "normalize": True, "factor": 1.0, "bias": False,
         "residual": True},
        # Ragged sizes: blocks that end inside a tile, 13 tokens.
        {"name": "moe_13_e60_k4", "op": "moe", "m": 13, "e": 60, "top": 4, "h": 2000, "i": 1000, "type": "F16",
         "weights": "F16", "act": "gelu_tanh", "score": "softmax", "normalize": False, "factor": 1.0, "bias": False,
         "residual": False},
        # The largest batch: 64 tokens, sigmoid scores with a balancing bias.
        {"name": "moe_64_e64_k6", "op": "moe", "m": 64, "e": 64, "top": 6, "h": 4096, "i": 1408, "type": "BF16",
         "weights": "F8_E4M3", "act": "silu", "score": "sigmoid", "normalize": True, "factor": 2.5, "bias": True,
         "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "act", "linear", "linear", "moe", "moe"])
    even = rng.random() < 0.5
    if op == "linear":
        while True:
            m, n, k = _log_int(rng, 1, 8192), _log_int(rng, 64, 16384), _log_int(rng, 64, 16384)
            if even:  # the usual sizes, multiples of 64
                n, k = -(-n // 64) * 64, -(-k // 64) * 64
            if m * n * k <= MOST_MNK:
                break
        return {"op": op, "m": m, "n": n, "k": k, "dst": rng.choice(["BF16", "BF16", "F16", "F32"]),
                "act": rng.choice(ACTS), "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    if op == "moe":
        while True:
            m, e, h, i = _log_int(rng, 1, 64), _log_int(rng, 4, 128), _log_int(rng, 256, 8192), _log_int(rng, 128, 14336)
            top = rng.randint(1, min(8, e))
            if even:
                h, i = -(-h // 128) * 128, -(-i // 128) * 128
            if e * 3 * h * i <= MOST_EXPERTS and m * top * 3 * h * i <= MOST_CHOICES:
                break
        kind = rng.choice(["BF16", "BF16", "F16"])
        return {"op": op, "m": m, "e": e, "top": top, "h": h, "i": i, "type": kind,
                "weights": rng.choice([kind, "F8_E4M3", "F8_E4M3"]), "act": rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]),
                "score": rng.choice(["softmax", "sigmoid"]), "normalize": rng.random() < 0.5,
                "factor": rng.choice([1.0, 2.5]), "bias": rng.random() < 0.3, "residual": rng.random() < 0.5}
    while True:
        m, c = _log_int(rng, 1, 16384), _log_int(rng, 64, 16384)
        if even:
            c = -(-c // 64) * 64
        if m * c <= MOST_ROWS:
            break
    kind = rng.choice(["BF16", "BF16", "F16", "F32"])
    if kind == "F32" and 2 * m * c > MOST_ROWS:
        kind = "BF16"
    if op == "norm":
        return {"op": op, "m": m, "c": c, "type": kind, "residual": rng.random() < 0.5}
    return {"op": op, "m": m, "c": c, "type": kind, "act": rng.choice(ACTS), "gated": rng.random() < 0.75}


# --------------------------------------------------------------- inputs

def _blocks(n):
    return -(-n // BLOCK)


def _padded(v, *sizes):
    """v with its last dimensions padded with zeros to `sizes`."""
    pad = []
    for have, want in zip(reversed(v.shape), reversed(sizes)):
        pad += [0, want - have]
    return torch.nn.functional.pad(v, pad) if any(pad) else v


def _weight(normal, lead, n, k, kind):
    """A weight as a checkpoint holds it: 16 bits, or E4M3 with a scale for
    every 128 x 128 block.  Rows of experts (lead) are laid out at multiples of
    16 bytes."""
    w = 0.02 * normal(*lead, n, k)
    scale = None
    if kind == "F8_E4M3":
        nb, kb = _blocks(n), _blocks(k)
        b = _padded(w, nb * BLOCK, kb * BLOCK).reshape(*lead, nb, BLOCK, kb, BLOCK)
        scale = (b.abs().amax((-3, -1)) / E4M3_MAX).clamp_min(2.0 ** -126)
        b /= scale[..., :, None, :, None]
        w = b.reshape(*lead, nb * BLOCK, kb * BLOCK)[..., :n, :k]
    step = 16 // SIZE[kind] if lead else 1
    return _padded(w, -(-k // step) * step).to(TYPES[kind]).contiguous()[..., :k], scale


def _inputs(case, seed):
    """What the caller holds: tensors on the GPU, made from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": dict(case)}
    m = case["m"]
    if case["op"] == "norm":
        c, dt = case["c"], TYPES[case["type"]]
        # A residual stream: some channels carry far larger values than others.
        spread = torch.exp(0.7 * normal(c))
        s["x"] = (normal(m, c) * spread).to(dt)
        s["r"] = (0.5 * normal(m, c)).to(dt) if case["residual"] else None
        s["w"] = (1.0 + 0.2 * normal(c)).to(dt)
    elif case["op"] == "act":
        c, dt = case["c"], TYPES[case["type"]]
        # Gate and up are the halves of one product's output, or one tensor.
        both = (1.5 * normal(m, 2 * c if case["gated"] else c)).to(dt)
        s["gate"] = both[:, :c]
        s["up"] = both[:, c:] if case["gated"] else None
    elif case["op"] == "linear":
        n, k = case["n"], case["k"]
        # Activations as the row operators hand them over, weights as stored.
        x = normal(m, k) * torch.exp(0.7 * normal(k))
        b = _padded(x, _blocks(k) * BLOCK).reshape(m, -1, BLOCK)
        s["xs"] = (b.abs().amax(2) / E4M3_MAX).clamp_min(2.0 ** -126)
        s["x"] = (b / s["xs"][:, :, None]).reshape(m, -1)[:, :k].to(torch.float8_e4m3fn).contiguous()
        s["w"], s["ws"] = _weight(normal, (), n, k, "F8_E4M3")
        out = TYPES[case["dst"]]
        s["b"] = (0.5 * normal(n)).to(out) if case["bias"] else None
        s["r"] = normal(m, n).to(out) if case["residual"] else None
    else:
        e, h, i, dt = case["e"], case["h"], case["i"], TYPES[case["type"]]
        # Normed hidden states, logits with a deviation of about 1.5.
        s["x"] = normal(m, h).to(dt)
        s["router"] = (1.5 / math.sqrt(h) * normal(e, h)).to(dt)
        s["bias"] = 0.1 * normal(e) if case["bias"] else None
        for name, n, k in (("gate", i, h), ("up", i, h), ("down", h, i)):
            s[name], s[name + "_scale"] = _weight(normal, (e,), n, k, case["weights"])
        s["r"] = normal(m, h).to(dt) if case["residual"] else None
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


def _expand(scale, n, k):
    """Block scales [..., nb, kb] for the [..., n, k] weight."""
    return scale.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _plain_rows(s):
    c = s["case"]
    kept = None
    if c["op"] == "norm":
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
            kept = h.to(s["x"].dtype)
        v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].float()
    else:
        v = _act(s["gate"].float(), c["act"])
        if s["up"] is not None:
            v = v * s["up"].float()
    cols = v.shape[1]
    b = _padded(v, _blocks(cols) * BLOCK).reshape(v.shape[0], -1, BLOCK)
    scales = (b.abs().amax(2) / E4M3_MAX).clamp_min(2.0 ** -126)
    codes = (b / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(v.shape[0], -1)[:, :cols]
    return [codes.to(torch.float8_e4m3fn), scales, kept]


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float() * s["xs"].repeat_interleave(BLOCK, 1)[:, :c["k"]]
    y = torch.matmul(x, (s["w"].float() * _expand(s["ws"], c["n"], c["k"])).t())
    if s["b"] is not None:
        y = y + s["b"].float()
    y = _act(y, c["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    return [y.to(TYPES[c["dst"]])]


def _route(s, logits):
    """(chosen experts, their weights) of logits in 64 bits."""
    c = s["case"]
    score = torch.softmax(logits, 1) if c["score"] == "softmax" else torch.sigmoid(logits)
    key = score if s["bias"] is None else score + s["bias"].double()
    experts = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["top"]]
    p = score.gather(1, experts)
    if c["normalize"]:
        p = p / p.sum(1, keepdim=True)
    return experts, c["factor"] * p


def _plain_moe(s):
    c = s["case"]
    m, top, h, i = c["m"], c["top"], c["h"], c["i"]
    # Which experts are chosen turns on the last digits of the logits.
    experts, p = _route(s, s["x"].double() @ s["router"].double().t())
    at, p = experts.flatten(), p.float()

    def chosen(name, n, k):
        w = s[name][at].float()
        return w if s[name + "_scale"] is None else w.mul_(_expand(s[name + "_scale"][at], n, k))

    x = s["x"].float().repeat_interleave(top, 0)[:, :, None]
    v = _act(torch.bmm(chosen("gate", i, h), x), c["act"]) * torch.bmm(chosen("up", i, h), x)
    y = (torch.bmm(chosen("down", h, i), v).reshape(m, top, h) * p[:, :, None]).sum(1)
    if s["r"] is not None:
        y = y + s["r"].float()
    return [y.to(s["x"].dtype), experts.int(), p]


def run(state):
    c = state["case"]
    if not own:
        return _plain_linear(state) if c["op"] == "linear" else _plain_moe(state) if c["op"] == "moe" else _plain_rows(state)
    from safetensors_materialization_gb300 import stmat
    if c["op"] == "linear":
        return [stmat.block_linear(state["x"], state["w"], state["xs"], state["ws"], bias=state["b"], act=c["act"],
                                   residual=state["r"], dst=c["dst"])]
    if c["op"] == "moe":
        return list(stmat.moe(state["x"], state["router"], state["gate"], state["up"], state["down"], c["top"],
                              gate_scale=state["gate_scale"], up_scale=state["up_scale"], down_scale=state["down_scale"],
                              act=c["act"], score=c["score"], normalize=c["normalize"], factor=c["factor"],
                              router_bias=state["bias"], residual=state["r"]))
    if c["op"] == "norm":
        return list(stmat.rms_norm(state["x"], state["w"], eps=EPS, residual=state["r"], dst="F8_E4M3", block=BLOCK))
    return [*stmat.gated_act(state["gate"], state["up"], act=c["act"], dst="F8_E4M3", block=BLOCK), None]


def work(case):
    m = case["m"]
    if case["op"] == "linear":
        n, k, out = case["n"], case["k"], SIZE[case["dst"]]
        moved = m * k + n * k + 4 * _blocks(k) * (m + _blocks(n)) + out * m * n * (2 if case["residual"] else 1)
        return {"bytes": moved + (out * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if case["op"] == "moe":
        e, h, i, size = case["e"], case["h"], case["i"], SIZE[case["type"]]
        # Experts that some token chooses, expected if all are alike.
        used = e * (1.0 - (1.0 - case["top"] / e) ** m)
        expert = 3 * h * i * SIZE[case["weights"]]
        expert += 4 * 3 * _blocks(h) * _blocks(i) if case["weights"] == "F8_E4M3" else 0
        moved = used * expert + size * (e * h + m * h * (3 if case["residual"] else 2)) + 8 * m * case["top"]
        return {"bytes": moved, "flops": 2 * m * h * e + 6 * m * case["top"] * h * i}
    c, size = case["c"], SIZE[case["type"]]
    if case["op"] == "norm":
        return {"bytes": m * c * ((3 if case["residual"] else 1) * size + 1) + c * size + 4 * m * _blocks(c), "flops": 6 * m * c}
    return {"bytes": m * c * ((2 if case["gated"] else 1) * size + 1) + 4 * m * _blocks(c), "flops": 8 * m * c}


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


def _exact_rows(s):
    c, kept = s["case"], None
    if c["op"] == "norm":
        h = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
        kept = h if s["r"] is not None else None
        v = h / (h.square().sum(1, keepdim=True) / c["c"] + EPS).sqrt() * s["w"].double()
    else:
        v = _exact_act(s["gate"].double(), c["act"])
        v = v if s["up"] is None else v * s["up"].double()
    scales = torch.stack([b.abs().max(dim=1).values for b in v.split(BLOCK, 1)], 1) / E4M3_MAX
    scales = torch.clamp(scales, min=2.0 ** -126)
    # Codes are compared with the quotient that they round.
    return [torch.cat([b / scales[:, j:j + 1] for j, b in enumerate(v.split(BLOCK, 1))], 1), scales, kept]


def _exact_weight(w, scale):
    """One weight [n, k] in 64 bits."""
    w = w.double()
    if scale is not None:
        w = w.clone()
        for a in range(scale.shape[0]):
            rows = w[a * BLOCK:(a + 1) * BLOCK]
            rows *= torch.cat([scale[a].double().reshape(-1, 1)] * BLOCK, 1).reshape(-1)[:w.shape[1]]
    return w


def _exact_linear(s):
    c = s["case"]
    wt, y = _exact_weight(s["w"], s["ws"]).t(), []
    step = max(1, min(c["m"], (1 << 27) // max(c["n"], c["k"])))
    for a in range(0, c["m"], step):
        x = s["x"][a:a + step].double()
        for j in range(s["xs"].shape[1]):
            x[:, j * BLOCK:(j + 1) * BLOCK] *= s["xs"][a:a + step, j:j + 1].double()
        v = x @ wt
        v = _exact_act(v if s["b"] is None else v + s["b"].double(), c["act"])
        y.append(v if s["r"] is None else v + s["r"][a:a + step].double())
    return [torch.cat(y)]


def _exact_moe(s):
    c = s["case"]
    logits = torch.einsum("mh,eh->me", s["x"].double(), s["router"].double())
    if c["score"] == "softmax":
        score = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    key = score.clone() if s["bias"] is None else score + s["bias"].double()
    rows = torch.arange(c["m"], device=key.device)
    experts = []
    for _ in range(c["top"]):  # argmax on the host: the first of equal ones
        best = torch.as_tensor(key.cpu().numpy().argmax(1), device=key.device)
        experts.append(best)
        key[rows, best] = -math.inf
    experts = torch.stack(experts, 1)
    p = torch.gather(score, 1, experts)
    p = c["factor"] * (p / p.sum(1, keepdim=True) if c["normalize"] else p)
    y = torch.zeros(c["m"], c["h"], dtype=torch.float64, device=key.device)
    for e in torch.unique(experts).tolist():
        token, place = torch.nonzero(experts == e, as_tuple=True)
        w = [_exact_weight(s[n][e], None if s[n + "_scale"] is None else s[n + "_scale"][e]) for n in ("gate", "up", "down")]
        x = s["x"][token].double()
        v = _exact_act(x @ w[0].t(), c["act"]) * (x @ w[1].t())
        y.index_add_(0, token, (v @ w[2].t()) * p[token, place].unsqueeze(1))
    return [y if s["r"] is None else y + s["r"].double(), experts.int(), p]


def exact(case, seed):
    """The formulas at the top in 64 bits, without the roundings at the end."""
    s = _inputs(case, seed)
    return _exact_linear(s) if case["op"] == "linear" else _exact_moe(s) if case["op"] == "moe" else _exact_rows(s)

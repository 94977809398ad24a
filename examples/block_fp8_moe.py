"""A mixture-of-experts layer run from a block-scaled FP8 checkpoint without ever
dequantizing its weights.

A checkpoint has a tensor for every expert's gate, up and down projection, and
one for its scales.  One launch materializes them, as they are stored, into the
stacked tensors that the layer takes: an output's destination is its expert's
place in the stack.  Each call then is

    y, _, h = rms_norm(x, norm, residual)
    out, experts, weights = moe(y, router, gate, up, down, top_k, gate_scale=..., residual=h)

for up to 64 tokens, without host synchronization.

    python examples/block_fp8_moe.py
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

PROJECTIONS = ("gate", "up", "down")


def blocks(n):
    return -(-n // 128)


def block_scaled(w):
    """E4M3 codes and the scales of 128 x 128 blocks, amax / 448."""
    import torch
    n, k = w.shape
    pad = torch.nn.functional.pad(w, (0, blocks(k) * 128 - k, 0, blocks(n) * 128 - n))
    b = pad.reshape(blocks(n), 128, blocks(k), 128)
    scale = (b.abs().amax((1, 3)) / 448).clamp_min(2.0 ** -126)
    codes = (b / scale[:, None, :, None]).reshape(pad.shape)[:n, :k].to(torch.float8_e4m3fn)
    return codes.contiguous(), scale


def checkpoint(hidden, inter, experts, seed=0):
    """File image of a one-layer checkpoint: weights N(0, 0.02)."""
    import torch
    from safetensors_materialization_gb300 import synth
    g = torch.Generator().manual_seed(seed)
    tensors = {"norm.weight": ("BF16", (1 + 0.1 * torch.randn(hidden, generator=g)).to(torch.bfloat16)),
               "router.weight": ("BF16", (1.5 / hidden ** 0.5 * torch.randn(experts, hidden, generator=g)).to(torch.bfloat16))}
    for e in range(experts):
        for name in PROJECTIONS:
            shape = (hidden, inter) if name == "down" else (inter, hidden)
            codes, scale = block_scaled(0.02 * torch.randn(*shape, generator=g))
            tensors[f"experts.{e}.{name}.weight"] = ("F8_E4M3", codes)
            tensors[f"experts.{e}.{name}.weight_scale_inv"] = ("F32", scale)
    entries = sorted((synth.Entry(n, dt, list(t.shape)) for n, (dt, t) in tensors.items()), key=lambda e: e.name)
    layout = synth.make_layout(entries)
    image = synth.build_file(layout, seed)
    for e in layout.entries:
        raw = tensors[e.name][1].contiguous().reshape(-1).view(torch.uint8).numpy()
        image[layout.data_start + e.begin:layout.data_start + e.end] = raw
    return image


class BlockFp8Moe:
    """The layer on the GPU, its experts stacked as the checkpoint stores them."""

    def __init__(self, image, top_k):
        import torch
        from safetensors_materialization_gb300 import stmat
        index = stmat.Index.from_file(image)
        plan = index.plan(dst="KEEP")
        outputs = plan.outputs()
        experts = 1 + max(int(o["name"].split(".")[1]) for o in outputs if o["name"].startswith("experts."))
        self.w, places = {}, []
        for o in outputs:
            parts, dtype, shape = o["name"].split("."), stmat.torch_dtype(o["dtype"]), tuple(o["shape"])
            if parts[0] == "experts":
                name = parts[2] if parts[3] == "weight" else parts[2] + "_scale"
                if name not in self.w:
                    self.w[name] = torch.empty(experts, *shape, dtype=dtype, device="cuda")
                places.append(self.w[name][int(parts[1])].data_ptr())
            else:
                self.w[parts[0]] = torch.empty(shape, dtype=dtype, device="cuda")
                places.append(self.w[parts[0]].data_ptr())
        section = torch.from_numpy(image[image.size - index.sizes()[1]:].copy()).cuda()
        plan.materialize(section, torch.tensor(places, dtype=torch.int64, device="cuda"))
        plan.check()  # waits, so that the section may go
        self.top_k = top_k

    def experts(self, y, residual=None):
        """(sum of the experts, with the residual's addition, chosen experts,
        their weights) of normed rows y."""
        from safetensors_materialization_gb300 import stmat
        w = self.w
        return stmat.moe(y, w["router"], w["gate"], w["up"], w["down"], self.top_k, gate_scale=w["gate_scale"],
                         up_scale=w["up_scale"], down_scale=w["down_scale"], residual=residual)

    def __call__(self, x, residual):
        """(layer's output added to the residual stream, that stream before)."""
        from safetensors_materialization_gb300 import stmat
        y, _, h = stmat.rms_norm(x, self.w["norm"], residual=residual)
        return self.experts(y, h)[0], h


def dequantized(layer, y, experts, weights):
    """The layer's sum of experts in 64 bits, on the stacked weights with their
    scales, for rows y and a given choice."""
    import torch
    w = layer.w

    def full(name, e):
        codes, scale = w[name][e].double(), w[name + "_scale"][e].double()
        return codes * scale.repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]

    out = torch.zeros(y.shape, dtype=torch.float64, device=y.device)
    for e in experts.unique().tolist():
        token, place = torch.nonzero(experts == e, as_tuple=True)
        x = y[token].double()
        v = torch.nn.functional.silu(x @ full("gate", e).t()) * (x @ full("up", e).t())
        out.index_add_(0, token, (v @ full("down", e).t()) * weights[token, place].double().unsqueeze(1))
    return out


def main(hidden=1024, inter=704, experts=16, top_k=4, tokens=(1, 13, 64)):
    """Relative difference of the experts' sum from the one in 64 bits, per
    number of tokens."""
    import torch
    from safetensors_materialization_gb300 import stmat
    layer = BlockFp8Moe(checkpoint(hidden, inter, experts), top_k)
    found = {}
    for m in tokens:
        g = torch.Generator().manual_seed(m)
        x, r = (torch.randn(m, hidden, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        out, h = layer(x, r)
        y = stmat.rms_norm(x, layer.w["norm"], residual=r)[0]
        added, chosen, weights = layer.experts(y)
        want = dequantized(layer, y, chosen, weights)
        assert out.shape == h.shape == x.shape
        found[m] = float((added.double() - want).norm() / want.norm())
        print(f"{m} tokens, {top_k} of {experts} experts of {hidden} -> {inter}: {found[m]:.5f} off the layer in 64 bits")
    return found


if __name__ == "__main__":
    main()

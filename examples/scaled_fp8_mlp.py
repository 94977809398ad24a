"""A transformer's gated MLP run from a scaled-FP8 checkpoint without ever
dequantizing its weights.

The checkpoint's weights are materialized as they are stored (E4M3 codes, one
F32 scale each); the norm's vector is BF16.  Each call then is

    y8, s, h = rms_norm(x, norm, residual, dst="F8_E4M3")   rows in 8 bits, one scale each
    z        = linear(y8, gate_up, x_scale=s, w_scale=...)  BF16
    a8, t    = gated_act(z[:, :i], z[:, i:], "silu", dst="F8_E4M3")
    out      = linear(a8, down, x_scale=t, w_scale=..., residual=h)

four launches, for one token or thousands,
without host synchronization (so that it can be captured in a CUDA graph).

    python examples/scaled_fp8_mlp.py
"""
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def checkpoint(hidden, inter, seed=0):
    """File image of a one-layer scaled-FP8 checkpoint: weights N(0, 0.02) with
    amax / 448 as their scale, the norm's vector near 1."""
    import torch
    from safetensors_materialization_gb300 import synth
    g = torch.Generator().manual_seed(seed)
    tensors = {"mlp.norm.weight": ("BF16", (1 + 0.1 * torch.randn(hidden, generator=g)).to(torch.bfloat16))}
    for name, shape in (("gate_up", (2 * inter, hidden)), ("down", (hidden, inter))):
        w = 0.02 * torch.randn(*shape, generator=g)
        scale = w.abs().max() / 448
        tensors[f"mlp.{name}.weight"] = ("F8_E4M3", (w / scale).to(torch.float8_e4m3fn))
        tensors[f"mlp.{name}.scale_weight"] = ("F32", scale.reshape(()))
    entries = sorted((synth.Entry(n, dt, list(t.shape)) for n, (dt, t) in tensors.items()), key=lambda e: e.name)
    layout = synth.make_layout(entries)
    image = synth.build_file(layout, seed)
    for e in layout.entries:
        raw = tensors[e.name][1].contiguous().reshape(-1).view(torch.uint8).numpy()
        image[layout.data_start + e.begin:layout.data_start + e.end] = raw
    return image


class ScaledFp8Mlp:
    """The block on the GPU, its weights as the checkpoint stores them."""

    def __init__(self, image, prefix="mlp."):
        import torch
        from safetensors_materialization_gb300 import stmat
        index = stmat.Index.from_file(image).view_prefix(prefix)
        plan = index.plan(dst="KEEP")
        self.outputs = stmat.Outputs(plan)
        section = torch.from_numpy(image[image.size - index.sizes()[1]:].copy()).cuda()
        plan.materialize(section, self.outputs.ptrs)
        plan.check()  # waits, so that the section may go
        self.w = self.outputs.tensors()

    def __call__(self, x, residual):
        """(block's output added to the residual stream, that stream before)."""
        from safetensors_materialization_gb300 import stmat
        w = self.w
        y8, s, h = stmat.rms_norm(x, w["norm.weight"], residual=residual, dst="F8_E4M3")
        z = stmat.linear(y8, w["gate_up.weight"], x_scale=s, w_scale=w["gate_up.scale_weight"])
        inter = z.shape[-1] // 2
        a8, t = stmat.gated_act(z[..., :inter], z[..., inter:], act="silu", dst="F8_E4M3")
        return stmat.linear(a8, w["down.weight"], x_scale=t, w_scale=w["down.scale_weight"], residual=h), h


def dequantized(image, x, residual):
    """The same block on weights materialized to F32 with their scales, in
    torch, nothing in 8 bits on the way: what the rounding of the activations
    is measured against."""
    import torch
    from safetensors_materialization_gb300 import stmat
    index = stmat.Index.from_file(image).view_prefix("mlp.")
    plan = index.plan(dst="F32", scale_suffix=(".weight", ".scale_weight"))
    outputs = stmat.Outputs(plan)
    section = torch.from_numpy(image[image.size - index.sizes()[1]:].copy()).cuda()
    plan.materialize(section, outputs.ptrs)
    plan.check()
    w = outputs.tensors()
    h = x.float() + residual.float()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5) * w["norm.weight"]
    z = y @ w["gate_up.weight"].t()
    inter = z.shape[-1] // 2
    return h + torch.nn.functional.silu(z[..., :inter]) * z[..., inter:] @ w["down.weight"].t(), h


def main(hidden=2048, inter=5504, tokens=(1, 37, 700)):
    """Relative difference of the block's addition to the residual stream from
    the one without 8-bit activations, per number of tokens."""
    import torch
    image = checkpoint(hidden, inter)
    mlp = ScaledFp8Mlp(image)
    found = {}
    for m in tokens:
        g = torch.Generator().manual_seed(m)
        x, r = (torch.randn(m, hidden, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        out, h = mlp(x, r)
        want, h32 = dequantized(image, x, r)
        added = want - h32
        found[m] = float((out.double() - h.double() - added.double()).norm() / added.double().norm())
        print(f"{m} tokens of {hidden} -> {inter}: {found[m]:.4f} off the block without 8-bit activations")
    return found


if __name__ == "__main__":
    main()

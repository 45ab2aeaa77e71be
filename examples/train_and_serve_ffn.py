"""A gated feed-forward block from training to serving.

Trains a block in bf16 to imitate another one (forward and backward on the
GPU, plain gradient descent on fp32 master weights), quantises the trained
weights to MXFP4, serves prompts and single tokens from them, and prints how
far the served outputs are from the trained block's.

  python examples/train_and_serve_ffn.py [--hidden 1024] [--inter 2048] [--tokens 2048] [--steps 200]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_ffn_gemv_gb300 import binding  # noqa: E402


def rel(a, b) -> float:
    return float((a.float() - b.float()).norm() / b.float().norm())


def run(hidden=1024, inter=2048, tokens=2048, steps=200, lr=0.05, act="silu", log=print):
    """Returns the first and last training loss, and the relative error of the block served
    from MXFP4 weights against the trained bf16 block, for a prompt and for one token."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, std):
        return torch.randn(shape, generator=g, device="cuda") * std

    shapes = ((inter, hidden, hidden ** -0.5), (inter, hidden, hidden ** -0.5), (hidden, inter, inter ** -0.5))
    teacher = binding.GatedFfn(*[normal(r, c, std=s).bfloat16() for r, c, s in shapes], act=act)
    master = [normal(r, c, std=s) for r, c, s in shapes]  # fp32
    weights = [w.bfloat16() for w in master]              # what the block reads, updated in place
    block = binding.GatedFfn(*weights, act=act)
    losses = []
    for step in range(steps):
        x = normal(tokens, hidden, std=1.0).bfloat16()
        want = teacher.forward(x)
        out, saved = block.forward(x, save=True)
        diff = out.float() - want.float()
        if step % 20 == 0 or step == steps - 1:
            losses.append(float(diff.square().sum(1).mean()))
            log(f"step {step:4d}  loss {losses[-1]:.4f}")
        _, dw1, dw3, dw2 = block.backward((2.0 / tokens * diff).bfloat16(), x, saved, need_dx=False)
        for m, w, dw in zip(master, weights, (dw1, dw3, dw2)):
            m.sub_(dw.float(), alpha=lr)
            w.copy_(m)
    served = binding.GatedFfn(*[binding.moe_mxfp4_quant(w) for w in master], act=act)
    x = normal(tokens, hidden, std=1.0).bfloat16()
    trained = block.forward(x)
    prompt, token = rel(served.forward(x), trained), rel(served.forward(x[:1]), trained[:1])
    if block.device_status() or served.device_status():
        raise RuntimeError("device error word set")
    held = sum(w.numel() * 2 for w in weights), sum(w.numel() * 17 // 32 for w in weights)
    log(f"served from MXFP4: {held[0]} -> {held[1]} weight bytes, relative error {prompt:.3f} (prompt), {token:.3f} (token)")
    return losses[0], losses[-1], prompt, token


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=2048)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--act", choices=("silu", "gelu"), default="silu")
    a = ap.parse_args()
    run(a.hidden, a.inter, a.tokens, a.steps, act=a.act)

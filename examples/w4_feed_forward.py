"""A gated feed-forward block on 4-bit group-quantized weights: trained for a few steps
with straight-through gradients, then asked for single tokens.

    python examples/w4_feed_forward.py [--tokens 4096] [--width 1024] [--hidden 2816] [--steps 5]

The float32 master weights are quantized group by group after every update
(fq.quant_groups); the products read the packed codes (fake_quant_amd.linear):

    h = silu(x Wg^T) (x Wu^T),  y = h Wd^T,  loss = |y - target|^2 / 2
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from fake_quant_amd import fq, linear  # noqa: E402

GROUP = 64


def quantized(master):
    return fq.quant_groups(master, GROUP, 4, fq.AFFINE, want_fq=False)


def run(tokens=4096, width=1024, hidden=2816, steps=5, lr=0.2, device="cuda"):
    """Losses per token before each step, and the largest difference between the block on
    one token alone and on all of them, relative to the largest output."""
    gen = torch.Generator(device=device).manual_seed(1)

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=gen, device=device) * sigma

    masters = [normal(hidden, width, sigma=width ** -0.5), normal(hidden, width, sigma=width ** -0.5),
               normal(width, hidden, sigma=hidden ** -0.5)]
    x = normal(tokens, width).bfloat16()
    target = normal(tokens, width, sigma=0.1).bfloat16()
    losses = []
    for _ in range(steps):
        wg, wu, wd = (quantized(m) for m in masters)
        h, g, u = linear.w4_gated(x, wg, wu, GROUP, "silu", save=True)
        y = linear.w4_matmul(h, wd, GROUP)
        diff = y.float() - target.float()
        losses.append(float(diff.square().sum()) / (2 * tokens))
        dh, dwd = linear.w4_matmul_backward(diff.bfloat16(), h, wd, GROUP)
        _, dwg, dwu = linear.w4_gated_backward(dh, x, g, u, wg, wu, GROUP, "silu", want_dx=False, dw_dtype=torch.float32)
        for master, grad in zip(masters, (dwg, dwu, dwd)):
            master -= lr / tokens * grad
    wg, wu, wd = (quantized(m) for m in masters)
    everything = linear.w4_matmul(linear.w4_gated(x, wg, wu, GROUP), wd, GROUP)
    apart = 0.0
    for i in range(min(4, tokens)):
        one = linear.w4_matmul(linear.w4_gated(x[i:i + 1], wg, wu, GROUP), wd, GROUP)
        apart = max(apart, float((one.float() - everything[i:i + 1].float()).abs().max()))
    return losses, apart / float(everything.float().abs().max())


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("width", 1024), ("hidden", 2816), ("steps", 5)):
        p.add_argument("--" + name, type=int, default=value)
    losses, apart = run(**vars(p.parse_args()))
    for i, loss in enumerate(losses):
        print(f"step {i}: loss {loss:.4f} a token")
    print(f"single tokens differ from the batch by {apart:.1e} of the largest output")


if __name__ == "__main__":
    main()

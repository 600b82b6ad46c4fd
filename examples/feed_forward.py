"""A feed-forward block trained, quantised and served with this library.

A gated block with 16-bit weights learns to imitate another one: forward and
backward pass (ffn_forward, ffn_backward), and an AdamW step (AdamW) with 8-bit
states on FP32 master weights that writes the 16-bit weights back.  Then its
weights are quantised to four bits (w4_quantize) and single tokens go through
the quantised block (W4Matrix.matvec) and through the 16-bit one.

    python examples/feed_forward.py [steps]
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import dense_fp32_sgemm_gb300 as sg


def block_weights(D, F, gen, dtype):
    def normal(rows, cols):
        return (torch.randn(rows, cols, generator=gen, device="cuda") * rows ** -0.5).to(dtype)

    return [normal(D, F), normal(D, F), normal(F, D)]


def train(steps=60, T=512, D=256, F=768, seed=1, dtype=torch.bfloat16):
    """Returns the trained weights and the mean squared errors, one per step."""
    gen = torch.Generator("cuda").manual_seed(seed)
    teacher, weights = block_weights(D, F, gen, dtype), block_weights(D, F, gen, dtype)
    masters = [w.float() for w in weights]
    grads = [torch.empty_like(w) for w in weights]
    opt = sg.AdamW(masters, grads, copies=weights, lr=4e-3, weight_decay=0.0, state_bits=8)
    saved = sg.ffn_saved(T, F, dtype=dtype)
    losses = []
    for _ in range(steps):
        x = torch.randn(T, D, generator=gen, device="cuda").to(dtype)
        want = sg.ffn_forward(x, *teacher)
        y = sg.ffn_forward(x, *weights, saved=saved)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        dy = (diff * (2.0 / diff.numel())).to(dtype)
        sg.ffn_backward(dy, x, *weights, dw_gate=grads[0], dw_up=grads[1], dw_down=grads[2],
                        saved=saved, need_dx=False)
        opt.step()
    return weights, [float(v) for v in torch.stack(losses).cpu()]


def serve(weights, tokens=4, group=64, seed=2):
    """Single tokens through the 4-bit and the 16-bit block; returns the relative
    difference of their outputs."""
    gen = torch.Generator("cuda").manual_seed(seed)
    gate, up, down = (sg.w4_quantize(w, group) for w in weights)
    off = size = 0.0
    for _ in range(tokens):
        x = torch.randn(1, gate.K, generator=gen, device="cuda").to(weights[0].dtype)
        g, u = gate.matvec(x).float(), up.matvec(x).float()
        y = down.matvec((g * torch.sigmoid(g) * u).to(x.dtype)).float()
        want = sg.ffn_forward(x, *weights).float()
        off += float((y - want).square().sum())
        size += float(want.square().sum())
    return (off / size) ** 0.5


def main(steps=60):
    sg.build()
    weights, losses = train(steps)
    print(f"mean squared error: {losses[0]:.4f} at the first step, {losses[-1]:.4f} at step {steps}")
    print(f"4-bit weights: outputs {serve(weights):.3f} off the 16-bit block's")


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 60)

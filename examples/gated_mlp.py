"""Fine-tune a gated MLP block, then serve it with the adapters of several requests.

    python examples/gated_mlp.py [--hidden 896 --intermediate 4864 --tokens 512 --steps 30]

Out = x + (SiLU(x W1) * (x W2)) W3. Training runs the fused forward, the
down-projection with its residual, and both gradients through torch.autograd;
the float32 master weights are packed once per step. Serving keeps the trained
block packed and answers a batch whose tokens belong to requests with adapters
of their own (or none) in one pass over the shared weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_gated_mlp_gb300 as sg  # noqa: E402


class GatedMLP(torch.autograd.Function):
    """x [M, H], w1 and w2 [H, N], w3 [N, H], all bf16 -> x + (SiLU(x w1) * (x w2)) w3."""

    @staticmethod
    def forward(ctx, x, w1, w2, w3):
        wp, w3p = sg.swiglu_pack_weights(w1, w2), sg.swiglu_pack_down_weights(w3)
        y = sg.swiglu_forward(x, wp, w1.shape[1])
        ctx.save_for_backward(x, y, wp, w3p)
        return sg.swiglu_down_forward(y, w3p, w3.shape[1], R=x)

    @staticmethod
    def backward(ctx, d_out):
        x, y, wp, w3p = ctx.saved_tensors
        d_out = d_out.contiguous()
        need_x, need_w1, need_w2, need_w3 = ctx.needs_input_grad
        d_y, d_w3 = sg.swiglu_down_backward(d_out, w3p, y, need_weight=need_w3)
        # one product makes both of the gate's and the up weight's gradients
        d_x, d_w1, d_w2 = sg.swiglu_backward(x, wp, d_y, need_input=need_x, need_weight=need_w1 or need_w2)
        return d_x + d_out if need_x else None, d_w1 if need_w1 else None, d_w2 if need_w2 else None, d_w3


def train(hidden, intermediate, tokens, steps, lr=2e-2):
    """Fits a random block to another one's outputs; returns the losses and the trained weights."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def weights():
        shapes = ((hidden, intermediate), (hidden, intermediate), (intermediate, hidden))
        return [torch.randn(*s, generator=g, device="cuda") / s[0] ** 0.5 for s in shapes]

    teacher = [w.bfloat16() for w in weights()]
    student = [torch.nn.Parameter(t.float() + 0.3 * w) for t, w in zip(teacher, weights())]
    opt = torch.optim.Adam(student, lr=lr / hidden ** 0.5)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
        out = GatedMLP.apply(x, *(w.bfloat16() for w in student))
        loss = (out.float() - GatedMLP.apply(x, *teacher).float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    sg.swiglu_check_device_status()
    return losses, [w.detach().bfloat16() for w in student]


def serve(w1, w2, w3, adapters=4, rank=16, tokens=24):
    """One batch of tokens of several requests; returns the outputs and those of merged weights."""
    hidden, n = w1.shape
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()

    # the table that the requests share: gate and up halves, then the down-projection's
    la, lb = normal(adapters, 2, rank, hidden, std=hidden ** -0.5), normal(adapters, 2, n, rank, std=0.3 * rank ** -0.5)
    la3, lb3 = normal(adapters, rank, n, std=n ** -0.5), normal(adapters, hidden, rank, std=0.3 * rank ** -0.5)
    scale = torch.full((adapters,), 2.0, device="cuda")
    x = normal(tokens, hidden, std=1.0)
    index = torch.arange(tokens, device="cuda", dtype=torch.int32) % (adapters + 1) - 1  # -1: no adapter

    wp, w3p = sg.swiglu_pack_weights(w1, w2), sg.swiglu_pack_down_weights(w3)
    ws = sg.swiglu_lora_workspace(tokens, hidden, n, rank)
    ws3 = sg.swiglu_down_lora_workspace(tokens, n, hidden, rank)
    y = sg.swiglu_forward_lora(x, wp, n, la, lb, index, scale, workspace=ws)
    out = sg.swiglu_down_forward_lora(y, w3p, hidden, la3, lb3, index, scale, R=x, workspace=ws3)
    sg.swiglu_check_device_status()

    want = torch.empty_like(out)
    for a in range(-1, adapters):  # each request alone, with its adapter merged into the weights
        rows = (index == a).nonzero().reshape(-1)
        m1, m2, m3 = w1.float(), w2.float(), w3.float()
        if a >= 0:
            m1 = m1 + scale[a] * (lb[a, 0].float() @ la[a, 0].float()).t()
            m2 = m2 + scale[a] * (lb[a, 1].float() @ la[a, 1].float()).t()
            m3 = m3 + scale[a] * (lb3[a].float() @ la3[a].float()).t()
        xr = x[rows].float()
        want[rows] = (xr + (torch.nn.functional.silu(xr @ m1) * (xr @ m2)) @ m3).bfloat16()
    return out, want


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=896)
    ap.add_argument("--intermediate", type=int, default=4864)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args(argv)
    losses, weights = train(a.hidden, a.intermediate, a.tokens, a.steps)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps of {a.tokens} tokens")
    out, want = serve(*weights)
    off = ((out.float() - want.float()).norm() / want.float().norm()).item()
    print(f"serving: {out.shape[0]} tokens of 5 requests, {off:.1e} off the merged weights")
    return losses, off


if __name__ == "__main__":
    main()

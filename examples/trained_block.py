"""A training step of one block, norm, router and experts, that keeps its activations in 8 bits.

  python examples/trained_block.py [--tokens 512] [--hidden 1024] [--inner 512] [--experts 16] [--topk 4]

Forward: h = x + residual goes through the norm (rms_norm), whose rows feed the router and
the experts and whose 8-bit form is what is kept of them; the experts' first product gives
gate and up, swiglu the activation times the router's weights, both kept in 8 bits; the
second product's rows are summed back to the tokens.

Backward: gradients of the experts' weights from the kept rows (weight_grad), of gate, up
and the router's weights from the kept gate and up (swiglu_backward), of the tokens
(permute_backward, route_backward) and of the norm (rms_norm_backward).

Kept between the two: h, 1 byte per element of the norm's rows (per token, not per expert),
3 of the inner rows, and their scales, a 32nd of that; no row of the experts' results.
Everything is compared with autograd in fp32, once as it is and once with the kept values
in the place of the activations that they were made from.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_forward_gb300 as M  # noqa: E402
from moe_expert_forward_gb300 import ops  # noqa: E402


def spans(r):
    """The rows of each expert."""
    blk, cnt = r.blk_off.tolist(), r.cnt.tolist()
    return [slice(blk[e] * r.block_m, blk[e] * r.block_m + cnt[e]) for e in range(r.E)]


def forward(x, residual, weight, router, w1, w2, k):
    """(output, h, what the backward pass takes)."""
    n = ops.rms_norm(x, weight, residual=residual, quant="mx")
    logits = n.y.float() @ router.t()
    idx, topk_w = ops.route(logits, k)
    r = ops.sort_tokens(idx, w1.shape[0])
    rows = ops.permute(n.y, r)
    first = torch.empty(r.rows, w1.shape[1], dtype=x.dtype, device=x.device)
    for e, s in enumerate(spans(r)):
        first[s] = rows[s] @ w1[e].t()
    f = ops.swiglu(first, r, topk_w, quant=True, keep=True)
    down = torch.empty(r.rows, w2.shape[1], dtype=x.dtype, device=x.device)
    for e, s in enumerate(spans(r)):
        down[s] = f.a[s] @ w2[e].t()
    out = ops.unpermute(down, r)                               # the weights are in the activation
    return out, n.h, (n.h, n.rstd, (n.codes, n.sf), logits, idx, topk_w, r, (f.codes, f.sf), (f.kept, f.kept_sf))


def backward(kept, d_out, d_h, weight, router, w1, w2):
    """Gradients of x (and the residual), the norm's weight, the logits and the experts' weights."""
    h, rstd, y8, logits, idx, topk_w, r, a8, gate_up8 = kept
    H, I = w1.shape[2], w2.shape[2]
    d_down, _ = ops.unpermute_backward(d_out, None, r)
    d_w2 = ops.weight_grad(d_down, *a8, I, r)
    d_a = torch.zeros(r.rows, I, dtype=d_out.dtype, device=d_out.device)
    for e, s in enumerate(spans(r)):
        d_a[s] = d_down[s] @ w2[e]
    d_first, d_topk_w = ops.swiglu_backward(d_a, *gate_up8, r, topk_w)
    d_w1 = ops.weight_grad(d_first, *y8, H, r, by_token=True)
    d_rows = torch.zeros(r.rows, H, dtype=d_out.dtype, device=d_out.device)
    for e, s in enumerate(spans(r)):
        d_rows[s] = d_first[s] @ w1[e]
    d_logits = ops.route_backward(logits, idx, d_topk_w)
    d_y = ops.permute_backward(d_rows, r).float() + d_logits @ router
    d_x, d_weight = ops.rms_norm_backward(d_y.to(d_out.dtype), h, weight, rstd, d_h=d_h)
    return {"x": d_x, "norm weight": d_weight, "logits": d_logits, "first weights": d_w1, "second weights": d_w2}


class _GatedAtKept(torch.autograd.Function):
    """gate * sigmoid(gate) * up * w forward, the gradients at the kept gate and up."""

    @staticmethod
    def forward(ctx, gate, up, w, kept_gate, kept_up):
        ctx.save_for_backward(kept_gate, kept_up, w)
        return gate * torch.sigmoid(gate) * up * w

    @staticmethod
    def backward(ctx, d):
        gate, up, w = ctx.saved_tensors
        s = torch.sigmoid(gate)
        return d * w * up * s * (1 + gate * (1 - s)), d * w * gate * s, (d * gate * s * up).sum(1, keepdim=True), None, None


class _Product(torch.autograd.Function):
    """x w^T forward, the weight's gradient at the kept x."""

    @staticmethod
    def forward(ctx, x, w, kept_x):
        ctx.save_for_backward(kept_x, w)
        return x @ w.t()

    @staticmethod
    def backward(ctx, d):
        x, w = ctx.saved_tensors
        return d @ w, d.t() @ x, None


def by_autograd(x, residual, weight, router, w1, w2, idx, d_out, d_h, kept=None):
    """(output, gradients) in fp32 with the experts idx; with `kept`, gradients at the values that the 8 bits stand for."""
    x, weight, w1, w2 = (t.detach().float().clone().requires_grad_() for t in (x, weight, w1, w2))
    h = x + residual.float()
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * weight
    logits = y @ router.t()
    logits.retain_grad()
    topk_w = torch.softmax(logits.gather(1, idx), dim=1)
    values = None
    if kept is not None:
        I = w2.shape[2]
        y8 = ops.dequantize8(*kept[2], x.shape[1], torch.float32)
        a8 = ops.dequantize8(*kept[7], I, torch.float32)
        codes, sf = kept[8]
        halves = [ops.dequantize8(codes[:, i].contiguous(), sf[:, i].contiguous(), I, torch.float32) for i in (0, 1)]
        values, slot = (y8, a8, *halves), kept[6].slot.long()
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        w = topk_w[t, j, None]
        if values is None:
            gate, up = (y[t] @ w1[e].t()).chunk(2, dim=1)
            part = (gate * torch.sigmoid(gate) * up * w) @ w2[e].t()
        else:
            rows = slot[t, j]
            gate, up = _Product.apply(y[t], w1[e], values[0][t]).chunk(2, dim=1)
            a = _GatedAtKept.apply(gate, up, w, values[2][rows], values[3][rows])
            part = _Product.apply(a, w2[e], values[1][rows])
        out = out.index_add(0, t, part)
    ((out * d_out.float()).sum() + (h * d_h.float()).sum()).backward()
    return out.detach(), {"x": x.grad, "norm weight": weight.grad, "logits": logits.grad, "first weights": w1.grad,
                          "second weights": w2.grad}


def off(a, b) -> float:
    """|a - b| / |b|, or |a| where b is nothing but rounding (one chosen expert's weight is always 1)."""
    size = float(b.float().norm())
    return float((a.float() - b.float()).norm()) / size if size > 1e-3 else float(a.float().norm()) * 1e-3


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 512), ("hidden", 1024), ("inner", 512), ("experts", 16), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()
    x, residual = randn(a.tokens, a.hidden), randn(a.tokens, a.hidden)
    weight = (1 + 0.1 * randn(a.hidden).float())
    router = torch.randn(a.experts, a.hidden, generator=g, device="cuda") * a.hidden ** -0.5
    w1 = randn(a.experts, 2 * a.inner, a.hidden, scale=a.hidden ** -0.5)
    w2 = randn(a.experts, a.hidden, a.inner, scale=a.inner ** -0.5)
    d_out, d_h = randn(a.tokens, a.hidden), randn(a.tokens, a.hidden)
    ops.sync_status()                                          # what other work of this process left there
    out, _, kept = forward(x, residual, weight, router, w1, w2, a.topk)
    mine = backward(kept, d_out, d_h, weight, router, w1, w2)
    code, where = ops.sync_status()                            # one check for all calls so far
    if code:
        raise M.MMError(code, f"a device wait (site {where})")
    idx = kept[4].long()               # one choice of experts for all: roundings of the logits move borders between them
    want, theirs = by_autograd(x, residual, weight, router, w1, w2, idx, d_out, d_h)
    _, at_kept = by_autograd(x, residual, weight, router, w1, w2, idx, d_out, d_h, kept)
    found = {"output against autograd": off(out, want)}
    for name in mine:
        found[f"gradient of {name} against autograd"] = off(mine[name], theirs[name])
        found[f"gradient of {name} at the kept values"] = off(mine[name], at_kept[name])
    for name, v in found.items():
        print(f"{name}: {v:.4f}")
    return found


if __name__ == "__main__":
    main()

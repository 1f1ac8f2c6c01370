"""One expert layer from bf16 tensors: routed, sorted, through 4-bit experts and back, and a training step.

  python examples/routed_layer.py [--tokens 512] [--hidden 1024] [--inner 512] [--experts 32] [--topk 4]

Serving: the experts' bf16 weights are quantised once into e2m1 with UE8M0
scales (mx_quantize).  A batch's router logits choose experts and weights
(route); the tokens go sorted by expert through gate and up, SwiGLU and down in
4 bits (sort_tokens, mx_linear, mx_quantize, mx_product) and back, weighted
(unpermute).  The same codes, choices and weights then run through the fused
layer (forward, 8-bit activations), which has to agree up to the activations'
formats.

Training: the same layer in bf16 between permute and unpermute, with its
gradients to the tokens and to the router's logits, one step against autograd.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_forward_gb300 as M  # noqa: E402
from moe_expert_forward_gb300 import ops  # noqa: E402


def quantised_experts(w):
    """w [E, N, C] bf16 -> codes [E, N, C/2] and scales [E, N, C/32], in the fused layer's layout."""
    E, N, C = w.shape
    codes, sf = ops.mx_quantize(w.reshape(E * N, C))
    return codes.view(E, N, C // 2), sf.view(E, N, C // 32)


def serve(x, router, w1, w2, k):
    """The layer on x [T, H] with 4-bit experts; returns the output and what the routing was."""
    (c1, s1), (c2, s2) = quantised_experts(w1), quantised_experts(w2)
    first, second = ops.mx_weights(c1, s1), ops.mx_weights(c2, s2)          # laid out once, kept with the model
    idx, weight = ops.route(x.float() @ router.t(), k)
    routing = ops.sort_tokens(idx, w1.shape[0], ops.PRODUCT_BLOCK)
    gate_up = ops.mx_linear(x, first, routing=routing)                      # [rows, 2 I], by expert
    gate, up = gate_up.float().chunk(2, dim=1)
    inner = (torch.nn.functional.silu(gate) * up).to(x.dtype)
    down = ops.mx_product(*ops.mx_quantize(inner, chunks=True), second, routing=routing)
    y = ops.unpermute(down, routing, weight)
    code, where = ops.sync_status()                                         # one check for all products so far
    if code:
        raise M.MMError(code, f"a 4-bit product (site {where})")
    return y, (idx, weight, c1, s1, c2, s2)


def fused(x, idx, weight, c1, s1, c2, s2):
    """The same codes through the fused layer: bf16 x, quantised to 8 bits on its way into the pool."""
    T, H = x.shape
    E, I = c1.shape[0], c1.shape[1] // 2
    opt = M.options(x_bf16=1)
    p1, p2 = M.prepare_weights(s1, s2, H, I, E, opt)
    ws = M.alloc_workspace(T, H, I, E, idx.shape[1], opt)
    out = torch.empty_like(x)
    M.forward(x, None, idx, weight, c1, p1, c2, p2, out, H, I, E, ws, opt)
    code, where = M.sync_status(ws)
    if code:
        raise M.MMError(code, f"forward (site {where})")
    return out


def train_step(x, router, w1, w2, k, d_out):
    """Gradients of sum(layer(x) * d_out) with respect to x (through the experts) and the router's logits."""
    logits = x.float() @ router.t()
    idx, weight = ops.route(logits, k)
    r = ops.sort_tokens(idx, w1.shape[0])
    rows = ops.permute(x, r)
    blk, cnt = r.blk_off.tolist(), r.cnt.tolist()
    spans = [slice(blk[e] * r.block_m, blk[e] * r.block_m + cnt[e]) for e in range(r.E)]
    down = torch.zeros_like(rows)
    kept = []
    for e, s in enumerate(spans):                                           # the experts' own products, in torch
        h = (rows[s] @ w1[e].t()).float()
        kept.append(h)
        gate, up = h.chunk(2, dim=1)
        down[s] = (torch.nn.functional.silu(gate) * up).to(x.dtype) @ w2[e].t()
    out = ops.unpermute(down, r, weight)
    d_down, d_weight = ops.unpermute_backward(d_out, down, r, weight)
    d_rows = torch.zeros_like(rows)
    for e, s in enumerate(spans):
        gate, up = kept[e].chunk(2, dim=1)
        d_inner = (d_down[s] @ w2[e]).float()
        sig = torch.sigmoid(gate)
        d_gate = d_inner * up * sig * (1 + gate * (1 - sig))
        d_rows[s] = torch.cat((d_gate, d_inner * gate * sig), 1).to(x.dtype) @ w1[e]
    return out, ops.permute_backward(d_rows, r), ops.route_backward(logits, idx, d_weight)


def train_step_autograd(x, router, w1, w2, k, d_out):
    """The same by autograd in fp32 over dense tensors."""
    x = x.float().requires_grad_()
    logits = (x.detach() @ router.t()).requires_grad_()
    top, idx = torch.topk(logits, k, dim=1)
    weight = torch.softmax(top, dim=1)
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        share = (weight * (idx == e)).sum(1, keepdim=True)
        gate, up = (x @ w1[e].float().t()).chunk(2, dim=1)
        out = out + share * ((torch.nn.functional.silu(gate) * up) @ w2[e].float().t())
    (out * d_out.float()).sum().backward()
    return out.detach(), x.grad, logits.grad


def off(a, b) -> float:
    """|a - b| / |b|."""
    return float((a.float() - b.float()).norm() / b.float().norm())


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 512), ("hidden", 1024), ("inner", 512), ("experts", 32), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()
    x = randn(a.tokens, a.hidden)
    router = torch.randn(a.experts, a.hidden, generator=g, device="cuda") * a.hidden ** -0.5
    w1 = randn(a.experts, 2 * a.inner, a.hidden, scale=a.hidden ** -0.5)
    w2 = randn(a.experts, a.hidden, a.inner, scale=a.inner ** -0.5)
    ops.sync_status()                                                       # what other work of this process left there
    y, kept = serve(x, router, w1, w2, a.topk)
    d_out = randn(a.tokens, a.hidden)
    mine = train_step(x, router, w1, w2, a.topk, d_out)
    theirs = train_step_autograd(x, router, w1, w2, a.topk, d_out)
    found = {"4-bit layer against the fused layer": off(y, fused(x, *kept)),
             "4-bit layer against fp32 weights": off(y, theirs[0]),
             "bf16 layer against autograd": off(mine[0], theirs[0]),
             "gradient of x against autograd": off(mine[1], theirs[1]),
             "gradient of the logits against autograd": off(mine[2], theirs[2])}
    for name, v in found.items():
        print(f"{name}: {v:.4f}")
    return found


if __name__ == "__main__":
    main()

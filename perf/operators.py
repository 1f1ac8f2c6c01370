"""Cases that measure the operators around the expert layer: the router's top-k
with its gradient, tokens sorted by expert and back with their gradients, and
microscaled 4-bit quantisation and product.

Each case is one call a user's program makes.  `run` computes it in plain torch
(32-bit arithmetic, rounded once), or through the package's operators where
`own` is true.  `exact` computes the same outputs in 64 bits from the
definitions.

Definitions
  route      key = logit, or sigmoid(logit) + bias; the K largest keys, ties to
             the lowest expert; -inf is never chosen (index -1, weight 0).
             weights = scale * softmax or sigmoid of the chosen logits, divided by
             their own sum where `renorm` (sigmoid: sum + 1e-20).
  sort       pairs (token, k) in ascending order inside each expert, every
             expert's segment padded to whole blocks of `block` rows.
  quantise   per 32 elements of a row: e the smallest integer with
             6 * 2^e >= max(amax, 1e-10), codes = e2m1(x / 2^e), nearest, ties to
             the even code; scale byte e + 127.
  linear     y = q(x) . w^T over 4-bit operands, of all rows, or of each expert's
             rows with that expert's matrix.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 128          # rows of a block where the 4-bit product reads the sorted rows


def listed():
    return [
        # one decoded token's router: sigmoid scores, a balancing bias, renormalised
        {"name": "route 1 token", "op": "route", "T": 1, "E": 256, "K": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "renorm": True, "scale": 2.5, "masked": 0.0, "train": False},
        # a training step's router at the largest routed configuration
        {"name": "route train 8192x384", "op": "route", "T": 8192, "E": 384, "K": 6, "dtype": "f32",
         "score": "softmax", "bias": False, "renorm": True, "scale": 1.0, "masked": 0.0, "train": True},
        # a long batch, an odd number of tokens, bf16 logits, a fifth of the experts masked, weights over all experts
        {"name": "route train 65521x160", "op": "route", "T": 65521, "E": 160, "K": 4, "dtype": "bf16",
         "score": "softmax", "bias": False, "renorm": False, "scale": 1.0, "masked": 0.2, "train": True},
        # a decode batch sorted by expert (skewed routing)
        {"name": "permute decode", "op": "permute", "T": 128, "H": 4096, "E": 256, "K": 8, "block": 16,
         "dtype": "bf16", "zipf": True, "masked": 0.0, "train": False},
        # a training step's tokens to the experts, and the gradient back
        {"name": "permute train 8192x7168", "op": "permute", "T": 8192, "H": 7168, "E": 384, "K": 6, "block": 16,
         "dtype": "bf16", "zipf": False, "masked": 0.0, "train": True},
        # experts' rows back to their tokens, weighted, with the gradients of rows and weights
        {"name": "unpermute train 8192x4096", "op": "unpermute", "T": 8192, "H": 4096, "E": 256, "K": 8, "block": 16,
         "dtype": "bf16", "zipf": False, "masked": 0.0, "train": True},
        # odd sizes in 32 bits: rows that start at no 16-byte boundary, a tenth of the slots masked
        {"name": "unpermute train odd f32", "op": "unpermute", "T": 1021, "H": 1001, "E": 37, "K": 3, "block": 32,
         "dtype": "f32", "zipf": True, "masked": 0.1, "train": True},
        # one token's activations into 4 bits
        {"name": "quantise 1x4096", "op": "quantise", "R": 1, "C": 4096, "dtype": "bf16"},
        # a checkpoint's experts into 4 bits
        {"name": "quantise 65536x4096", "op": "quantise", "R": 65536, "C": 4096, "dtype": "bf16"},
        # one token through a dense 4-bit projection
        {"name": "linear 1 token", "op": "linear", "T": 1, "C": 4096, "N": 8192, "E": 1, "K": 0, "dtype": "bf16"},
        # a prefill through a dense 4-bit projection
        {"name": "linear 8192x7168x4096", "op": "linear", "T": 8192, "C": 7168, "N": 4096, "E": 1, "K": 0,
         "dtype": "bf16"},
        # a batch of routed tokens through their experts' 4-bit projection
        {"name": "linear 256 experts", "op": "linear", "T": 2048, "C": 4096, "N": 4096, "E": 256, "K": 6,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "permute", "unpermute", "quantise", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        E = _log(rng, 8, 512)
        T = _log(rng, 1, min(65536, 65536 * 160 // E))
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": T, "E": E, "K": rng.randint(1, min(8, E)), "dtype": dtype, "score": score,
                "bias": score == "sigmoid" and rng.random() < 0.5, "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.0, 0.3, 0.9]),
                "train": rng.random() < 0.5}
    if op in ("permute", "unpermute"):
        H = _log(rng, 64, 7168)
        if rng.random() < 0.5:
            H = (H + 7) // 8 * 8
        E = _log(rng, 2, 384)
        return {"op": op, "T": _log(rng, 1, 8192 if dtype != "f32" else 4096), "H": H, "E": E,
                "K": rng.randint(1, min(6, E)), "block": rng.choice([16, 32, 128]), "dtype": dtype,
                "zipf": rng.random() < 0.5, "masked": rng.choice([0.0, 0.1, 0.9]), "train": rng.random() < 0.7}
    if op == "quantise":
        C = _log(rng, 32, 8192)
        return {"op": op, "R": _log(rng, 1, min(65536, 65536 * 2048 // C)), "C": C, "dtype": dtype}
    C, N = 32 * _log(rng, 2, 224), _log(rng, 64, 8192)
    if rng.random() < 0.5:
        return {"op": op, "T": _log(rng, 1, min(8192, 8192 * 7168 * 4096 // (C * N))), "C": C, "N": N, "E": 1,
                "K": 0, "dtype": dtype}
    E = _log(rng, 4, 256)
    C, N = min(C, 4096), min(N, 4096)
    return {"op": op, "T": _log(rng, 1, 2048), "C": C, "N": N, "E": E, "K": rng.randint(1, min(6, E)),
            "dtype": dtype}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _routing(g, T, E, K, zipf, masked):
    """K distinct experts of each token, uniform or skewed; a share of the slots masked."""
    u = torch.rand(T, E, generator=g, device="cuda", dtype=torch.float32)
    keys = -torch.log(-torch.log(u.clamp(1e-30, 1 - 1e-7)))
    if zipf:
        keys = keys - 1.1 * torch.log1p(torch.randperm(E, generator=g, device="cuda").float())
    idx = torch.topk(keys, K, dim=1).indices.to(torch.int32)
    off = torch.rand(T, K, generator=g, device="cuda") < masked
    return idx.masked_fill(off, -1).contiguous()


def _logits(case, g):
    T, E, K = case["T"], case["E"], case["K"]
    off = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
    bias = 0.1 * _randn(g, E) if case["bias"] else None
    out = _randn(g, T, E).to(DTYPES[case["dtype"]]).masked_fill(off, -math.inf)
    for _ in range(4 if bias is not None else 0):
        # scores and biases add up to real numbers: where two of a row's first K + 1 sums lie so near that
        # their order hangs on the last bit of a sigmoid, the row is drawn again
        key = torch.sigmoid(out.double()).masked_fill(off, -math.inf) + bias.double()
        top = torch.topk(key, min(K + 1, E), dim=1).values
        near = ((top[:, :-1] - top[:, 1:]) < 1e-6).any(dim=1)
        again = _randn(g, T, E).to(out.dtype).masked_fill(off, -math.inf)
        out = torch.where(near[:, None], again, out)
    return out, bias


def _capacity(T, E, K, block):
    return -(-(T * K + min(T * K, E) * (block - 1)) // block) * block


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "route":
        s["logits"], s["bias"] = _logits(case, g)
        s["d_w"] = _randn(g, case["T"], case["K"])
    elif op in ("permute", "unpermute"):
        T, H, E, K = case["T"], case["H"], case["E"], case["K"]
        s["idx"] = _routing(g, T, E, K, case["zipf"], case["masked"])
        rows = _capacity(T, E, K, case["block"])
        s["x"] = _randn(g, T, H).to(DTYPES[case["dtype"]])       # the tokens, or the gradient of the result
        s["rows"] = _randn(g, rows, H).to(DTYPES[case["dtype"]])  # the experts' rows, or their gradient
        s["w"] = torch.rand(T, K, generator=g, device="cuda")
        if op == "unpermute":                                     # the sort of the way there, still in hand
            s["routing"] = _sort(s["idx"], E, case["block"])
    elif op == "quantise":
        R, C = case["R"], case["C"]
        x = torch.randn(R, C, generator=g, device="cuda", dtype=DTYPES[case["dtype"]])
        x *= torch.exp2(torch.randint(-6, 7, (R, 1), generator=g, device="cuda").float()).to(x.dtype)
        s["x"] = x
    else:
        T, C, N, E, K = case["T"], case["C"], case["N"], case["E"], case["K"]
        s["x"] = _randn(g, T, C).to(DTYPES[case["dtype"]])
        s["codes"] = torch.randint(0, 256, (E, N, C // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["sf"] = torch.randint(119, 123, (E, N, C // 32), generator=g, device="cuda", dtype=torch.uint8)
        if K:
            s["idx"] = _routing(g, T, E, K, True, 0.0)
            s["routing"] = _sort(s["idx"], E, BLOCK)
            s["most"] = int(torch.bincount(s["idx"].flatten().long()).max())
    if own:
        from moe_expert_forward_gb300 import ops
        if op == "linear":
            s["weights"] = ops.mx_weights(s["codes"], s["sf"])   # the scales laid out once, as a program keeps them
        if "routing" in s:
            s["sorted"] = ops.sort_tokens(s["idx"], case["E"], case.get("block", BLOCK))
        if op == "linear" and case["K"]:                          # rows of padding are left as they are
            s["out"] = torch.zeros(_capacity(case["T"], case["E"], case["K"], BLOCK), case["N"],
                                   dtype=s["x"].dtype, device="cuda")
    return s


# ------------------------------------------------------------------ the plain form
def _route(logits, K, bias, score, renorm, scale):
    """(indices, weights) and what the gradient needs: scores of every expert, and which are chosen."""
    x = logits.float()
    if score == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True).clamp_min(-3e38))
        p = e / e.sum(1, keepdim=True).clamp_min(1e-38)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = x if bias is None else torch.where(x == -math.inf, x, p + bias)
    top, idx = torch.sort(key, dim=1, descending=True, stable=True)
    top, idx = top[:, :K], idx[:, :K]
    chosen = top != -math.inf
    w = torch.gather(p, 1, idx) * chosen
    total = w.sum(1, keepdim=True) + 1e-20 if renorm else torch.ones_like(w[:, :1])
    return torch.where(chosen, idx, -1).int(), w / total * scale, p, idx, chosen, w, total


def _route_backward(logits, d_w, p, idx, chosen, w, total, score, renorm, scale):
    g = d_w * chosen * scale
    d = (g - (g * (w / total)).sum(1, keepdim=True)) / total if renorm else g   # of the chosen scores
    full = torch.zeros_like(p).scatter(1, idx, d * chosen)
    if score == "softmax":
        d_x = p * (full - (full * p).sum(1, keepdim=True))
    else:
        d_x = full * p * (1 - p)
    return d_x.to(logits.dtype)


def _sort(idx, E, block):
    """counts, first blocks and the row of every pair (-1: masked)."""
    T, K = idx.shape
    e = idx.flatten().long()
    key = torch.where(e < 0, E, e)
    order = torch.sort(key, stable=True).indices
    cnt = torch.zeros(E + 1, dtype=torch.long, device=idx.device).index_add_(0, key, torch.ones_like(key))[:E]
    blk = torch.nn.functional.pad(torch.cumsum((cnt + block - 1) // block, 0), (1, 0))
    first = torch.nn.functional.pad(torch.cumsum(cnt, 0), (1, 0))
    sorted_key = key[order]
    row = blk[sorted_key.clamp_max(E)] * block + torch.arange(T * K, device=idx.device) - first[sorted_key]
    slot = torch.empty_like(key).scatter(0, order, torch.where(sorted_key < E, row, -1))
    return cnt.int(), blk.int(), slot.int().view(T, K)


def _spread(values, slot, rows):
    """values [T, K, H] (or [T, 1, H]) at their rows of a zeroed [rows, H]."""
    T, K = slot.shape
    at = torch.where(slot < 0, rows, slot).flatten().long()
    out = torch.zeros(rows + 1, values.shape[-1], dtype=values.dtype, device=values.device)
    out[at] = values.expand(T, K, -1).reshape(T * K, -1)
    return out[:rows]


def _collect(rows, slot):
    """The rows of every pair in 32 bits [T, K, H]; zeros where masked."""
    got = rows[slot.clamp_min(0).flatten().long()].view(*slot.shape, -1).float()
    return torch.where((slot < 0)[:, :, None], 0.0, got)


def _blocks(x):
    """x [R, C] in 32 bits as [R, C/32, 32], zeros past C."""
    R, C = x.shape
    return torch.nn.functional.pad(x.float(), (0, -C % 32)).view(R, -1, 32)


def _power(e):
    """2^e in 32 bits, exactly, for -127 < e < 128."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """4-bit values times their scales in 32 bits [R, C], and the scale bytes [R, ceil(C / 32)]."""
    b = _blocks(x)
    m, ex = torch.frexp(b.abs().amax(-1).clamp_min(1e-10))
    e = torch.where(m <= 0.75, ex - 3, ex - 2)
    scale = _power(e)[:, :, None]
    v = (b / scale).abs()
    near = ((v > 0.25) * 0.5 + (v >= 0.75) * 0.5 + (v > 1.25) * 0.5 + (v >= 1.75) * 0.5 + (v > 2.5) * 1.0
            + (v >= 3.5) * 1.0 + (v > 5.0) * 2.0)
    q = torch.copysign(near, b) * scale
    return q.view(x.shape[0], -1)[:, :x.shape[1]], (e + 127).to(torch.uint8)


def _weights(codes, sf):
    """The matrices that packed codes and scale bytes stand for, in 32 bits."""
    E, N, half = codes.shape
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    nib = torch.stack((codes & 15, codes >> 4), dim=-1)
    vals = lut[nib.int()].view(E, N, -1, 32)
    return (vals * _power(sf.int() - 127)[..., None]).view(E, N, 2 * half)


def _linear(s):
    c = s["case"]
    q, _ = _quantise(s["x"])
    w = _weights(s["codes"], s["sf"])
    if not c["K"]:
        return (q @ w[0].t()).to(s["x"].dtype)
    # every expert's rows side by side, padded to the largest expert's
    _, blk, slot = s["routing"]
    rows = _capacity(c["T"], c["E"], c["K"], BLOCK)
    e = s["idx"].long()
    at = e * s["most"] + (slot.long() - blk[e].long() * BLOCK)    # expert, then rank inside it
    wide = torch.zeros(c["E"] * s["most"], c["C"], device="cuda")
    wide[at.flatten()] = q[:, None, :].expand(-1, c["K"], -1).reshape(-1, c["C"])
    y = torch.bmm(wide.view(c["E"], s["most"], -1), w.transpose(1, 2)).view(-1, c["N"])
    return _spread(y[at.flatten()].view(c["T"], c["K"], -1).to(s["x"].dtype), slot, rows)


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    op = c["op"]
    if op == "route":
        idx, w, *kept = _route(s["logits"], c["K"], s["bias"], c["score"], c["renorm"], c["scale"])
        out = {"idx": idx, "w": w}
        if c["train"]:
            out["d_logits"] = _route_backward(s["logits"], s["d_w"], *kept, c["score"], c["renorm"], c["scale"])
        return out
    if op == "permute":
        cnt, blk, slot = _sort(s["idx"], c["E"], c["block"])
        out = {"cnt": cnt, "blk": blk, "slot": slot, "rows": _spread(s["x"][:, None, :], slot, s["rows"].shape[0])}
        if c["train"]:
            out["d_x"] = _collect(s["rows"], slot).sum(1).to(s["x"].dtype)
        return out
    if op == "unpermute":
        slot = s["routing"][2]
        got = _collect(s["rows"], slot)
        out = {"y": (got * s["w"][:, :, None]).sum(1).to(s["x"].dtype)}
        if c["train"]:
            d = s["x"].float()[:, None, :]
            out["d_rows"] = _spread((s["w"][:, :, None] * d).to(s["x"].dtype), slot, s["rows"].shape[0])
            out["d_w"] = (got * d).sum(2)
        return out
    if op == "quantise":
        q, sf = _quantise(s["x"])
        return {"values": q.to(torch.bfloat16), "sf": sf}
    return _linear(s)


# ------------------------------------------------------------------ the package's operators
def _run_own(s, c):
    from moe_expert_forward_gb300 import ops
    op = c["op"]
    if op == "route":
        how = {"score": c["score"], "renorm": c["renorm"], "scale": c["scale"]}
        idx, w = ops.route(s["logits"], c["K"], bias=s["bias"], **how)
        out = {"idx": idx, "w": w}
        if c["train"]:
            out["d_logits"] = ops.route_backward(s["logits"], idx, s["d_w"], **how)
        return out
    if op == "permute":
        r = ops.sort_tokens(s["idx"], c["E"], c["block"])
        out = {"cnt": r.cnt, "blk": r.blk_off, "slot": r.slot, "rows": ops.permute(s["x"], r)}
        if c["train"]:
            out["d_x"] = ops.permute_backward(s["rows"], r)
        return out
    if op == "unpermute":
        out = {"y": ops.unpermute(s["rows"], s["sorted"], s["w"])}
        if c["train"]:
            out["d_rows"], out["d_w"] = ops.unpermute_backward(s["x"], s["rows"], s["sorted"], s["w"])
        return out
    if op == "quantise":
        codes, sf = ops.mx_quantize(s["x"])
        return {"values": ops.mx_dequantize(codes, sf, s["x"].shape[1]), "sf": sf}
    if c["K"]:
        return ops.mx_linear(s["x"], s["weights"], routing=s["sorted"], out=s["out"])
    return ops.mx_linear(s["x"], s["weights"])


# ------------------------------------------------------------------ 64 bits, from the definitions
def _exact_route(s, c):
    x = s["logits"].double().cpu().numpy()
    T, E, K = c["T"], c["E"], c["K"]
    with np.errstate(over="ignore", invalid="ignore"):
        key = x if s["bias"] is None else np.where(np.isneginf(x), x, 1 / (1 + np.exp(-x)) + s["bias"].double().cpu().numpy())
        idx = np.argsort(-key, axis=1, kind="stable")[:, :K]
        at = np.arange(T)[:, None]
        live = ~np.isneginf(key[at, idx])
        if c["score"] == "softmax":
            top = x.max(1, keepdims=True)
            p = np.exp(x - np.where(np.isneginf(top), 0, top))
            z = p.sum(1, keepdims=True)
            p = p / np.where(z > 0, z, 1)
        else:
            p = 1 / (1 + np.exp(-x))
    pk = np.where(live, p[at, idx], 0)
    z = pk.sum(1, keepdims=True) + 1e-20 if c["renorm"] else np.ones((T, 1))
    w = c["scale"] * pk / z
    out = {"idx": None, "w": torch.from_numpy(w)}
    if c["train"]:
        g = s["d_w"].double().cpu().numpy() * live
        d = np.zeros_like(x)
        # d p_k: w = scale p / z with z the sum of the chosen p, or one
        dp = c["scale"] * ((g - (g * (pk / z)).sum(1, keepdims=True)) / z if c["renorm"] else g) * live
        if c["score"] == "softmax":
            d = -p * (dp * pk).sum(1, keepdims=True)
            d[at, idx] += pk * dp
        else:
            d[at, idx] = dp * pk * (1 - pk)
        out["d_logits"] = torch.from_numpy(d)
    return out


def _two_to(e):
    """2^e in 64 bits from its bits: a power function may be off in the last one."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_linear(s, c):
    x = s["x"].double()
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
    val = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    q = _exact_quantise(x, mid, val)[0]

    def matrix(e):
        two = torch.empty(c["N"], c["C"], dtype=torch.float64, device="cuda")
        for half in (0, 1):
            nib = (s["codes"][e] >> (4 * half)) % 16
            two[:, half::2] = val[(nib % 8).long()] * (1.0 - 2.0 * (nib // 8).double())
        return two * _two_to(s["sf"][e].long() - 127).repeat_interleave(32, dim=1)

    if not c["K"]:
        return q @ matrix(0).t()
    out = torch.zeros(_capacity(c["T"], c["E"], c["K"], BLOCK), c["N"], dtype=torch.float64, device="cuda")
    row = 0
    for e in range(c["E"]):
        t = (s["idx"] == e).any(1).nonzero()[:, 0]
        if len(t):
            out[row:row + len(t)] = q[t] @ matrix(e).t()
        row += -(-len(t) // BLOCK) * BLOCK
    return out


def _exact_quantise(x, mid, val):
    R, C = x.shape
    n = -(-C // 32)
    b = torch.zeros(R, n * 32, dtype=torch.float64, device="cuda")
    b[:, :C] = x
    b = b.view(R, n, 32)
    most = b.abs().amax(2).clamp_min(1e-10)
    e = torch.ceil(torch.log2(most / 6))
    e = torch.where(6 * _two_to(e) < most, e + 1, e)
    e = torch.where(3 * _two_to(e) >= most, e - 1, e)
    v = b / _two_to(e)[:, :, None]
    a = v.abs()
    k = torch.searchsorted(mid, a.contiguous(), right=False)      # midpoints below |v|
    tie = (k < 7) & (mid[k.clamp_max(6)] == a) & (k % 2 == 1)     # on a midpoint: the even code
    q = val[k + tie.long()] * torch.sign(v) * _two_to(e)[:, :, None]
    return q.view(R, -1)[:, :C], e + 127


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "route":
        return _exact_route(s, c)
    if op in ("permute", "unpermute"):
        T, K = c["T"], c["K"]
        idx = s["idx"].cpu().numpy()
        slot, row = np.full((T, K), -1, np.int64), 0
        for e in range(c["E"]):
            t, k = np.nonzero(idx == e)
            slot[t, k] = row + np.arange(len(t))
            row += -(-len(t) // c["block"]) * c["block"]
        rows = s["rows"].shape[0]
        total = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
        there = torch.zeros(rows, c["H"], dtype=torch.float64, device="cuda")
        d_w = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for k in range(K):
            t = torch.from_numpy(np.nonzero(slot[:, k] >= 0)[0]).cuda()
            r = torch.from_numpy(slot[slot[:, k] >= 0, k]).cuda()
            w = s["w"][t, k, None].double() if op == "unpermute" else 1.0
            got = s["rows"][r].double()
            total[t] += w * got
            there[r] = w * x[t]
            d_w[t, k] = (got * x[t]).sum(1)
        if op == "permute":
            return {"cnt": None, "blk": None, "slot": None, "rows": there, **({"d_x": total} if c["train"] else {})}
        return {"y": total, **({"d_rows": there, "d_w": d_w} if c["train"] else {})}
    if op == "quantise":
        mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
        val = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        out = torch.empty(c["R"], c["C"], dtype=torch.float64, device="cuda")
        for r in range(0, c["R"], 8192):
            out[r:r + 8192] = _exact_quantise(s["x"][r:r + 8192].double(), mid, val)[0]
        return {"values": out, "sf": None}
    return _exact_linear(s, c)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, op = case, case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}[c["dtype"]]
    if op == "route":
        T, E, K = c["T"], c["E"], c["K"]
        n = T * E * size + T * K * 8 + (E * 4 if c["bias"] else 0)
        if c["train"]:
            n += T * K * 4 + T * E * size
        return {"bytes": n, "flops": T * E * (4 if c["train"] else 2)}
    if op in ("permute", "unpermute"):
        T, H, K = c["T"], c["H"], c["K"]
        pairs = T * K * (1 - c["masked"])
        one, all_rows = T * H * size, pairs * H * size
        if op == "permute":
            n = one + all_rows + 8 * T * K
            return {"bytes": n + (one + all_rows if c["train"] else 0), "flops": pairs * H if c["train"] else T * K}
        n = one + all_rows + 8 * T * K
        return {"bytes": n + (one + all_rows + 4 * T * K if c["train"] else 0),
                "flops": pairs * H * (5 if c["train"] else 2)}
    if op == "quantise":
        # the input, the codes and scales written, and read for the values they stand for, written in 16 bits
        return {"bytes": c["R"] * c["C"] * (size + 2 + 2 * 17 / 32), "flops": 2 * c["R"] * c["C"]}
    rows = c["T"] * max(c["K"], 1)
    touched = min(c["E"], rows)
    return {"bytes": c["T"] * c["C"] * size + touched * c["N"] * c["C"] * 17 / 32 + rows * c["N"] * size,
            "flops": 2 * rows * c["N"] * c["C"]}

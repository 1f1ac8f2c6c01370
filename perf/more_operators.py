"""Cases that measure the operators on rows held in 8 bits: the quantiser, the norm in
front of the expert layer, the activation between its two products, and the weight
gradient from rows kept in 8 bits.

Each case is one call, or one training step's calls, of a user's program.  `run`
computes it in plain torch (32-bit arithmetic, rounded once), or through the package's
operators where `own` is true.  `exact` computes the same outputs in 64 bits from the
definitions.

Definitions
  8 bits     "mx": per 32 elements of a row, e the smallest integer with
             448 * 2^e >= max(amax, 1e-10), codes e4m3(x / 2^e), scale byte e + 127.
             "f8": per 128 elements, scale s = max(amax, 1e-10) / 448 in fp32, codes
             e4m3(x / s).  e4m3 rounds to nearest, ties to the even code.
  norm       h = x + residual, rounded to their type; rstd = 1 / sqrt(mean(h^2) + 1e-6);
             y = h * rstd * weight, in the rows' type and in 8 bits.
             Gradients: with n = h * rstd and g = d_y * weight,
             d_x = d_h + rstd * (g - n * mean(g * n)), d_weight = sum over rows of d_y * n.
  swiglu     a = gate * sigmoid(gate) * up * w over rows [gate | up]; with a routing w is
             the weight of the row's (token, k) pair and padding is zero.  A training
             step keeps gate and up in 8 bits ("mx", each half in blocks of its own) and
             takes the gradients of gate, up and w at the kept values.
  weights    d_w[e] = sum over expert e's rows of d_y[r]^T x[r], x in 8 bits ("mx"): one
             row per row of d_y, or per token.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
FLOOR = 1e-10        # the least amax a scale is made for
E4M3_MAX = 448.0
BLOCK = 16           # rows of a routed block in front of the weight gradient


def listed():
    return [
        # one decoded token in front of the layer: rows for the router, 8 bits for the experts
        {"name": "norm 1 token", "op": "norm", "T": 1, "H": 4096, "dtype": "bf16", "weight": "bf16", "residual": True,
         "quant": "mx", "train": False},
        # a prefill in front of the layer's FP8 form
        {"name": "norm 8192x7168 f8", "op": "norm", "T": 8192, "H": 7168, "dtype": "bf16", "weight": "bf16",
         "residual": True, "quant": "f8", "train": False},
        # a training step through the norm: the residual stream's gradient comes in, the weight's goes out
        {"name": "norm train 8192x4096", "op": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "weight": "f32",
         "residual": True, "quant": "", "train": True},
        # odd sizes in 32 bits, no residual: rows that start at no 16-byte boundary
        {"name": "norm train odd f32", "op": "norm", "T": 1021, "H": 1001, "dtype": "f32", "weight": "f32",
         "residual": False, "quant": "mx", "train": True},
        # one decoded token's eight experts, between their products
        {"name": "swiglu 8 pairs", "op": "swiglu", "R": 1, "I": 2048, "E": 256, "K": 8, "block": 16, "dtype": "bf16",
         "masked": 0.0, "quant": True, "train": False},
        # a training step between the experts' products, gate and up kept in 8 bits
        {"name": "swiglu train 2048x6", "op": "swiglu", "R": 2048, "I": 2048, "E": 256, "K": 6, "block": 16,
         "dtype": "bf16", "masked": 0.0, "quant": False, "train": True},
        # a dense layer's step of an odd width in fp16
        {"name": "swiglu train odd f16", "op": "swiglu", "R": 4093, "I": 2731, "E": 0, "K": 0, "block": 0,
         "dtype": "f16", "masked": 0.0, "quant": False, "train": True},
        # a small odd batch in 32 bits into 8 bits and back
        {"name": "keep 33x1001 f32", "op": "keep", "R": 33, "C": 1001, "dtype": "f32", "quant": "mx"},
        # a long batch's activations, kept and read back
        {"name": "keep 65536x4096", "op": "keep", "R": 65536, "C": 4096, "dtype": "bf16", "quant": "mx"},
        # the router's weight gradient: few output tiles, a long sum
        {"name": "weights router", "op": "weights", "T": 8192, "N": 256, "C": 4096, "E": 1, "K": 0, "tokens": False,
         "out": "f32"},
        # a dense projection's weight gradient
        {"name": "weights 8192x4096x4096", "op": "weights", "T": 8192, "N": 4096, "C": 4096, "E": 1, "K": 0,
         "tokens": False, "out": "bf16"},
        # the experts' first projection, its input kept once per token
        {"name": "weights 64 experts", "op": "weights", "T": 4096, "N": 4096, "C": 4096, "E": 64, "K": 6,
         "tokens": True, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "swiglu", "swiglu", "keep", "weights", "weights"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        H = _log(rng, 32, 16384)
        if rng.random() < 0.5:
            H = (H + 127) // 128 * 128
        return {"op": op, "T": _log(rng, 1, min(16384, 8192 * 4096 // H)), "H": H, "dtype": dtype,
                "weight": rng.choice([dtype, "f32"]), "residual": rng.random() < 0.7,
                "quant": rng.choice(["", "mx", "f8"]), "train": rng.random() < 0.5}
    if op == "swiglu":
        I = _log(rng, 32, 8192)
        if rng.random() < 0.5:
            I = (I + 31) // 32 * 32
        routed = rng.random() < 0.6
        K = rng.randint(1, 6) if routed else 0
        rows = 8192 * 2048 // I
        return {"op": op, "R": _log(rng, 1, max(1, min(16384, rows // max(K, 1)))), "I": I,
                "E": rng.randint(6, 256) if routed else 0, "K": K, "block": rng.choice([16, 32, 128]) if routed else 0,
                "dtype": dtype, "masked": rng.choice([0.0, 0.1, 0.9]) if routed else 0.0, "quant": rng.random() < 0.5,
                "train": rng.random() < 0.6}
    if op == "keep":
        C = _log(rng, 32, 8192)
        return {"op": op, "R": _log(rng, 1, min(65536, 65536 * 2048 // C)), "C": C, "dtype": dtype,
                "quant": rng.choice(["mx", "mx", "f8"])}
    N, C = _log(rng, 16, 4096), _log(rng, 32, 4096)
    if rng.random() < 0.6:
        N, C = (N + 7) // 8 * 8, (C + 31) // 32 * 32
    out = rng.choice(["bf16", "f32"])
    if rng.random() < 0.5:
        return {"op": op, "T": _log(rng, 1, 8192), "N": N, "C": C, "E": 1, "K": 0, "tokens": False, "out": out}
    E = _log(rng, 4, 48)
    return {"op": op, "T": _log(rng, 1, 4096), "N": N, "C": C, "E": E, "K": rng.randint(1, min(6, E)),
            "tokens": rng.random() < 0.5, "out": out}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def _routing(g, T, E, K, masked):
    """K distinct experts of each token, skewed; a share of the slots masked."""
    u = torch.rand(T, E, generator=g, device="cuda", dtype=torch.float32)
    keys = -torch.log(-torch.log(u.clamp(1e-30, 1 - 1e-7)))
    keys = keys - 0.5 * torch.log1p(torch.randperm(E, generator=g, device="cuda").float())
    idx = torch.topk(keys, K, dim=1).indices.to(torch.int32)
    off = torch.rand(T, K, generator=g, device="cuda") < masked
    return idx.masked_fill(off, -1).contiguous()


def _capacity(T, E, K, block):
    return -(-(T * K + min(T * K, E) * (block - 1)) // block) * block


def prepare(case, seed):
    g, c = _gen(seed), case
    op, s = c["op"], {"case": case}
    if op == "norm":
        T, H, dt = c["T"], c["H"], DTYPES[c["dtype"]]
        s["x"] = _randn(g, T, H, dtype=dt)
        s["residual"] = 2 * _randn(g, T, H, dtype=dt) if c["residual"] else None
        s["weight"] = (1 + 0.2 * _randn(g, H)).to(DTYPES[c["weight"]])
        if c["train"]:
            s["d_y"], s["d_h"] = _randn(g, T, H, dtype=dt), _randn(g, T, H, dtype=dt)
    elif op == "swiglu":
        T, I, K, dt = c["R"], c["I"], c["K"], DTYPES[c["dtype"]]
        rows = T
        if K:
            s["idx"] = _routing(g, T, c["E"], K, c["masked"])
            s["w"] = torch.rand(T, K, generator=g, device="cuda")
            s["slot"] = _sort(s["idx"], c["E"], c["block"])
            rows = _capacity(T, c["E"], K, c["block"])
        s["h"] = 1.5 * _randn(g, rows, 2 * I, dtype=dt)
        if c["train"]:
            s["d_a"] = _randn(g, rows, I, dtype=dt)
    elif op == "keep":
        x = _randn(g, c["R"], c["C"], dtype=DTYPES[c["dtype"]])
        x *= torch.exp2(torch.randint(-6, 7, (c["R"], 1), generator=g, device="cuda").float()).to(x.dtype)
        s["x"] = x
    else:
        T, N, C, E, K = c["T"], c["N"], c["C"], c["E"], c["K"]
        rows = T
        if K:
            s["idx"] = _routing(g, T, E, K, 0.0)
            s["slot"] = _sort(s["idx"], E, BLOCK)
            s["most"] = int(torch.bincount(s["idx"].flatten().long()).max())
            rows = _capacity(T, E, K, BLOCK)
        s["d_y"] = _randn(g, rows, N, dtype=torch.bfloat16)
        s["codes"], s["sf"] = _pack(_randn(g, T if c["tokens"] else rows, C))   # kept by the forward pass
    if own and "idx" in s:
        from moe_expert_forward_gb300 import ops
        s["routing"] = ops.sort_tokens(s["idx"], c["E"], c.get("block", BLOCK))   # of the forward pass, in hand
    return s


# ------------------------------------------------------------------ the plain form
def _sort(idx, E, block):
    """The row of every pair: ascending inside each expert, whole blocks per expert; -1 where masked."""
    T, K = idx.shape
    e = idx.flatten().long()
    key = torch.where(e < 0, E, e)
    order = torch.sort(key, stable=True).indices
    cnt = torch.zeros(E + 1, dtype=torch.long, device=idx.device).index_add_(0, key, torch.ones_like(key))[:E]
    blk = torch.nn.functional.pad(torch.cumsum((cnt + block - 1) // block, 0), (1, 0))
    first = torch.nn.functional.pad(torch.cumsum(cnt, 0), (1, 0))
    sorted_key = key[order]
    row = blk[sorted_key] * block + torch.arange(T * K, device=idx.device) - first[sorted_key]
    slot = torch.empty_like(key).scatter(0, order, torch.where(sorted_key < E, row, -1))
    return slot.view(T, K)


def _power(e):
    """2^e in 32 bits, exactly, for -127 < e < 128."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _blocks(x, size):
    """x [R, C] in 32 bits as [R, C / size, size], zeros past C."""
    R, C = x.shape
    return torch.nn.functional.pad(x.float(), (0, -C % size)).view(R, -1, size)


def _mx(x):
    """e4m3 values [R, blocks, 32] and exponents [R, blocks]."""
    b = _blocks(x, 32)
    m, ex = torch.frexp(b.abs().amax(-1).clamp_min(FLOOR))
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    return (b * _power(-e)[:, :, None]).to(torch.float8_e4m3fn), e


def _pack(x):
    v, e = _mx(x)
    return v.reshape(x.shape[0], -1).view(torch.uint8), (e + 127).to(torch.uint8)


def _values(x, quant):
    """What the 8 bits of x stand for, in 32 bits."""
    R, C = x.shape
    if quant == "mx":
        v, e = _mx(x)
        return (v.float() * _power(e)[:, :, None]).view(R, -1)[:, :C]
    b = _blocks(x, 128)
    # by a tensor: torch multiplies by the reciprocal of a number
    s = b.abs().amax(-1, keepdim=True).clamp_min(FLOOR) / torch.full((), E4M3_MAX, device=x.device)
    return ((b / s).to(torch.float8_e4m3fn).float() * s).view(R, -1)[:, :C]


def _norm(s, c):
    x, weight = s["x"], s["weight"].float()
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1) + EPS)
    n = f * rstd[:, None]
    y = n * weight
    out = {"y": y.to(x.dtype), "rstd": rstd}
    if c["residual"]:
        out["h"] = h
    if c["quant"]:
        out["values"] = _values(y, c["quant"]).to(torch.bfloat16)
    if c["train"]:
        d_y = s["d_y"].float()
        g = d_y * weight
        d = rstd[:, None] * (g - n * (g * n).mean(1, keepdim=True))
        out["d_x"] = (d + s["d_h"].float()).to(x.dtype)
        out["d_weight"] = (d_y * n).sum(0)
    return out


def _row_weights(s, rows):
    """Each pool row's weight [rows, 1] and whether it holds a pair."""
    pair = torch.full((rows + 1,), -1, dtype=torch.long, device="cuda")
    slot = s["slot"].flatten()
    pair[torch.where(slot < 0, rows, slot)] = torch.arange(slot.numel(), device="cuda")
    pair = pair[:rows, None]
    return s["w"].flatten()[pair.clamp_min(0)], pair >= 0


def _swiglu(s, c):
    h, I = s["h"], c["I"]
    w, live = 1.0, True
    if c["K"]:
        w, live = _row_weights(s, h.shape[0])
        h = torch.where(live, h, 0)
    gate, up = h[:, :I].float(), h[:, I:].float()
    a = gate / (1 + torch.exp(-gate)) * up * w
    out = {"a": a.to(h.dtype)}
    if c["quant"]:
        out["values"] = _values(a, "mx").to(torch.bfloat16)
    if c["train"]:
        gate, up = _values(gate, "mx"), _values(up, "mx")
        d = s["d_a"].float()
        if c["K"]:
            d = torch.where(live, d, 0)
        sig = 1 / (1 + torch.exp(-gate))
        d_gate = d * w * up * sig * (1 + gate * (1 - sig))
        out["d_h"] = torch.cat((d_gate, d * w * gate * sig), 1).to(h.dtype)
        if c["K"]:
            dot = torch.nn.functional.pad((d * gate * sig * up).sum(1), (0, 1))
            out["d_w"] = dot[s["slot"]]              # a masked pair's -1 is the zero behind the last row
    return out


def _weights(s, c):
    x = s["codes"].view(torch.float8_e4m3fn).float().view(s["sf"].shape + (32,)) * _power(s["sf"].int() - 127)[..., None]
    x, d = x.view(x.shape[0], -1)[:, :c["C"]], s["d_y"].float()
    dt = DTYPES[c["out"]]
    if not c["K"]:
        return (d.t() @ x).to(dt)
    # every expert's rows side by side, padded to the largest expert's
    e, slot = s["idx"].long(), s["slot"]
    first = torch.full((c["E"],), slot.numel() + c["E"] * BLOCK, dtype=torch.long, device="cuda")
    first = first.scatter_reduce(0, e.flatten(), slot.flatten(), "amin")
    at = (e * s["most"] + slot - first[e]).flatten()
    pairs = slot.flatten()
    wide_d = torch.zeros(c["E"] * s["most"], c["N"], device="cuda")
    wide_x = torch.zeros(c["E"] * s["most"], c["C"], device="cuda")
    wide_d[at] = d[pairs]
    wide_x[at] = x[torch.arange(pairs.numel(), device="cuda") // c["K"]] if c["tokens"] else x[pairs]
    y = torch.bmm(wide_d.view(c["E"], s["most"], -1).transpose(1, 2), wide_x.view(c["E"], s["most"], -1))
    return y.to(dt)


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm":
        return _norm(s, c)
    if c["op"] == "swiglu":
        return _swiglu(s, c)
    if c["op"] == "keep":
        return {"values": _values(s["x"], c["quant"]).to(torch.bfloat16)}
    return {"d_w": _weights(s, c)}


# ------------------------------------------------------------------ the package's operators
def _run_own(s, c):
    from moe_expert_forward_gb300 import ops
    if c["op"] == "norm":
        n = ops.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quant=c["quant"] or None)
        out = {"y": n.y, "rstd": n.rstd}
        if c["residual"]:
            out["h"] = n.h
        if c["quant"]:
            out["values"] = ops.dequantize8(n.codes, n.sf, c["H"])
        if c["train"]:
            out["d_x"], out["d_weight"] = ops.rms_norm_backward(s["d_y"], n.h, s["weight"], n.rstd, d_h=s["d_h"])
        return out
    if c["op"] == "swiglu":
        how = {"routing": s["routing"], "topk_w": s["w"]} if c["K"] else {}
        f = ops.swiglu(s["h"], quant=c["quant"], keep=c["train"], **how)
        out = {"a": f.a}
        if c["quant"]:
            out["values"] = ops.dequantize8(f.codes, f.sf, c["I"])
        if c["train"]:
            out["d_h"], d_w = ops.swiglu_backward(s["d_a"], f.kept, f.kept_sf, **how)
            if c["K"]:
                out["d_w"] = d_w
        return out
    if c["op"] == "keep":
        codes, sf = ops.quantize8(s["x"], c["quant"])
        return {"values": ops.dequantize8(codes, sf, c["C"])}
    return {"d_w": ops.weight_grad(s["d_y"], s["codes"], s["sf"], c["C"], routing=s.get("routing"),
                                   by_token=c["tokens"], dtype=DTYPES[c["out"]])}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _two_to(e):
    """2^e in 64 bits from its bits: a power function may be off in the last one."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _near_e4m3(v):
    """v (at most 448 in magnitude) to the nearest e4m3 value, ties to even, in 64 bits."""
    _, ex = torch.frexp(v.abs().clamp_min(2.0 ** -20))
    step = _two_to((ex.long() - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _exact_values(x, quant):
    """The values that x [R, C], in 64 bits, is held as."""
    R, C = x.shape
    size = 32 if quant == "mx" else 128
    b = torch.zeros(R, -(-C // size) * size, dtype=torch.float64, device=x.device)
    b[:, :C] = x
    b = b.view(R, -1, size)
    most = b.abs().amax(2, keepdim=True).clamp_min(FLOOR)
    if quant == "mx":
        e = torch.ceil(torch.log2(most / E4M3_MAX))
        e = torch.where(E4M3_MAX * _two_to(e) < most, e + 1, e)
        e = torch.where(E4M3_MAX / 2 * _two_to(e) >= most, e - 1, e)
        scale = _two_to(e)
    else:
        scale = most / E4M3_MAX
    return (_near_e4m3(b / scale) * scale).view(R, -1)[:, :C]


def _exact_norm(s, c):
    dt = s["x"].dtype
    total = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    h = total.to(dt).double()
    weight = s["weight"].double()
    rstd = (h.square().sum(1) / c["H"] + EPS).rsqrt()
    y = weight * (h * rstd.unsqueeze(1))
    out = {"y": y, "rstd": rstd}
    if c["residual"]:
        out["h"] = total
    if c["quant"]:
        out["values"] = _exact_values(y, c["quant"])
    if c["train"]:
        # through y_i = w_i h_i r with r = (mean(h^2) + eps)^(-1/2): dr/dh_j = -r^3 h_j / H
        d_y = s["d_y"].double()
        inner = torch.einsum("th,th,h->t", d_y, h, weight)
        out["d_x"] = s["d_h"].double() + rstd[:, None] * d_y * weight - (rstd ** 3 * inner / c["H"])[:, None] * h
        out["d_weight"] = torch.einsum("th,th,t->h", d_y, h, rstd)
    return out


def _exact_slots(idx, E, block):
    """(row of each pair or -1, and each expert's (tokens, first row)) by walking the experts."""
    idx = idx.cpu().numpy()
    slot, row, spans = np.full(idx.shape, -1, np.int64), 0, []
    for e in range(E):
        t, k = np.nonzero(idx == e)
        slot[t, k] = row + np.arange(len(t))
        spans.append((t, row))
        row += -(-len(t) // block) * block
    return slot, spans


def _exact_swiglu(s, c):
    h, I = s["h"].double(), c["I"]
    rows = h.shape[0]
    w = torch.ones(rows, 1, dtype=torch.float64, device="cuda")
    if c["K"]:
        slot, _ = _exact_slots(s["idx"], c["E"], c["block"])
        t, k = np.nonzero(slot >= 0)
        at = torch.from_numpy(slot[t, k]).cuda()
        live = torch.zeros(rows, 1, dtype=torch.bool, device="cuda")
        live[at] = True
        w = torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
        w[at, 0] = s["w"].double()[torch.from_numpy(t).cuda(), torch.from_numpy(k).cuda()]
        h = h * live
    gate, up = h.split(I, dim=1)
    a = w * up * gate * torch.sigmoid(gate)
    out = {"a": a}
    if c["quant"]:
        out["values"] = _exact_values(a, "mx")
    if c["train"]:
        gate, up = _exact_values(gate, "mx"), _exact_values(up, "mx")
        sig, d = torch.sigmoid(gate), s["d_a"].double()
        slope = sig + gate * sig * (1 - sig)
        if c["K"]:
            d = d * live
        out["d_h"] = torch.cat((w * d * up * slope, w * d * gate * sig), dim=1)
        if c["K"]:
            d_w = torch.zeros(slot.shape, dtype=torch.float64, device="cuda")
            dot = torch.einsum("ri,ri,ri->r", d, gate * sig, up)
            d_w[torch.from_numpy(t).cuda(), torch.from_numpy(k).cuda()] = dot[at]
            out["d_w"] = d_w
    return out


def _exact_weights(s, c):
    b = s["codes"].int()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * _two_to(e - 7)) * (1 - 2 * (b >> 7)).double()
    x = (v * _two_to(s["sf"].long() - 127).repeat_interleave(32, dim=1))[:, :c["C"]]
    if not c["K"]:
        return torch.einsum("rn,rc->nc", s["d_y"].double(), x)
    _, spans = _exact_slots(s["idx"], c["E"], BLOCK)
    out = torch.zeros(c["E"], c["N"], c["C"], dtype=torch.float64, device="cuda")
    for e, (t, row) in enumerate(spans):
        if len(t):
            mine = x[torch.from_numpy(t).cuda()] if c["tokens"] else x[row:row + len(t)]
            out[e] = s["d_y"][row:row + len(t)].double().t() @ mine
    return out


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        return _exact_norm(s, c)
    if c["op"] == "swiglu":
        return _exact_swiglu(s, c)
    if c["op"] == "keep":
        out = torch.empty(c["R"], c["C"], dtype=torch.float64, device="cuda")
        for r in range(0, c["R"], 8192):
            out[r:r + 8192] = _exact_values(s["x"][r:r + 8192].double(), c["quant"])
        return {"values": out}
    return {"d_w": _exact_weights(s, c)}


# ------------------------------------------------------------------ what a pass cannot do without
def _held(n, quant):
    """Bytes of n elements in 8 bits."""
    return n * (33 / 32 if quant == "mx" else 33 / 32 if quant else 0)     # one byte per 32, or four per 128


def work(case):
    c, op = case, case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}[c["dtype"]] if "dtype" in c else 2
    if op == "norm":
        n = c["T"] * c["H"]
        # x, the residual and their sum, y; in 8 bits written, and read for the values they stand for
        b = n * size * (4 if c["residual"] else 2) + 4 * c["T"] + 4 * c["H"]
        if c["quant"]:
            b += 2 * _held(n, c["quant"]) + 2 * n
        if c["train"]:
            b += n * size * 4 + 4 * c["H"]       # d_y, h, d_h and d_x
        return {"bytes": b, "flops": n * (16 if c["train"] else 6)}
    if op == "swiglu":
        n = c["R"] * max(c["K"], 1) * (1 - c["masked"]) * c["I"]
        b = 3 * n * size
        if c["quant"]:
            b += 2 * _held(n, "mx") + 2 * n
        if c["train"]:
            b += 2 * _held(2 * n, "mx") + 3 * n * size     # gate and up written and read in 8 bits; d_a, d_h
        return {"bytes": b + 8 * c["R"] * c["K"], "flops": n * (24 if c["train"] else 8)}
    if op == "keep":
        n = c["R"] * c["C"]
        return {"bytes": n * (size + 2) + 2 * _held(n, c["quant"]), "flops": 2 * n}
    rows, size = c["T"] * max(c["K"], 1), 4 if c["out"] == "f32" else 2
    kept = c["T"] if c["tokens"] else rows
    return {"bytes": rows * c["N"] * 2 + _held(kept * c["C"], "mx") + c["E"] * c["N"] * c["C"] * size,
            "flops": 2 * rows * c["N"] * c["C"]}

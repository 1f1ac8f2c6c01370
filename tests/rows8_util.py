"""Plain 64-bit forms of the operators on rows in 8 bits, and the bounds their tests use.

A rounding is off by at most half a step: HALF[type] relative to the value.  A sum of n fp32 terms in any order is off by
at most n * 2^-24 of the sum of magnitudes (to first order, which a factor of 1.01 covers at these sizes)."""
import numpy as np
import torch

import oracle as O

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # finfo.eps / 2
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # the least step, of subnormals
U = 2.0 ** -24
BLOCK = {"mx": 32, "f8": 128}


def d64(t):
    return t.detach().double().cpu().numpy()


def hold(x, quant):
    """x [R, C] (exact values of fp32 or less) -> (codes, scales, values fp64 [R, C]) of quantize8."""
    size, (R, C) = BLOCK[quant], x.shape
    nb = -(-C // size)
    b = np.zeros((R, nb * size), np.float32)
    b[:, :C] = x
    bad = ~np.isfinite(b.reshape(R, nb, size)).all(2)
    clean = np.where(np.repeat(bad, size, axis=1), 0, b)
    codes, sf = O.quantise_x(clean, quant)
    if quant == "mx":
        sf = np.where(bad, 255, sf).astype(np.uint8)
        scale = np.where(bad, np.nan, np.ldexp(1.0, sf.astype(int) - 127))
    else:
        sf = np.where(bad, np.nan, sf).astype(np.float32)
        scale = sf.astype(np.float64)
    return codes, sf, (O.e4m3_decode(codes) * np.repeat(scale, size, axis=1))[:, :C]


def values(codes, sf, C):
    """What codes and scales (torch) stand for, fp64 [R, C]."""
    codes, sf = codes.cpu().numpy(), sf.cpu().numpy()
    if sf.dtype == np.uint8:
        scale, size = np.where(sf == 255, np.nan, np.ldexp(1.0, sf.astype(int) - 127)), 32
    else:
        scale, size = sf.astype(np.float64), 128
    return (O.e4m3_decode(codes) * np.repeat(scale, size, axis=-1))[..., :C]


def check_held(codes, sf, want, off):
    """codes and sf hold values that are within `off` (relative, an array or a number) of want [R, C]: their scales fit
    such values, and no element is further than a rounding of e4m3 from them."""
    R, C = want.shape
    quant = "mx" if sf.dtype == torch.uint8 else "f8"
    size, nb = BLOCK[quant], -(-C // BLOCK[quant])
    assert codes.shape == (R, nb * size) and sf.shape == (R, nb)
    assert not codes.cpu().numpy()[:, C:].any()
    pad = np.zeros((R, nb * size))
    pad[:, :C] = np.abs(want)
    amax = np.maximum(pad.reshape(R, nb, size).max(2), 1e-10)
    off = float(np.max(off)) if np.size(off) else 0.0
    if quant == "mx":
        scale = np.ldexp(1.0, sf.cpu().numpy().astype(int) - 127)
        assert (448 * scale >= amax * (1 - off)).all() and (224 * scale < amax * (1 + off)).all()
    else:
        scale = sf.double().cpu().numpy()
        assert (np.abs(scale * 448 - amax) <= (off + 2 * U) * amax * 1.01).all()
    got = values(codes, sf, C)
    step = np.repeat(scale, size, axis=1)[:, :C] * 2.0 ** -10      # half of e4m3's least step
    assert (np.abs(got - want) <= (2.0 ** -4 + off + 2 * U) * 1.01 * np.abs(want) + step).all()


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-g))


def sigmoid_off(g, dt):
    """How far (relative) the kernels' sigmoid may be: fp32 rows use expf (2 ulp) and a division, 16-bit rows __expf
    (2 + 1.173 |g| ulp) and a reciprocal of 1 ulp; an ulp is 2 U, and the additions and products around it 4 U."""
    return (4 * U + 4 * U) * np.ones_like(g) if dt == "f32" else 2 * U * (2 + 1.173 * np.abs(g) + 1 + 2)


def randn(seed, *shape, dt="f32"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(DT[dt])


def routing(T, E, K, masked, seed):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, K), np.int32)
    idx[rng.random(idx.shape) < masked] = -1
    return torch.from_numpy(idx)

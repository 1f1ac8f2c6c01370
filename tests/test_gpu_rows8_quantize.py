"""quantize8 and dequantize8 against the oracle's block rules, bit for bit."""
import numpy as np
import pytest
import torch

import oracle as O
from rows8_util import DT, HALF, d64, hold, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def check(ops, x, quant):
    codes, sf = ops.quantize8(x, quant)
    want_codes, want_sf, want = hold(d64(x), quant)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    assert np.array_equal(sf.cpu().numpy(), want_sf, equal_nan=True)
    C = x.shape[1]
    back = d64(ops.dequantize8(codes, sf, C, torch.float32))
    # one fp32 product; that of mx is exact below 2^128, to which the largest fp32 rounds up (2^8 times 2^120)
    with np.errstate(over="ignore"):
        assert np.array_equal(back, want.astype(np.float32), equal_nan=True)
    if quant == "mx":
        assert np.array_equal(back[np.abs(want) < 2.0 ** 128], want[np.abs(want) < 2.0 ** 128])
    for dt in ("bf16", "f16"):
        got = ops.dequantize8(codes, sf, C, DT[dt])
        assert torch.equal(got.cpu().nan_to_num(7.0), torch.from_numpy(back).float().to(DT[dt]).nan_to_num(7.0))


@pytest.mark.parametrize("quant", ["mx", "f8"])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 31), (3, 32), (2, 33), (7, 127), (5, 128), (4, 129), (33, 1001),
                                 (300, 4096), (17, 7168), (129, 48), (1000, 16)])
def test_shapes(ops, R, C, dt, quant):
    x = randn(R + C, R, C, dt=dt).cuda()
    x *= torch.exp2(torch.arange(R, device="cuda") % 13 - 6).to(x.dtype)[:, None]
    check(ops, x, quant)


def test_ties_borders_and_extremes(ops):
    """Rows scaled to e = 0 (one element 448) hold every e4m3 value, every midpoint and their fp32 neighbours; amax just
    below, at and above 448 * 2^e; the floor; the largest and the least fp32."""
    pos = O.E4M3[:127]
    mid = (pos[1:] + pos[:-1]) / 2
    v = np.concatenate([pos, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = v[:len(v) // 31 * 31].reshape(-1, 31)
    x = np.concatenate([np.full((len(v), 1), 448, np.float32), v], 1)
    check(ops, torch.from_numpy(x).cuda(), "mx")
    for quant, size in (("mx", 32), ("f8", 128)):
        edge = np.zeros((12, size), np.float32)
        for i, e in enumerate((-40, 0, 100)):
            top = np.float32(448 * 2.0 ** e)
            edge[3 * i:3 * i + 3, 5] = np.nextafter(top, np.float32(0)), top, np.nextafter(top, np.float32(np.inf))
            edge[3 * i:3 * i + 3, 6:] = top / 3
        edge[9, :] = 1e-11
        edge[10, 0], edge[10, 1] = np.finfo(np.float32).max, 2.0 ** -149
        edge[11, 0] = -2.0 ** -140
        check(ops, torch.from_numpy(edge).cuda(), quant)
        check(ops, torch.zeros(3, size, device="cuda"), quant)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("quant", ["mx", "f8"])
def test_blocks_that_are_not_finite_stand_for_nan(ops, dt, quant):
    x = randn(5, 6, 300, dt=dt).cuda()
    x[0, 5], x[1, 40], x[2, 299], x[4, 256] = float("nan"), float("inf"), float("-inf"), float("nan")
    check(ops, x, quant)
    codes, sf = ops.quantize8(x, quant)
    back = ops.dequantize8(codes, sf, 300)
    size = 32 if quant == "mx" else 128
    for r, c in ((0, 5), (1, 40), (2, 299), (4, 256)):
        lo = c // size * size
        assert torch.isnan(back[r, lo:lo + size]).all() and torch.isfinite(back[r, :lo]).all()
    assert torch.isfinite(back[[3, 5]]).all()


def test_f8_of_many_values_divides_as_ieee_does(ops):
    """Quotients next to e4m3 borders under scales of every kind."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(4000, 1024, generator=g, device="cuda") * torch.exp2(torch.randn(4000, 1, generator=g, device="cuda") * 10)
    codes, sf = ops.quantize8(x, "f8")
    b = x.view(4000, 8, 128)
    s = b.abs().amax(2, keepdim=True).clamp_min(1e-10) / torch.full((), 448.0, device="cuda")
    assert torch.equal(sf, s[:, :, 0])
    assert torch.equal(codes, (b / s).to(torch.float8_e4m3fn).view(torch.uint8).view(4000, 1024))
    border = torch.from_numpy((O.E4M3[1:127] + O.E4M3[:126]) / 2).float().cuda()
    for k in range(8):
        amax = float(torch.rand(1, generator=g, device="cuda") + 0.5)
        s = torch.full((), amax, device="cuda") / torch.full((), 448.0, device="cuda")
        near = torch.stack([torch.nextafter(border * s, torch.full_like(border, d)) for d in (0.0, 1e9)] + [border * s])
        x = torch.nn.functional.pad(near, (2, 0), value=amax)
        codes, sf = ops.quantize8(x, "f8")
        assert torch.equal(codes, (x / s).to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(0, 64), (1, 65), (3, 100), (16, 200), (8, 24)])
def test_strided_and_unaligned_rows(ops, lo, hi, dt):
    wide = randn(2, 50, 200, dt=dt).cuda()
    for quant in ("mx", "f8"):
        a, b = ops.quantize8(wide[:, lo:hi], quant), ops.quantize8(wide[:, lo:hi].contiguous(), quant)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = wide.t().contiguous().t()[:1, :1]                # a single element: any stride
    assert ops.quantize8(one)[0].shape == (1, 32)


def test_the_layer_takes_it(ops):
    """x and x_sf of both variants, bf16 rows, as the oracle quantises them."""
    x = randn(9, 40, 512, dt="bf16")
    for quant in ("mx", "f8"):
        codes, sf = ops.quantize8(x.cuda(), quant)
        want_codes, want_sf = O.quantise_x(x.float().numpy(), quant)
        assert np.array_equal(codes.cpu().numpy(), want_codes) and np.array_equal(sf.cpu().numpy(), want_sf)


def test_empty_and_large(ops):
    for quant in ("mx", "f8"):
        codes, sf = ops.quantize8(torch.empty(0, 70, device="cuda"), quant)
        assert codes.shape[0] == 0 and sf.shape[0] == 0 and ops.dequantize8(codes, sf, 70).shape == (0, 70)


def test_offsets_past_32_bits(ops):
    R, C = 1_060_000, 4096
    x = torch.empty(R, C, device="cuda", dtype=torch.bfloat16)
    for r in range(0, R, 100_000):
        x[r:r + 100_000].normal_()
    codes, sf = ops.quantize8(x)
    assert codes.numel() > 2 ** 32
    back = ops.dequantize8(codes, sf, C)
    for at in (0, 524_288, 1_048_570, R - 7):
        c, s = ops.quantize8(x[at:at + 7].contiguous())
        assert torch.equal(codes[at:at + 7], c) and torch.equal(sf[at:at + 7], s)
        assert torch.equal(back[at:at + 7], ops.dequantize8(c, s, C))


def test_rounding_of_f8_values(ops):
    """fp32 product of code and scale, then the type's own rounding: within HALF and the product's."""
    x = randn(1, 20, 256, dt="f32").cuda()
    codes, sf = ops.quantize8(x, "f8")
    _, _, want = hold(d64(x), "f8")
    for dt in DT:
        got = d64(ops.dequantize8(codes, sf, 256, DT[dt]))
        assert (np.abs(got - want) <= (HALF[dt] + 2.0 ** -24) * 1.01 * np.abs(want) + 2.0 ** -25).all()


@pytest.mark.parametrize("quant", ["mx", "f8"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1040, 1025])
def test_many_rows_as_few(ops, quant, dt, C):
    """More than 2^22 groups of 16 columns, where a thread takes several: the bits of the same rows in a small call."""
    R = 65539
    x = randn(1, R, C, dt=dt).cuda()
    codes, sf = ops.quantize8(x, quant)
    back = ops.dequantize8(codes, sf, C, x.dtype)
    for at in (0, 1234, 32766, R - 5):
        part = slice(at, at + 5)
        c, s = ops.quantize8(x[part], quant)
        assert torch.equal(codes[part], c) and torch.equal(sf[part], s)
        assert torch.equal(back[part], ops.dequantize8(c, s, C, x.dtype))
    # and each row once: the rows between the parts, by a call of a tenth of them at a time
    for at in range(0, R, 6554):
        part = slice(at, at + 6554)
        assert torch.equal(codes[part], ops.quantize8(x[part], quant)[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_the_largest_elements_round_to_infinity(ops, dt):
    """248 * 2^120 is half way between the codes of 240 and 256, and the latter is even: 2^128, past both types."""
    top = torch.finfo(DT[dt])
    border = torch.tensor(248.0 * 2.0 ** 120, dtype=DT[dt])
    below = torch.nextafter(border, torch.zeros((), dtype=DT[dt]))
    x = torch.zeros(1, 64, dtype=DT[dt])
    x[0, 0], x[0, 1], x[0, 32], x[0, 33] = border, top.min, below, -below
    codes, sf = ops.quantize8(x.cuda())
    inf, edge = float("inf"), 240.0 * 2.0 ** 120
    want = torch.zeros(1, 64)
    want[0, [0, 1, 32, 33]] = torch.tensor([inf, -inf, edge, -edge])
    assert torch.equal(ops.dequantize8(codes, sf, 64, torch.float32).cpu(), want)
    assert torch.equal(ops.dequantize8(codes, sf, 64).cpu(), want.bfloat16())
    for N in (1, 1025):
        got = ops.weight_grad(torch.ones(1, N, device="cuda", dtype=torch.bfloat16), codes, sf, 64, dtype=torch.float32)
        assert torch.equal(got.cpu(), want.repeat(N, 1))

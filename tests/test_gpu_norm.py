"""rms_norm and its gradients against the formulas in 64 bits (tolerances: rows8_util)."""
import numpy as np
import pytest
import torch

from rows8_util import DT, HALF, TINY, U, check_held, d64, randn

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    ops.sync_status()              # what other tests let run out
    return ops


def sum_off(H):
    """Roundings in a row's sum: a thread adds at most 16 (H / 512 + 1) terms in turn, then up to 40 parts and a
    division."""
    return (H / 32 + 16 + 44) * U


def forward(ops, x, res, w, quant, rows=True, eps=EPS):
    n = ops.rms_norm(x.cuda(), w.cuda(), None if res is None else res.cuda(), eps=eps, rows=rows, quant=quant)
    dt = {v: k for k, v in DT.items()}[x.dtype]
    H = x.shape[1]
    total = d64(x) if res is None else d64(x) + d64(res)
    h = d64(n.h)
    # the fp32 sum, then the type's rounding
    assert (np.abs(h - total) <= (HALF[dt] + (0 if dt == "f32" else U)) * 1.01 * np.abs(total) + TINY[dt]).all()
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    off = (sum_off(H) / 2 + 3 * U) * 1.01                  # half of the sum's, root, division, the addition of eps
    assert n.rstd.dtype == torch.float32 and (np.abs(d64(n.rstd) - r) <= off * r).all()
    y = h * r[:, None] * d64(w)
    off += 2 * U * 1.01
    if rows:
        assert n.y.dtype == x.dtype
        assert (np.abs(d64(n.y) - y) <= (off + HALF[dt]) * 1.01 * np.abs(y) + TINY[dt]).all()
    else:
        assert n.y is None
    if quant:
        check_held(n.codes, n.sf, y, off)
    else:
        assert n.codes is None and n.sf is None
    return n


def backward(ops, d_y, h, w, rstd, d_h):
    dx, dw = ops.rms_norm_backward(d_y.cuda(), h.cuda(), w.cuda(), rstd.cuda(), None if d_h is None else d_h.cuda())
    dt = {v: k for k, v in DT.items()}[d_y.dtype]
    T, H = h.shape
    y, hh, ww, r = d64(d_y), d64(h), d64(w), d64(rstd)[:, None]
    n, g = hh * r, y * ww
    extra = 0 if d_h is None else d64(d_h)
    mean = (g * n).mean(1, keepdims=True) if H else 0
    want = extra + r * (g - n * mean)
    size = np.abs(r * g) + np.abs(extra) + np.abs(r * n) * np.abs(g * n).mean(1, keepdims=True)
    # the products and differences: 8 roundings of parts no larger than `size`; the mean's sum
    tol = 8 * U * size + np.abs(r * n) * np.abs(g * n).mean(1, keepdims=True) * (sum_off(H) + 3 * U)
    assert dx.dtype == d_y.dtype and (np.abs(d64(dx) - want) <= tol * 1.01 + HALF[dt] * 1.01 * np.abs(want) + TINY[dt]).all()
    assert dw.dtype == torch.float32
    assert (np.abs(d64(dw) - (y * n).sum(0)) <= (T + 50) * U * np.abs(y * n).sum(0) + 1e-30).all()
    return dx, dw


WIDTHS = [1, 2, 15, 16, 17, 31, 32, 33, 100, 127, 128, 512, 513, 1000, 1001, 4096, 5000, 7168, 8192, 8208, 16384]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H", WIDTHS + [16400, 32768, 32769, 40000])
def test_forward_widths(ops, H, dt):
    T = 5 if H > 8192 else 11
    for i, quant in enumerate((None, "mx", "f8")):
        x, res = randn(H + i, T, H, dt=dt), randn(H + 9, T, H, dt=dt) if i != 1 else None
        forward(ops, x, res, (1 + 0.3 * randn(H + 1, H)).to(DT[dt if i else "f32"]), quant, rows=i != 2)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H", WIDTHS + [16400, 20000])
def test_backward_widths(ops, H, dt):
    T = 5 if H > 8192 else 13
    h = randn(H, T, H, dt=dt)
    r = (1 / torch.sqrt(h.double().square().mean(1) + EPS)).float()
    w = (1 + 0.3 * randn(H + 1, H)).to(DT["f32" if H % 2 else dt])
    backward(ops, randn(H + 2, T, H, dt=dt), h, w, r, None if H % 3 == 0 else randn(H + 3, T, H, dt=dt))


@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 303, 304, 305, 2500, 5001])
@pytest.mark.parametrize("H", [40, 96, 384])
def test_tokens(ops, T, H):
    x, res = randn(T, T, H, dt="bf16"), randn(T + 1, T, H, dt="bf16")
    w = 1 + 0.3 * randn(3, H)
    n = forward(ops, x, res, w, "mx")
    backward(ops, randn(T + 2, T, H, dt="bf16"), n.h.cpu(), w, n.rstd.cpu(), randn(T + 3, T, H, dt="bf16"))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H", [512, 1024, 2032, 2048, 2064, 3584, 4096, 4112, 7168, 8192, 8208, 16384])
@pytest.mark.parametrize("T", [305, 700])
def test_many_long_rows(ops, T, H, dt):
    """Rows that come by copies into a ring, with and without a residual, weights of both types."""
    for i in range(2):
        x, res = randn(H + i, T, H, dt=dt), randn(H + 9, T, H, dt=dt) if i else None
        w = (1 + 0.3 * randn(H + 1, H)).to(DT[dt if i else "f32"])
        n = forward(ops, x, res, w, ("mx", "f8")[i])
        backward(ops, randn(H + 2, T, H, dt=dt), n.h.cpu(), w, n.rstd.cpu(), randn(H + 3, T, H, dt=dt) if i else None)
    assert ops.sync_status() == (0, 0)


def test_no_rows_give_a_zero_weight_gradient(ops):
    e = torch.empty(0, 64, device="cuda")
    dx, dw = ops.rms_norm_backward(e, e, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and dw.shape == (64,) and not dw.any()


def test_zero_large_and_small_rows(ops):
    """Rows of zeros (eps alone), of 1e-12 (below eps), of 1e15, and eps = 0."""
    x = torch.cat([torch.zeros(1, 96), randn(1, 1, 96) * 1e-12, randn(2, 1, 96) * 1e15, randn(3, 1, 96)])
    forward(ops, x, None, 1 + 0.1 * randn(4, 96), "mx")
    forward(ops, x[1:], None, 1 + 0.1 * randn(4, 96), "f8", eps=0.0)


def test_a_row_that_is_not_finite_stays_alone(ops):
    x = randn(1, 20, 200, dt="bf16").cuda()
    w = torch.ones(200, device="cuda")
    clean = ops.rms_norm(x, w, quant="mx")
    bad = x.clone()
    bad[3, 7], bad[11, 199] = float("nan"), float("inf")
    n = ops.rms_norm(bad, w, quant="mx")
    keep = [i for i in range(20) if i not in (3, 11)]
    assert torch.equal(n.y[keep], clean.y[keep]) and torch.equal(n.codes[keep], clean.codes[keep])
    assert torch.equal(n.sf[keep], clean.sf[keep])
    assert torch.isnan(n.y[3]).all() and (n.sf[3] == 255).all() and (n.sf[11, 6] == 255)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(0, 64), (1, 65), (3, 100), (16, 208), (8, 24)])
def test_strided_and_unaligned_inputs(ops, lo, hi, dt):
    """The same bits wherever the rows lie: the lanes' shares do not depend on alignment."""
    wide, wide2 = randn(2, 50, 300, dt=dt).cuda(), randn(3, 50, 300, dt=dt).cuda()
    w = torch.rand(300, device="cuda")[lo:hi]
    a = ops.rms_norm(wide[:, lo:hi], w, wide2[:, lo:hi], quant="mx")
    b = ops.rms_norm(wide[:, lo:hi].contiguous(), w.clone(), wide2[:, lo:hi].contiguous(), quant="mx")
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    c = ops.rms_norm_backward(wide2[:, lo:hi], wide[:, lo:hi], w, a.rstd, wide2[:, lo:hi])
    d = ops.rms_norm_backward(wide2[:, lo:hi].contiguous(), wide[:, lo:hi].contiguous(), w.clone(), a.rstd,
                              wide2[:, lo:hi].contiguous())
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])


def test_gradients_against_differences(ops):
    """<d_x, v> + <d_w, u> against the central difference of <d_y, y> along (v, u), in 64 bits."""
    T, H, step = 6, 40, 1e-5
    x, v, dy = (randn(i, T, H) for i in range(3))
    w, u = 1 + 0.2 * randn(4, H), randn(5, H)

    def loss(a, b):
        return float((dy.double() * a / (a.square().mean(1, keepdim=True) + EPS).sqrt() * b).sum())
    a, b = x.double(), w.double()
    slope = (loss(a + step * v.double(), b + step * u.double()) - loss(a - step * v.double(), b - step * u.double())) / (2 * step)
    n = ops.rms_norm(x.cuda(), w.cuda(), eps=EPS)
    dx, dw = ops.rms_norm_backward(dy.cuda(), n.h, w.cuda(), n.rstd)
    along = float((d64(dx) * d64(v)).sum() + (d64(dw) * d64(u)).sum())
    # fp32 gradients (1e-6 of their size) against a difference whose error is step^2 = 1e-10 and 1e-16 / step = 1e-11
    assert abs(along - slope) <= 1e-5 * max(1.0, abs(slope))


def test_repeats_are_bit_equal(ops):
    x, dy = randn(1, 3000, 520, dt="bf16").cuda(), randn(2, 3000, 520, dt="bf16").cuda()
    w = torch.rand(520, device="cuda")
    n = ops.rms_norm(x, w)
    first = ops.rms_norm_backward(dy, n.h, w, n.rstd)
    for _ in range(3):
        again = ops.rms_norm_backward(dy, n.h, w, n.rstd)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("H", [520, 2048, 2064, 3584, 4096, 4112, 6000, 8192, 8208, 12000, 16384])
def test_a_row_does_not_depend_on_the_batch(ops, dt, H):
    """Bits of one row among few rows, among many, and in rows on other boundaries."""
    x, r, dy = randn(1, 700, H, dt=dt).cuda(), randn(2, 700, H, dt=dt).cuda(), randn(3, 700, H, dt=dt).cuda()
    w = randn(4, H, dt=dt).cuda()
    n = ops.rms_norm(x, w, r, quant="mx")
    dx, _ = ops.rms_norm_backward(dy, n.h, w, n.rstd, r)
    some = slice(41, 44)
    m = ops.rms_norm(x[some], w, r[some], quant="mx")
    wide = [torch.empty(3, H + 5, dtype=t.dtype, device="cuda")[:, 3:H + 3].copy_(t[some]) for t in (x, r, dy)]
    v = ops.rms_norm(wide[0], w, wide[1], quant="mx")
    for k in (m, v):
        assert all(torch.equal(a[some], b) for a, b in zip(n, k))
    assert torch.equal(ops.rms_norm_backward(dy[some], m.h, w, m.rstd, r[some])[0], dx[some])
    assert torch.equal(ops.rms_norm_backward(wide[2], m.h, w, m.rstd, wide[1])[0], dx[some])


def test_offsets_past_32_bits(ops):
    T, H = 600_000, 4096
    x = torch.empty(T, H, device="cuda", dtype=torch.bfloat16)
    for r in range(0, T, 100_000):
        x[r:r + 100_000].normal_()
    w = torch.rand(H, device="cuda")
    n = ops.rms_norm(x, w, x, quant="mx")
    dx, _ = ops.rms_norm_backward(x, n.h, w, n.rstd, x)
    for at in (0, 2 ** 31 // H - 3, 2 ** 32 // (2 * H) - 3, T - 7):
        part = slice(at, at + 7)
        m = ops.rms_norm(x[part].clone(), w, x[part].clone(), quant="mx")
        assert torch.equal(n.y[part], m.y) and torch.equal(n.codes[part], m.codes) and torch.equal(n.sf[part], m.sf)
        assert torch.equal(dx[part], ops.rms_norm_backward(x[part].clone(), m.h, w, m.rstd, x[part].clone())[0])


def test_the_layer_takes_what_the_norm_writes(ops):
    """The fused layer on the norm's 8 bits, and on the codes of the same rows by quantize8 of the fp32 norm."""
    import moe_expert_forward_gb300 as M
    import workload as W
    cfg = W.CONFIGS["tiny"]
    inp = {k: v.cuda() for k, v in W.make_inputs(cfg, "cpu").items()}
    x = randn(3, cfg.T, cfg.H, dt="bf16").cuda()
    n = ops.rms_norm(x, torch.ones(cfg.H, device="cuda"), x, quant="mx")
    opt = M.options()
    p1, p2 = M.prepare_weights(inp["w1_sf"], inp["w2_sf"], cfg.H, cfg.I, cfg.E, opt)
    ws = M.alloc_workspace(cfg.T, cfg.H, cfg.I, cfg.E, cfg.K, opt)
    outs = []
    for codes, sf in ((n.codes, n.sf), ops.quantize8(ops.dequantize8(n.codes, n.sf, cfg.H, torch.float32))):
        out = torch.empty(cfg.T, cfg.H, dtype=torch.bfloat16, device="cuda")
        M.forward(codes, sf, inp["topk_idx"], inp["topk_w"], inp["w1"], p1, inp["w2"], p2, out, cfg.H, cfg.I, cfg.E, ws, opt)
        assert M.sync_status(ws) == (0, 0)
        outs.append(out)
    # quantising what 8 bits stand for gives the same values: at most the scale's byte moves with the codes
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])

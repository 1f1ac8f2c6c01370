"""swiglu and its gradients from kept rows against the formulas in 64 bits (tolerances: rows8_util)."""
import numpy as np
import pytest
import torch

from rows8_util import DT, HALF, TINY, U, check_held, d64, hold, randn, routing, sigmoid, sigmoid_off, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def pairs_of(r):
    """pool row -> (t, k), and the live rows."""
    slot = r.slot.cpu().numpy()
    t, k = np.nonzero(slot >= 0)
    return slot[t, k], t, k


def forward(ops, h, r=None, w=None, **how):
    """h on the host; what swiglu returns, checked."""
    dt = {v: k for k, v in DT.items()}[h.dtype]
    R, I = h.shape[0], h.shape[1] // 2
    f = ops.swiglu(h.cuda(), r, None if w is None else w.cuda(), **how)
    x = d64(h)
    scale = np.ones((R, 1))
    if r is not None:
        at, t, k = pairs_of(r)
        live = np.zeros((R, 1), bool)
        live[at] = True
        x = np.where(live, x, 0)
        scale = np.zeros((R, 1))
        scale[at, 0] = 1 if w is None else d64(w)[t, k]
    gate, up = x[:, :I], x[:, I:]
    want = gate * sigmoid(gate) * up * scale
    off = (sigmoid_off(gate, dt) + 3 * U) * 1.01           # and three products
    if how.get("rows", True):
        assert f.a.dtype == h.dtype
        assert (np.abs(d64(f.a) - want) <= (off + HALF[dt]) * np.abs(want) + TINY[dt]).all()
        if r is not None:
            assert not d64(f.a)[~live[:, 0]].any()
    else:
        assert f.a is None
    if how.get("quant"):
        check_held(f.codes, f.sf, want, off)
    else:
        assert f.codes is None and f.sf is None
    if how.get("keep"):
        nb = -(-I // 32)
        assert f.kept.shape == (R, 2, 32 * nb) and f.kept_sf.shape == (R, 2, nb)
        for half, part in enumerate((gate, up)):
            codes, sf, _ = hold(part, "mx")
            assert np.array_equal(f.kept[:, half].cpu().numpy(), codes)
            assert np.array_equal(f.kept_sf[:, half].cpu().numpy(), sf)
    else:
        assert f.kept is None and f.kept_sf is None
    return f


def backward(ops, d_a, f, r=None, w=None):
    dt = {v: k for k, v in DT.items()}[d_a.dtype]
    R, I = d_a.shape
    d_h, d_w = ops.swiglu_backward(d_a.cuda(), f.kept, f.kept_sf, r, None if w is None else w.cuda())
    gate, up = (values(f.kept[:, i].contiguous(), f.kept_sf[:, i].contiguous(), I) for i in (0, 1))
    d = d64(d_a)
    scale = np.ones((R, 1))
    if r is not None:
        at, t, k = pairs_of(r)
        live = np.zeros((R, 1), bool)
        live[at] = True
        d = np.where(live, d, 0)
        scale = np.zeros((R, 1))
        scale[at, 0] = 1 if w is None else d64(w)[t, k]
    s, k_off = sigmoid(gate), sigmoid_off(gate, dt)
    g = np.abs(gate)
    slope = s * (1 + gate * (1 - s))
    want = np.concatenate([d * scale * up * slope, d * scale * gate * s], 1)
    # s enters the slope twice: k_off (1 + |g|) of s, and (1 - s, the product, the sum: 3 U of up to 1 + |g|); 1 - s is
    # as far off as s, at most k_off + U
    tol = np.concatenate([np.abs(d * scale * up * s) * ((1 + g) * (2 * k_off + 8 * U)),
                          np.abs(want[:, I:]) * (k_off + 4 * U)], 1)
    assert d_h.dtype == d_a.dtype
    assert (np.abs(d64(d_h) - want) <= tol * 1.01 + HALF[dt] * 1.01 * np.abs(want) + TINY[dt]).all()
    if w is None:
        assert d_w is None
    else:
        terms = d * gate * s * up
        off = (np.abs(terms) * (k_off + 4 * U)).sum(1) + (I / 32 + 64) * U * np.abs(terms).sum(1)
        got = d64(d_w)
        want_w = terms.sum(1)
        assert (np.abs(got[t, k] - want_w[at]) <= off[at] * 1.01 + 1e-30).all()
        dead = np.ones(got.shape, bool)
        dead[t, k] = False
        assert not got[dead].any()
    return d_h, d_w


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("I", [1, 2, 15, 16, 17, 31, 32, 33, 48, 100, 511, 512, 513, 1001, 2048, 4096, 5000, 8192])
def test_dense_widths(ops, I, dt):
    R = 9
    h = 1.5 * randn(I, R, 2 * I, dt=dt)
    f = forward(ops, h.to(DT[dt]), quant=True, keep=True)
    backward(ops, randn(I + 1, R, I, dt=dt), f)
    forward(ops, h.to(DT[dt]), rows=False, quant=True)
    forward(ops, h.to(DT[dt]))


@pytest.mark.parametrize("R", [0, 1, 2, 7, 8, 9, 300])
def test_dense_rows(ops, R):
    h = randn(R, R, 2 * 72, dt="bf16")
    backward(ops, randn(R + 1, R, 72, dt="bf16"), forward(ops, h, quant=True, keep=True))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,K,block,masked", [(1, 256, 8, 16, 0.0), (1, 3, 1, 16, 1.0), (40, 6, 2, 16, 0.1), (7, 5, 5, 128, 0.9),
                                                (130, 9, 3, 32, 0.0), (33, 4, 2, 256, 1.0), (0, 4, 2, 16, 0.0)])
@pytest.mark.parametrize("I", [64, 33])
def test_routed(ops, T, E, K, block, masked, I, dt):
    """Padding, before and past the last block, holds NaN and is neither read nor left as it was."""
    r = ops.sort_tokens(routing(T, E, K, masked, T).cuda(), E, block)
    h = torch.full((r.rows, 2 * I), float("nan")).to(DT[dt])
    d_a = torch.full((r.rows, I), float("nan")).to(DT[dt])
    at, t, k = pairs_of(r)
    h[at], d_a[at] = randn(1, len(at), 2 * I, dt=dt), randn(2, len(at), I, dt=dt)
    w = torch.rand(T, K, generator=torch.Generator().manual_seed(4))
    w[torch.from_numpy(r.slot.cpu().numpy() < 0)] = float("nan")
    for weights in (w, None):
        f = forward(ops, h, r, weights, quant=True, keep=True)
        backward(ops, d_a, f, r, weights)


def test_large_gates_and_zeros(ops):
    """Gates far into both tails, and exact zeros: nothing overflows on the way."""
    gate = torch.tensor([0.0, -0.0, 1e-20, 30.0, -30.0, 87.0, -87.0, -88.8, -100.0, 1e4, -1e4, 3e4, -3e4, 1.0, -1.2784645, 5.0])
    for dt in DT:
        h = torch.cat([gate, torch.linspace(-2, 2, 16)]).to(DT[dt])[None].repeat(3, 1)
        f = ops.swiglu(h.cuda(), keep=True)
        g, u = d64(h[:, :16]), d64(h[:, 16:])
        assert torch.isfinite(f.a).all()
        want = g * sigmoid(g) * u
        # beyond |g| = 88 exp(-g) passes the largest fp32 and the product is -0 instead of at most 88 e^-88 = 2^-120
        assert (np.abs(d64(f.a) - want) <= (sigmoid_off(np.minimum(np.abs(g), 100), dt) + HALF[dt] + 3 * U) * 1.01 * np.abs(want)
                + 2.0 ** -118 + TINY[dt]).all()
        d_h, _ = ops.swiglu_backward(torch.ones(3, 16, device="cuda", dtype=DT[dt]), f.kept, f.kept_sf)
        assert torch.isfinite(d_h).all()


def test_not_finite_rows_stay_alone(ops):
    r = ops.sort_tokens(routing(30, 4, 2, 0.0, 1).cuda(), 4)
    h = randn(2, r.rows, 128, dt="bf16").cuda()
    w = torch.rand(30, 2, device="cuda")
    clean = ops.swiglu(h, r, w, quant=True, keep=True)
    row = int(r.slot[11, 1])
    bad = h.clone()
    bad[row, 5] = float("nan")
    f = ops.swiglu(bad, r, w, quant=True, keep=True)
    keep = torch.arange(r.rows, device="cuda") != row
    assert all(torch.equal(p[keep], q[keep]) for p, q in zip(f, clean))
    assert torch.isnan(f.a[row, 5]) and f.sf[row, 0] == 255 and f.kept_sf[row, 0, 0] == 255
    d_h, d_w = ops.swiglu_backward(torch.ones(r.rows, 64, device="cuda"), f.kept, f.kept_sf, r, w)
    assert torch.isnan(d_w[11, 1]) and torch.isnan(d_w).sum() == 1 and torch.isfinite(d_h[keep]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi", [(0, 64), (1, 65), (3, 101), (16, 208), (8, 24)])
def test_strided_and_unaligned_inputs(ops, lo, hi, dt):
    wide = randn(2, 50, 400, dt=dt).cuda()
    a = ops.swiglu(wide[:, lo:hi], quant=True, keep=True)
    b = ops.swiglu(wide[:, lo:hi].contiguous(), quant=True, keep=True)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    d = wide[:, hi:hi + (hi - lo) // 2]
    assert torch.equal(ops.swiglu_backward(d, a.kept, a.kept_sf)[0], ops.swiglu_backward(d.contiguous(), a.kept, a.kept_sf)[0])


def test_gradients_against_differences(ops):
    """<d_h, v> + <d_w, u> against the central difference along (v, u) at the kept values, in 64 bits."""
    T, E, K, I, step = 9, 4, 2, 40, 1e-5
    r = ops.sort_tokens(routing(T, E, K, 0.2, 3).cuda(), E)
    h, v = randn(1, r.rows, 2 * I), randn(2, r.rows, 2 * I)
    w, u = randn(3, T, K), randn(4, T, K)
    d_a = randn(5, r.rows, I)
    f = ops.swiglu(h.cuda(), r, w.cuda(), keep=True)
    at, t, k = pairs_of(r)
    x = np.concatenate([values(f.kept[:, i].contiguous(), f.kept_sf[:, i].contiguous(), I) for i in (0, 1)], 1)

    def loss(a, b):
        gate, up = a[at, :I], a[at, I:]
        return float((d64(d_a)[at] * gate * sigmoid(gate) * up * b[t, k][:, None]).sum())
    slope = (loss(x + step * d64(v), d64(w) + step * d64(u)) - loss(x - step * d64(v), d64(w) - step * d64(u))) / (2 * step)
    d_h, d_w = ops.swiglu_backward(d_a.cuda(), f.kept, f.kept_sf, r, w.cuda())
    along = float((d64(d_h) * d64(v)).sum() + (d64(d_w) * d64(u)).sum())
    # fp32 gradients (1e-6 of their size) against a difference whose error is of the order step^2 = 1e-10
    assert abs(along - slope) <= 1e-5 * max(1.0, abs(slope))


def test_offsets_past_32_bits(ops):
    R, I = 600_000, 2048
    h = torch.empty(R, 2 * I, device="cuda", dtype=torch.bfloat16)
    for r in range(0, R, 100_000):
        h[r:r + 100_000].normal_()
    f = ops.swiglu(h, quant=True, keep=True)
    d_h, _ = ops.swiglu_backward(f.a, f.kept, f.kept_sf)
    for at in (0, 2 ** 31 // (2 * I) - 3, 2 ** 32 // (4 * I) - 3, R - 7):
        part = slice(at, at + 7)
        g = ops.swiglu(h[part].clone(), quant=True, keep=True)
        assert all(torch.equal(p[part], q) for p, q in zip(f, g))
        assert torch.equal(d_h[part], ops.swiglu_backward(g.a, g.kept, g.kept_sf)[0])

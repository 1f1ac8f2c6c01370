"""The router's top-k and its gradient against a plain implementation in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# fp32 weights: exp of a rounded difference (|l - m| <= 32: 32 * 2^-24) and a few roundings of 2^-24
W_TOL = 4e-6
# a gradient adds the rounding of its own type to that, relative to the largest incoming gradient
ROUND = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def plain(x, K, bias, score, renorm, scale):
    """(idx, w, p) in 64 bits; x [T, E] float64 numpy."""
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    idx = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    p = np.zeros((T, E))
    for t in range(T):
        live = x[t] > -np.inf
        if live.any():
            if score == "softmax":
                e = np.where(live, np.exp(x[t] - x[t][live].max()), 0)
                p[t] = e / e.sum()
            else:
                p[t] = np.where(live, 1 / (1 + np.exp(-x[t])), 0)
        key = np.where(live, x[t] if bias is None else p[t] + bias, -np.inf)
        order = sorted(np.nonzero(live)[0], key=lambda e: (-key[e], e))[:K]
        idx[t, :len(order)] = order
        z = p[t, order].sum() + (1e-20 if score == "sigmoid" else 0) if renorm else 1.0
        w[t, :len(order)] = scale * p[t, order] / z
    return idx, w, p


def plain_gradient(x, idx, g, p, score, renorm, scale):
    d = np.zeros_like(p)
    for t in range(len(p)):
        e = idx[t][idx[t] >= 0]
        if not len(e):
            continue
        gt, pt = scale * g[t][idx[t] >= 0], p[t][e]
        z = pt.sum() + (1e-20 if score == "sigmoid" else 0) if renorm else 1.0
        dp = (gt - (gt * pt).sum() / z) / z if renorm else gt
        if score == "softmax":
            d[t] = -p[t] * (dp * pt).sum()
            d[t][e] += pt * dp
        else:
            d[t][e] = dp * pt * (1 - pt)
    return d


def check(ops, x, K, bias=None, score="softmax", renorm=True, scale=1.0, dt="f32", gradient=True):
    dev = x.cuda()
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32)
    idx, w = ops.route(dev, K, bias=None if b is None else b.cuda(), score=score, renorm=renorm, scale=scale)
    x64 = x.double().numpy()
    r_idx, r_w, p = plain(x64, K, None if b is None else b.double().numpy(), score, renorm, scale)
    assert np.array_equal(idx.cpu().numpy(), r_idx)
    got = w.cpu().numpy().astype(np.float64)
    assert np.abs(got - r_w).max(initial=0) <= W_TOL * scale, np.abs(got - r_w).max()
    assert (got[r_idx < 0] == 0).all()
    if gradient:
        g = torch.randn(r_w.shape, generator=torch.Generator().manual_seed(3))
        d = ops.route_backward(dev, idx, g.cuda(), score=score, renorm=renorm, scale=scale)
        assert d.dtype == dev.dtype and d.shape == dev.shape
        ref = plain_gradient(x64, r_idx, g.double().numpy(), p, score, renorm, scale)
        err = np.abs(d.double().cpu().numpy() - ref)
        tol = W_TOL * scale * np.abs(g.numpy()).max(initial=0) * 2 + ROUND[dt] * np.abs(ref) + (1e-7 if dt == "f16" else 0)
        assert (err <= tol).all(), err.max()


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (8, 3), (31, 4), (33, 16), (64, 6), (129, 8), (256, 8), (384, 6),
                                 (513, 2), (1000, 16), (1024, 10)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_sizes(ops, E, K, score, renorm):
    g = torch.Generator().manual_seed(E * 17 + K)
    check(ops, 2 * torch.randn(37, E, generator=g), K, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("T", [0, 1, 3, 4, 5, 1000])
def test_rows(ops, T):
    check(ops, torch.randn(T, 40, generator=torch.Generator().manual_seed(T)), 4)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("sigmoid", True)])
def test_sixteen_bit_logits_with_ties(ops, dt, score, renorm):
    # two decimals of N(0, 1) over 256 experts: nearly every row holds equal logits
    x = (torch.randn(200, 256, generator=torch.Generator().manual_seed(5)) * 8).round().div(8).to(DT[dt])
    check(ops, x, 8, score=score, renorm=renorm, dt=dt)


@pytest.mark.parametrize("E,K,dt", [(8, 2, "f32"), (62, 8, "bf16"), (160, 4, "bf16"), (160, 4, "f16"), (256, 8, "f32"),
                                    (250, 1, "bf16"), (161, 4, "bf16"), (64, 9, "f32")])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_many_rows(ops, E, K, dt, score, renorm):
    """Four of many rows share a warp (up to 256 experts, an even number, and 8 choices): the same as those rows in
    small batches, which take a warp each."""
    g = torch.Generator().manual_seed(E + K)
    x = (torch.randn(16387, E, generator=g) * 2).to(DT[dt])
    x[torch.rand(x.shape, generator=g) < 0.3] = -float("inf")
    x[5], x[6, 1:] = -float("inf"), float("nan")
    x, dw = x.cuda(), torch.randn(16387, K, generator=g).cuda()
    bias = torch.randn(E, generator=g).cuda() if score == "sigmoid" and E != 160 else None
    idx, w = ops.route(x, K, bias=bias, score=score, renorm=renorm)
    d = ops.route_backward(x, idx, dw, score=score, renorm=renorm)
    parts = [slice(0, 6000), slice(6000, 12000), slice(12000, 16387)]
    i2, w2 = zip(*[ops.route(x[p], K, bias=bias, score=score, renorm=renorm) for p in parts])
    assert torch.equal(idx, torch.cat(i2))
    assert (w - torch.cat(w2)).abs().max() <= W_TOL
    d2 = torch.cat([ops.route_backward(x[p], idx[p], dw[p], score=score, renorm=renorm) for p in parts]).float()
    assert ((d.float() - d2).abs() <= 2 * W_TOL * dw.abs().max() + 2 * ROUND[dt] * d2.abs() + (1e-7 if dt == "f16" else 0)).all()


def test_bias_moves_the_choice_only(ops):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(300, 64, generator=g)
    bias = torch.randn(64, generator=g)
    key = np.sort(1 / (1 + np.exp(-x.double().numpy())) + bias.double().numpy(), axis=1)[:, ::-1]
    x = x[torch.from_numpy((np.diff(-key[:, :9], axis=1) > 1e-6).all(axis=1))]   # rows whose order fp32 resolves
    assert len(x) > 250
    check(ops, x, 8, bias=bias, score="sigmoid", scale=1.5)
    check(ops, x, 8, bias=bias, score="sigmoid", renorm=False)


def test_masked_rows(ops):
    g = torch.Generator().manual_seed(11)
    x = torch.randn(8, 70, generator=g)
    inf = float("inf")
    x[0] = -inf                                # nothing left
    x[1] = -inf
    x[1, 69] = 0.5                             # one expert left, fewer than K
    x[2] = torch.finfo(torch.float32).min      # the type's lowest value is a number: all equal, lowest experts first
    x[3, ::2] = float("nan")                   # never chosen
    x[4] = float("nan")
    x[5, :] = 0.0
    x[5, 1::2] = -0.0                          # equal keys
    x[6] = torch.finfo(torch.float32).min
    x[6, 3] = 1.0
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check(ops, x, 6, score=score, renorm=renorm)


def test_scores_that_underflow_together(ops):
    x = torch.full((2, 16), -200.0)            # every sigmoid is zero in fp32
    idx, w = ops.route(x.cuda(), 4, score="sigmoid")
    assert idx.cpu().tolist() == [[0, 1, 2, 3]] * 2 and torch.isfinite(w).all() and (w == 0).all()
    d = ops.route_backward(x.cuda(), idx, torch.ones_like(w), score="sigmoid")
    assert torch.isfinite(d).all() and (d == 0).all()


def test_infinite_logit(ops):
    x = torch.zeros(1, 8)
    x[0, 5] = float("inf")
    idx, w = ops.route(x.cuda(), 2)
    assert idx.cpu().tolist() == [[5, 0]] and torch.isnan(w).any()
    idx, w = ops.route(x.cuda(), 2, score="sigmoid", renorm=False)
    assert w.cpu().tolist() == [[1.0, 0.5]]


def test_strided_rows_and_streams(ops):
    g = torch.Generator().manual_seed(13)
    wide = torch.randn(50, 101, generator=g)
    x = wide[:, 3:70]
    dev = wide.cuda()[:, 3:70]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = ops.route(dev, 5)
    b = ops.route(dev, 5, stream=s)
    s.synchronize()
    idx, w, _ = plain(x.double().numpy(), 5, None, "softmax", True, 1.0)
    for got in (a, b):
        assert np.array_equal(got[0].cpu().numpy(), idx)
        assert np.abs(got[1].cpu().numpy() - w).max() <= W_TOL


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_gradient_against_differences(ops, score, renorm):
    """The directional derivative of the 64-bit forward, by central differences of 1e-5."""
    g = torch.Generator().manual_seed(21)
    x = torch.randn(20, 24, generator=g)
    dw = torch.randn(20, 5, generator=g)
    v = torch.randn(20, 24, generator=g).double().numpy()
    idx, _ = ops.route(x.cuda(), 5, score=score, renorm=renorm)
    d = ops.route_backward(x.cuda(), idx, dw.cuda(), score=score, renorm=renorm).double().cpu().numpy()
    h, x64 = 1e-5, x.double().numpy()
    up = plain(x64 + h * v, 5, None, score, renorm, 1.0)
    down = plain(x64 - h * v, 5, None, score, renorm, 1.0)
    same = (up[0] == down[0]).all(axis=1)      # rows whose choice the step does not change
    assert same.sum() > 15
    by_steps = (dw.double().numpy() * (up[1] - down[1]) / (2 * h)).sum(1)
    # third derivatives of the scores are below 1, so the step's own error is below h^2 |v|^3 ~ 1e-8
    assert np.abs((d * v).sum(1) - by_steps)[same].max() <= 1e-4


def test_same_inputs_same_bits(ops):
    x = torch.randn(3000, 160, generator=torch.Generator().manual_seed(2)).cuda()
    a, b = ops.route(x, 6, renorm=False), ops.route(x, 6, renorm=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals(ops):
    from moe_expert_forward_gb300 import MMError
    x = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for call in (lambda: ops.route(x, 9), lambda: ops.route(x, 0), lambda: ops.route(x.cpu(), 2),
                 lambda: ops.route(x.double(), 2), lambda: ops.route(x.t(), 2), lambda: ops.route(x[0], 1),
                 lambda: ops.route(torch.zeros(2, 1025, device="cuda"), 2), lambda: ops.route(x, 2, score="tanh"),
                 lambda: ops.route(x, 2, bias=torch.zeros(8, device="cuda")),               # softmax has no bias
                 lambda: ops.route(x, 2, bias=torch.zeros(7, device="cuda"), score="sigmoid"),
                 lambda: ops.route(torch.zeros(4, 40, device="cuda"), 17),
                 lambda: ops.route(x[:1].expand(4, 8), 2),
                 lambda: ops.route_backward(x, idx.long(), w), lambda: ops.route_backward(x, idx[:3], w[:3]),
                 lambda: ops.route_backward(x, idx, w[:, :1])):
        with pytest.raises(MMError):
            call()

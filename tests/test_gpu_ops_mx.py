"""4-bit quantisation and product against plain implementations in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import workload as W

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # significands of 24, 8 and 11 bits


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def plain_quantise(x):
    """x [R, C] float64 -> (values, scale bytes) in 64 bits."""
    R, C = x.shape
    n = -(-C // 32)
    b = np.zeros((R, n * 32))
    b[:, :C] = x
    b = b.reshape(R, n, 32)
    bad = ~np.isfinite(b).all(2)
    most = np.maximum(np.where(bad, 0, np.abs(np.nan_to_num(b, posinf=0, neginf=0)).max(2)), 1e-10)
    m, ex = np.frexp(most)
    e = np.where(m <= 0.75, ex - 3, ex - 2)
    v = np.where(bad[:, :, None], 0, b) / np.ldexp(1.0, e)[:, :, None]
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    d = np.abs(np.abs(v)[..., None] - grid)
    near = d.argmin(-1)
    up = np.minimum(near + 1, 7)                       # argmin takes the lower of two equals: an odd one goes up
    near = np.where((np.take_along_axis(d, near[..., None], -1) == np.take_along_axis(d, up[..., None], -1))[..., 0]
                    & (near % 2 == 1), up, near)
    q = np.sign(v) * grid[near] * np.ldexp(1.0, e)[:, :, None]
    q = np.where(bad[:, :, None], np.nan, q).reshape(R, -1)[:, :C]
    return q, np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, sf, C):
    """What packed codes and row-major scales stand for, in 64 bits."""
    codes, sf = codes.cpu().numpy(), sf.cpu().numpy()
    nib = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    return (O.e2m1_decode(nib) * np.repeat(np.where(sf == 255, np.nan, np.exp2(sf.astype(float) - 127)), 32, axis=1))[:, :C]


def spread_values(shape, seed, dt):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-8, 8, (shape[0], 1), generator=g).float())).to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 32), (3, 31), (2, 33), (5, 100), (129, 64), (7, 256), (33, 1000),
                                 (130, 1001), (4, 4096), (300, 96)])
def test_quantise(ops, R, C, dt):
    x = spread_values((R, C), R + C, dt)
    codes, sf = ops.mx_quantize(x.cuda())
    want, want_sf = plain_quantise(x.double().numpy())
    assert np.array_equal(sf.cpu().numpy(), want_sf)
    assert np.array_equal(values(codes, sf, C), want)
    assert (values(codes, sf, -(-C // 32) * 32)[:, C:] == 0).all()
    for out in ("f32", "bf16"):                        # every value fits both types
        assert np.array_equal(ops.mx_dequantize(codes, sf, C, DT[out]).double().cpu().numpy(), want)


def test_quantise_ties_and_scale_boundaries(ops):
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    edges = sorted(m + s * 2.0 ** -20 for m in mids for s in (-1, 0, 1))
    row = torch.tensor([6.0] + edges + [-v for v in edges[:10]])
    x = torch.stack([row * 2.0 ** k for k in range(-30, 31, 5)])
    amax = torch.tensor([[6.0, 6.0000005, 5.9999995, 12.0, 1e-10, 5e-11, 0.0, 3.4e38, 1e-38, 6 * 2.0 ** -36]]).t()
    x = torch.cat([x, amax.repeat(1, 32) * torch.linspace(0, 1, 32)])
    codes, sf = ops.mx_quantize(x.cuda())
    want, want_sf = plain_quantise(x.double().numpy())
    assert np.array_equal(sf.cpu().numpy(), want_sf) and np.array_equal(values(codes, sf, 32), want)


def test_quantise_agrees_with_the_weight_recipe(ops):
    w = torch.randn(64, 512, generator=torch.Generator().manual_seed(1)) * 0.02
    packed, sf = W.quant_e2m1_ue8m0(w)
    codes, got_sf = ops.mx_quantize(w.cuda())
    assert torch.equal(got_sf.cpu(), sf)
    assert np.array_equal(values(codes, got_sf, 512), values(packed, sf, 512))


def test_quantise_marks_blocks_that_are_not_finite(ops):
    x = torch.ones(4, 96)
    x[0, 5], x[1, 40], x[2, 95] = float("nan"), float("inf"), float("-inf")
    codes, sf = ops.mx_quantize(x.cuda())
    want, want_sf = plain_quantise(x.double().numpy())
    assert np.array_equal(sf.cpu().numpy(), want_sf)
    assert np.array_equal(ops.mx_dequantize(codes, sf, 96).double().cpu().numpy(), want, equal_nan=True)


def test_quantise_strided_rows(ops):
    wide = torch.randn(20, 300, device="cuda", dtype=torch.bfloat16)
    for lo, hi in ((0, 256), (1, 257), (8, 136), (4, 104)):
        a, b = ops.mx_quantize(wide[:, lo:hi]), ops.mx_quantize(wide[:, lo:hi].contiguous())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_quantise_into_slots(ops):
    rng = np.random.default_rng(0)
    idx = np.stack([rng.choice(6, 3, replace=False) for _ in range(50)]).astype(np.int32)
    idx[rng.random(idx.shape) < 0.2] = -1
    r = ops.sort_tokens(torch.from_numpy(idx).cuda(), 6, 128)
    x = torch.randn(50, 160, device="cuda")
    codes, sf = ops.mx_quantize(x, routing=r)
    one, one_sf = ops.mx_quantize(x)
    slot = r.slot.cpu().numpy()
    for t, k in zip(*np.nonzero(slot >= 0)):
        assert torch.equal(codes[slot[t, k]], one[t]) and torch.equal(sf[slot[t, k]], one_sf[t])


# ------------------------------------------------------------------ products
def weights(E, N, C, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (E, N, C // 2), generator=g, dtype=torch.uint8)
    sf = torch.randint(118, 134, (E, N, C // 32), generator=g, dtype=torch.uint8)
    w = values(codes.view(E * N, -1), sf.view(E * N, -1), C).reshape(E, N, C)
    return codes, sf, w


def close(got, q, w, dt):
    """got [R, N] against q [R, C] and w [N, C]: products are exact; every 64-wide step may drop what lies
    2^-22 below the sum of the magnitudes so far; then one rounding to the type."""
    want, size = q @ w.T, np.abs(q) @ np.abs(w).T
    tol = (-(-q.shape[1] // 64) * 2.0 ** -22) * size + 1.01 * HALF_ULP[dt] * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("T", [1, 2, 31, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("N,C", [(1, 32), (7, 96), (64, 64), (65, 256), (200, 288), (256, 512), (1000, 1056)])
def test_linear_dense(ops, T, N, C):
    codes, sf, w = weights(1, N, C, N + C)
    x = spread_values((T, C), T, "f32")
    y = ops.mx_linear(x.cuda(), ops.mx_weights(codes.cuda(), sf.cuda()))
    assert y.shape == (T, N) and y.dtype == torch.float32
    close(y, plain_quantise(x.double().numpy())[0], w[0], "f32")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N", [96, 301, 2048])
def test_linear_types(ops, N, dt):
    codes, sf, w = weights(1, N, 512, 3)
    x = torch.randn(70, 512, generator=torch.Generator().manual_seed(4)).to(DT[dt])
    y = ops.mx_linear(x.cuda(), ops.mx_weights(codes.cuda(), sf.cuda()))
    assert y.dtype == DT[dt]
    close(y, plain_quantise(x.double().numpy())[0], w[0], dt)


@pytest.mark.parametrize("T,N", [(2500, 2600), (1300, 4100), (3000, 700)])
def test_linear_many_tiles(ops, T, N):
    """More tiles than SMs: several tasks a CTA, at every tile width."""
    codes, sf, w = weights(1, N, 320, 5)
    x = torch.randn(T, 320, generator=torch.Generator().manual_seed(6))
    y = ops.mx_linear(x.cuda(), ops.mx_weights(codes.cuda(), sf.cuda()))
    close(y, plain_quantise(x.double().numpy())[0], w[0], "f32")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,C", [(2500, 2600, 4096), (5000, 1030, 3872), (2561, 2560, 7200), (20000, 333, 4128)])
def test_linear_pairs(ops, T, N, C, dt):
    """Long contractions over many rows: CTA pairs, with odd blocks, partial tiles and rows of any alignment. The
    reference takes the quantiser's own values (tested above) and is summed in 64 bits."""
    codes, sf, w = weights(1, N, C, N)
    x = torch.randn(T, C, generator=torch.Generator().manual_seed(T)).to(DT[dt]).cuda()
    y = ops.mx_linear(x, ops.mx_weights(codes.cuda(), sf.cuda()))
    q = ops.mx_dequantize(*ops.mx_quantize(x), C, torch.float32).double()
    w = torch.from_numpy(w[0]).cuda()
    want, size = q @ w.t(), q.abs() @ w.abs().t()
    tol = (-(-C // 64) * 2.0 ** -22) * size + 1.01 * HALF_ULP[dt] * want.abs()
    assert y.dtype == DT[dt] and ((y.double() - want).abs() <= tol).all()
    if dt == "f32":
        buf = torch.full((T, N + 5), 7.0, device="cuda")
        ops.mx_linear(x, ops.mx_weights(codes.cuda(), sf.cuda()), out=buf[:, 3:N + 3])
        assert torch.equal(buf[:, 3:N + 3], y) and (buf[:, :3] == 7).all() and (buf[:, N + 3:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,N,C", [(1, 130, 4128), (2, 129, 8224), (3, 17, 3968), (4, 300, 4096), (1, 1, 12320), (5, 64, 4128)])
def test_linear_few_rows(ops, T, N, C, dt):
    """One launch for up to four rows, over several steps of the contraction, and one row more."""
    codes, sf, w = weights(1, N, C, T)
    wide = torch.randn(T, C + 3, generator=torch.Generator().manual_seed(C)).to(DT[dt])
    x = wide[:, 1:C + 1]
    wt = ops.mx_weights(codes.cuda(), sf.cuda())
    y = ops.mx_linear(x.contiguous().cuda(), wt)
    close(y, plain_quantise(x.double().numpy())[0], w[0], dt)
    assert torch.equal(ops.mx_linear(wide.cuda()[:, 1:C + 1], wt), y)          # rows on no 32-byte boundary


@pytest.mark.parametrize("T,N,C", [(5, 300, 2080), (64, 1000, 4096), (128, 520, 2048), (128, 2048, 3104), (200, 70, 7168),
                                   (300, 1030, 1280), (2, 16400, 4128)])
def test_linear_split_contraction(ops, T, N, C):
    """Few tiles: clusters of CTAs share a tile's contraction, unevenly where it has an odd number of stages."""
    codes, sf, w = weights(1, N, C, N)
    x = torch.randn(T, C, generator=torch.Generator().manual_seed(T))
    wt = ops.mx_weights(codes.cuda(), sf.cuda())
    y = ops.mx_linear(x.cuda(), wt)
    close(y, plain_quantise(x.double().numpy())[0], w[0], "f32")
    assert torch.equal(ops.mx_linear(x.cuda(), wt), y)
    half = ops.mx_linear(x.cuda().bfloat16(), wt)
    close(half, plain_quantise(x.bfloat16().double().numpy())[0], w[0], "bf16")


def run_routed(ops, T, N, C, E, K, masked=0.0, seed=0, idx=None, dt="f32"):
    rng = np.random.default_rng(seed)
    if idx is None:
        idx = np.stack([rng.choice(E, K, replace=False) for _ in range(T)]).astype(np.int32)
        idx[rng.random(idx.shape) < masked] = -1
    codes, sf, w = weights(E, N, C, seed)
    x = torch.randn(T, C, generator=torch.Generator().manual_seed(seed)).to(DT[dt])
    wt = ops.mx_weights(codes.cuda(), sf.cuda())
    r = ops.sort_tokens(torch.from_numpy(idx).cuda(), E, 128)
    out = torch.full((r.rows, N), 7.0, device="cuda", dtype=DT[dt])
    ws = ops.mx_linear_workspace(r.rows, C)
    y = ops.mx_linear(x.cuda(), wt, routing=r, out=out, workspace=ws)
    from moe_expert_forward_gb300 import sync_status
    assert y is out and sync_status(ws)[0] == 0
    q = plain_quantise(x.double().numpy())[0]
    slot = r.slot.cpu().numpy()
    untouched = np.ones(r.rows, bool)
    for e in range(E):
        t, k = np.nonzero((idx == e))
        if len(t):
            close(out[torch.from_numpy(slot[t, k]).long().cuda()], q[t], w[e], dt)
            untouched[slot[t, k]] = False
    assert (out.cpu().float().numpy()[untouched] == 7.0).all()
    # the same from rows quantised on their own: bit for bit, but for the few pairs that one launch sums in another order
    c2, s2 = ops.mx_quantize(x.cuda(), routing=r, chunks=True)
    again = ops.mx_product(c2, s2, wt, routing=r, out=torch.full_like(out, 7.0), dtype=DT[dt])
    if T * K > 16:
        assert torch.equal(again, out)
    for e in range(E):
        t, k = np.nonzero((idx == e))
        if len(t):
            close(again[torch.from_numpy(slot[t, k]).long().cuda()], q[t], w[e], dt)
    assert (again.cpu().float().numpy()[untouched] == 7.0).all()


@pytest.mark.parametrize("T,N,C,E,K", [(1, 64, 64, 4, 2), (5, 130, 96, 8, 3), (128, 256, 256, 16, 4), (400, 200, 288, 3, 2),
                                       (700, 520, 160, 40, 6), (300, 96, 1024, 256, 8)])
def test_linear_routed(ops, T, N, C, E, K):
    run_routed(ops, T, N, C, E, K, seed=T)


def test_linear_routed_masked_and_types(ops):
    run_routed(ops, 150, 160, 128, 12, 4, masked=0.3, seed=1, dt="bf16")
    run_routed(ops, 150, 161, 128, 12, 4, masked=0.9, seed=2, dt="f16")
    run_routed(ops, 2, 160, 4128, 12, 8, masked=0.3, seed=3, dt="bf16")         # few pairs, masked ones among them
    run_routed(ops, 16, 40, 64, 1024, 1, seed=4)
    run_routed(ops, 64, 72, 96, 5, 2, idx=np.full((64, 2), -1, np.int32))       # nothing routed
    run_routed(ops, 520, 300, 128, 5, 1, idx=np.full((520, 1), 4, np.int32))    # one expert, several blocks


def test_linear_not_finite_rows_stay_alone(ops):
    codes, sf, w = weights(1, 128, 256, 9)
    x = torch.randn(40, 256, generator=torch.Generator().manual_seed(2))
    x[3, 200], x[17, 0] = float("nan"), float("inf")
    wt = ops.mx_weights(codes.cuda(), sf.cuda())
    y = ops.mx_linear(x.cuda(), wt)
    assert torch.isnan(y[[3, 17]]).all()
    few = ops.mx_linear(x[2:5].cuda(), wt)
    assert torch.isnan(few[1]).all() and torch.isfinite(few[[0, 2]]).all()
    keep = [t for t in range(40) if t not in (3, 17)]
    close(y[keep], plain_quantise(x[keep].double().numpy())[0], w[0], "f32")


def test_linear_strides_streams_and_repeats(ops):
    codes, sf, w = weights(1, 192, 256, 10)
    wt = ops.mx_weights(codes[0].cuda(), sf[0].cuda())
    wide = torch.randn(50, 300, device="cuda")
    x = wide[:, 3:259]
    ref = ops.mx_linear(x.contiguous(), wt)
    buf = torch.zeros(50, 401, device="cuda")
    assert torch.equal(ops.mx_linear(x, wt, out=buf[:, 5:197]), ref) and (buf[:, 197:] == 0).all() and (buf[:, :5] == 0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = [ops.mx_linear(x, wt, stream=s) for _ in range(20)]
    s.synchronize()
    assert all(torch.equal(v, ref) for v in a)


def test_linear_empty(ops):
    codes, sf, _ = weights(1, 64, 64, 1)
    wt = ops.mx_weights(codes.cuda(), sf.cuda())
    assert ops.mx_linear(torch.zeros(0, 64, device="cuda"), wt).shape == (0, 64)
    c, s = ops.mx_quantize(torch.zeros(0, 64, device="cuda"))
    assert c.shape == (0, 32) and ops.mx_dequantize(c, s, 64).shape == (0, 64)


def test_linear_in_a_graph(ops):
    codes, sf, w = weights(1, 256, 512, 12)
    wt = ops.mx_weights(codes.cuda(), sf.cuda())
    x = torch.randn(20, 512, device="cuda")
    out, ws = torch.empty(20, 256, device="cuda"), ops.mx_linear_workspace(20, 512)
    ops.mx_linear(x, wt, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.mx_linear(x, wt, out=out, workspace=ws)
    for seed in range(3):
        x.copy_(torch.randn(20, 512, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ops.mx_linear(x, wt))


def test_refusals(ops):
    from moe_expert_forward_gb300 import MMError
    codes, sf, _ = weights(2, 64, 64, 1)
    codes, sf = codes.cuda(), sf.cuda()
    one, two = ops.mx_weights(codes[0], sf[0]), ops.mx_weights(codes, sf)
    x = torch.zeros(4, 64, device="cuda")
    idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    r16, r128, r3 = ops.sort_tokens(idx, 2, 16), ops.sort_tokens(idx, 2, 128), ops.sort_tokens(idx, 3, 128)
    c, s = ops.mx_quantize(x, chunks=True)
    for call in (lambda: ops.mx_linear(x[:, :32], one), lambda: ops.mx_linear(x.double(), one),
                 lambda: ops.mx_linear(x, two), lambda: ops.mx_linear(x, two, routing=r16),
                 lambda: ops.mx_linear(x, two, routing=r3), lambda: ops.mx_linear(x[:3], two, routing=r128),
                 lambda: ops.mx_linear(x, one, out=torch.zeros(4, 63, device="cuda")),
                 lambda: ops.mx_linear(x, one, out=torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)),
                 lambda: ops.mx_linear(x.repeat(2, 1), one, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                 lambda: ops.mx_weights(codes[:, :, :8], sf), lambda: ops.mx_weights(codes, sf[:, :, :1]),
                 lambda: ops.mx_weights(codes.cpu(), sf), lambda: ops.mx_quantize(x.int()),
                 lambda: ops.mx_quantize(x[:, :0]), lambda: ops.mx_quantize(x, routing=ops.sort_tokens(idx[:2], 2, 128)),
                 lambda: ops.mx_product(c, s[:-1], one), lambda: ops.mx_product(c[:, :16], s, one),
                 lambda: ops.mx_product(c, s, two), lambda: ops.mx_product(c, s, one, dtype=torch.float64),
                 lambda: ops.mx_dequantize(c, s, 64)):
        with pytest.raises(MMError):
            call()

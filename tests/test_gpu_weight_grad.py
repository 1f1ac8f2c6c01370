"""weight_grad against the formula in 64 bits."""
import time

import numpy as np
import pytest
import torch

from rows8_util import U, d64, randn, routing, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    ops.sync_status()              # what other tests let run out
    return ops


def whole(seed, *shape):
    """Whole numbers from -4 to 4: sums of products are exact in fp32, in any order."""
    return torch.randint(-4, 5, shape, generator=torch.Generator().manual_seed(seed)).float()


def check(ops, d_y, x, r=None, by_token=False, exact=True):
    """d_y [rows, N] bf16 and x (fp32, held in 8 bits here) on the host."""
    C = x.shape[1]
    codes, sf = ops.quantize8(x.cuda())
    got = ops.weight_grad(d_y.cuda(), codes, sf, C, r, by_token, torch.float32)
    xv, dv = values(codes, sf, C), d64(d_y)
    if r is None:
        spans = [(dv, xv)]
    else:
        cnt, blk, src = r.cnt.cpu().numpy(), r.blk_off.cpu().numpy(), r.src.cpu().numpy()
        spans = []
        for e in range(r.E):
            rows = np.arange(cnt[e]) + blk[e] * r.block_m
            spans.append((dv[rows], xv[src[rows] // r.K] if by_token else xv[rows]))
    want = np.stack([d.T @ v for d, v in spans])
    # fp32 sums of exact products, each addition off by at most one step (2 U) of the magnitudes added up
    tol = np.stack([np.abs(d).T @ np.abs(v) * (len(d) + 4) * 2 * U for d, v in spans])
    got64 = d64(got).reshape(want.shape)
    if exact:
        assert np.array_equal(got64, want)
    assert (np.abs(got64 - want) <= tol).all()
    half = ops.weight_grad(d_y.cuda(), codes, sf, C, r, by_token)
    assert half.dtype == torch.bfloat16 and torch.equal(half, got.bfloat16())      # the same sums, rounded once
    assert ops.sync_status() == (0, 0)
    return got


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 63, 64, 65, 128, 300, 1000])
@pytest.mark.parametrize("N,C", [(128, 256), (8, 32), (136, 288)])
def test_dense_rows(ops, rows, N, C):
    check(ops, whole(rows, rows, N).bfloat16(), whole(rows + 1, rows, C))


@pytest.mark.parametrize("N,C", [(1, 1), (1, 256), (7, 33), (64, 31), (127, 255), (129, 257), (130, 1000), (200, 48), (333, 1001),
                                 (16, 4096), (4096, 16), (264, 520), (384, 768)])
def test_dense_widths(ops, N, C):
    check(ops, whole(N, 150, N).bfloat16(), whole(C, 150, C))


@pytest.mark.parametrize("rows,N,C", [(1, 1800, 40), (70, 2048, 96), (200, 1793, 300), (17, 2304, 33), (33, 1024, 64), (33, 1025, 64)])
def test_dense_decoded_first(ops, rows, N, C):
    check(ops, whole(N, rows, N).bfloat16(), whole(C, rows, C))


@pytest.mark.parametrize("by_token", [False, True])
def test_routed_decoded_first(ops, by_token):
    """Many columns of d_y, experts of 0 to 40 rows, NaN in the padding of both operands."""
    T, E, N, C = 61, 7, 1900, 100
    r = ops.sort_tokens(routing(T, E, 2, 0.2, 3).cuda(), E)
    at = r.slot.cpu().flatten()
    at = at[at >= 0].long()
    d_y = torch.full((r.rows, N), float("nan"))
    d_y[at] = whole(1, len(at), N)
    x = whole(2, T if by_token else r.rows, C)
    if not by_token:
        pad = torch.ones(r.rows, dtype=torch.bool)
        pad[at] = False
        x[pad] = float("nan")
    check(ops, d_y.bfloat16(), x, r, by_token)


@pytest.mark.parametrize("N,C", [(1024, 2560), (1024, 2561), (2048, 1537)])
def test_long_sums_of_many_tiles(ops, N, C):
    """33 stages in one task: fp32 results are sums of three accumulators."""
    check(ops, whole(N, 2100, N).bfloat16(), whole(C, 2100, C))


@pytest.mark.parametrize("rows", [1, 70, 1100])
@pytest.mark.parametrize("N,C", [(2600, 1800), (2601, 1799), (5000, 950), (2048, 2560)])
def test_last_tiles_in_halves(ops, rows, N, C):
    """80 to 88 tiles: those past the last whole round of 76 pairs go in halves, some of them past C."""
    check(ops, whole(N, rows, N).bfloat16(), whole(C, rows, C))


def test_last_tiles_of_experts_in_halves(ops):
    """96 tiles of four experts, the last of them without rows, then with most."""
    for seed, dead in ((3, 3), (4, 1)):
        idx = torch.randint(0, 3, (150, 1), generator=torch.Generator().manual_seed(seed))
        r = ops.sort_tokens((idx + (idx >= dead).long()).int().cuda(), 4)
        for by_token in (False, True):
            x = whole(2, 150 if by_token else r.rows, 1000)
            check(ops, whole(1, r.rows, 1400).bfloat16(), x, r, by_token)


def test_many_experts_without_rows(ops):
    r = ops.sort_tokens(torch.tensor([[5], [200], [5]], dtype=torch.int32, device="cuda"), 256)
    for C in (520, 519):
        got = check(ops, whole(1, r.rows, 300).bfloat16(), whole(2, 3, C), r, True)
        dead = torch.ones(256, dtype=torch.bool, device="cuda")
        dead[[5, 200]] = False
        assert not got[dead].any() and got[5].any() and got[200].any()


def test_dense_random_values(ops):
    """Scales of every size, sums of 20000 rows."""
    x = randn(1, 20000, 96) * torch.exp2(torch.arange(96).remainder(17) - 8.0)
    check(ops, randn(2, 20000, 72, dt="bf16"), x, exact=False)


def test_bf16_results_of_very_long_sums(ops):
    """270000 rows of one sign over 42 tiles: the sums of both result types are the same, and right."""
    R, N, C = 270_000, 1792, 1536
    g = torch.Generator(device="cuda").manual_seed(5)
    d_y = torch.rand(R, N, device="cuda", generator=g).bfloat16()
    codes, sf = ops.quantize8(torch.rand(R, C, device="cuda", generator=g))
    got = ops.weight_grad(d_y, codes, sf, C, dtype=torch.float32)
    assert torch.equal(ops.weight_grad(d_y, codes, sf, C), got.bfloat16())
    xv = ops.dequantize8(codes, sf, C, torch.float32)[:, ::100].double()
    want = d_y[:, ::100].double().t() @ xv
    # 16 rows an MMA and 64 MMAs an accumulator, each dropping less than a step (2 U) of it; then 264 additions of U
    assert ((got[::100, ::100].double() - want).abs() <= (64 * 16 * 2 + 266) * U * want).all()


def test_scales_at_the_ends_of_their_range(ops):
    """Codes and scale bytes as a caller may hold them: 2^-127 to 2^127, subnormal codes, both zeros."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 127) != 127]                    # every code but NaN
    codes = torch.cat([codes, codes[:2]])[None].repeat(4, 1).contiguous()
    for byte in (0, 1, 60, 119, 127, 134, 135, 136, 200, 245):
        sf = torch.full((4, 8), byte, dtype=torch.uint8)
        for row, N in ((0, 1), (3, 1), (2, 2000)):             # by the converters, and decoded first
            d_y = torch.zeros(4, N, dtype=torch.bfloat16, device="cuda")
            d_y[row] = 1
            got = d64(ops.weight_grad(d_y, codes.cuda(), sf.cuda(), 256, dtype=torch.float32))[0]
            want = values(codes[:1], sf[:1], 256)[0]
            # bf16 has every value but those between its subnormals, which are 2^-133 apart
            assert (np.abs(got - want) <= (2.0 ** -134 if byte < 4 else 0)).all(), byte
    sf = torch.full((4, 8), 255, dtype=torch.uint8, device="cuda")
    for N in (1, 2000):
        ones = torch.ones(4, N, dtype=torch.bfloat16, device="cuda")
        assert torch.isnan(ops.weight_grad(ones, codes.cuda(), sf, 256, dtype=torch.float32)).all()


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("T,E,K,block,masked", [(1, 3, 1, 16, 0.0), (40, 6, 2, 16, 0.1), (200, 5, 5, 128, 0.5), (300, 40, 3, 32, 0.0),
                                                (33, 4, 2, 256, 1.0), (0, 4, 2, 16, 0.0), (700, 3, 2, 48, 0.0)])
@pytest.mark.parametrize("N,C", [(136, 288), (33, 70)])
def test_routed(ops, T, E, K, block, masked, by_token, N, C):
    """Padding holds NaN in d_y, and in x where x has pool rows."""
    idx = routing(T, E, K, masked, T)
    r = ops.sort_tokens(idx.cuda(), E, block)
    at = r.slot.cpu().flatten()
    at = at[at >= 0].long()
    d_y = torch.full((r.rows, N), float("nan"))
    d_y[at] = whole(1, len(at), N)
    x = whole(2, T if by_token else r.rows, C)
    if not by_token:
        pad = torch.ones(r.rows, dtype=torch.bool)
        pad[at] = False
        x[pad] = float("nan")
    got = check(ops, d_y.bfloat16(), x, r, by_token)
    empty = (r.cnt == 0).cpu()
    assert not got.cpu()[empty].any()


def test_one_expert_takes_everything(ops):
    r = ops.sort_tokens(torch.full((500, 1), 3, dtype=torch.int32, device="cuda"), 6)
    d_y = whole(1, r.rows, 200)
    check(ops, d_y.bfloat16(), whole(2, 500, 100), r, True)


def test_strided_and_unaligned_d_y(ops):
    wide = whole(1, 100, 500).bfloat16().cuda()
    x = whole(2, 100, 300).cuda()
    codes, sf = ops.quantize8(x)
    for lo, hi in ((0, 256), (1, 257), (3, 100), (8, 500), (4, 12)):
        a, b = ops.weight_grad(wide[:, lo:hi], codes, sf, 300), ops.weight_grad(wide[:, lo:hi].contiguous(), codes, sf, 300)
        assert torch.equal(a, b)
        assert torch.equal(a.float(), (wide[:, lo:hi].float().t() @ ops.dequantize8(codes, sf, 300, torch.float32)).bfloat16().float())


def test_many_tiles_and_repeats(ops):
    """More tiles than SMs, several a CTA, bit-equal from run to run."""
    d_y, x = randn(1, 700, 2048, dt="bf16").cuda(), randn(2, 700, 3000).cuda()
    codes, sf = ops.quantize8(x)
    first = ops.weight_grad(d_y, codes, sf, 3000, dtype=torch.float32)
    want = d_y.double().t() @ ops.dequantize8(codes, sf, 3000, torch.float32).double()
    size = d_y.double().abs().t() @ ops.dequantize8(codes, sf, 3000, torch.float32).double().abs()
    assert ((first.double() - want).abs() <= 704 * 2 * U * size).all()
    for _ in range(5):
        assert torch.equal(ops.weight_grad(d_y, codes, sf, 3000, dtype=torch.float32), first)


def test_nan_reaches_its_own_sums_only(ops):
    d_y, x = whole(1, 90, 40).bfloat16().cuda(), whole(2, 90, 100).cuda()
    codes, sf = ops.quantize8(x)
    clean = ops.weight_grad(d_y, codes, sf, 100, dtype=torch.float32)
    d_y[50, 7] = float("nan")
    x[60, 70] = float("inf")                               # its block: columns 64 to 95
    codes, sf = ops.quantize8(x)
    got = ops.weight_grad(d_y, codes, sf, 100, dtype=torch.float32)
    bad = torch.zeros(40, 100, dtype=torch.bool, device="cuda")
    bad[7], bad[:, 64:96] = True, True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], clean[~bad])


def test_empty(ops):
    codes, sf = ops.quantize8(torch.empty(0, 40, device="cuda"))
    for dtype in (torch.bfloat16, torch.float32):
        w = ops.weight_grad(torch.empty(0, 24, device="cuda", dtype=torch.bfloat16), codes, sf, 40, dtype=dtype)
        assert w.shape == (24, 40) and not w.any()


def test_output_past_four_gigabytes(ops):
    """200 experts of 4096 x 4096 in bf16: 6.7 GB."""
    E, N, C = 200, 4096, 4096
    idx = torch.arange(1000, device="cuda", dtype=torch.int32).remainder(E - 1).view(-1, 1).contiguous()
    r = ops.sort_tokens(idx, E)
    d_y, x = torch.randn(r.rows, N, device="cuda", dtype=torch.bfloat16), torch.randn(1000, C, device="cuda")
    codes, sf = ops.quantize8(x)
    got = ops.weight_grad(d_y, codes, sf, C, r, True)
    xv = ops.dequantize8(codes, sf, C, torch.float32)
    for e in (0, 57, 128, 129, 198):
        t = torch.nonzero(idx[:, 0] == e)[:, 0]
        rows = d_y[r.slot[t, 0].long()].double()
        want, size = rows.t() @ xv[t].double(), rows.abs().t() @ xv[t].double().abs()
        assert ((got[e].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 20 * U * size).all()
    assert not got[199].any()


@pytest.mark.parametrize("rows,N,C,routed", [(300, 300, 600, False), (3000, 2000, 6000, False), (3000, 1000, 6000, False), (8192, 128, 256, False),
                                             (600, 300, 600, True)])
def test_a_stage_that_never_comes(ops, monkeypatch, rows, N, C, routed):
    """The call gives up after its limit, says so once, and leaves the GPU in order."""
    import moe_expert_forward_gb300 as M
    r = None
    if routed:
        r = ops.sort_tokens(torch.arange(rows, device="cuda", dtype=torch.int32).remainder(3).view(-1, 1).contiguous(), 3)
        rows = r.rows
    d_y = torch.ones(rows, N, device="cuda", dtype=torch.bfloat16)
    codes, sf = ops.quantize8(torch.ones(rows, C, device="cuda"))
    want = ops.weight_grad(d_y, codes, sf, C, r)
    assert ops.sync_status() == (0, 0)

    class Short:
        def __getattr__(self, name):
            return getattr(real, name)

        def mm_moe_weight_grad(self, *a):
            return real.mm_moe_weight_grad(*a[:19], 50, 1, a[21])
    real = M.lib()
    monkeypatch.setattr(ops, "lib", lambda: Short())
    torch.cuda.synchronize()
    began = time.monotonic()
    ops.weight_grad(d_y, codes, sf, C, r)
    code, where = ops.sync_status()
    assert time.monotonic() - began < 5
    assert code == M.MM_MOE_ERR_TIMEOUT and 181 <= where <= 191
    assert ops.sync_status() == (0, 0)
    monkeypatch.setattr(ops, "lib", lambda: real)
    assert torch.equal(ops.weight_grad(d_y, codes, sf, C, r), want) and ops.sync_status() == (0, 0)


@pytest.mark.parametrize("N", [8, 1025])
def test_codes_of_nan(ops, N):
    """0x7F and 0xFF, which the quantiser does not write but a caller's tensor may hold: NaN, as dequantize8 has it, in
    their own sums alone; none of it from rows that are no expert's."""
    codes, sf = ops.quantize8(whole(1, 40, 70).cuda())
    d_y = whole(2, 40, N).bfloat16().cuda()
    clean = ops.weight_grad(d_y, codes, sf, 70, dtype=torch.float32)
    for row, col, code in ((0, 0, 0x7F), (3, 17, 0xFF), (21, 38, 0x7F), (39, 69, 0xFF)):
        codes[row, col] = code
    bad = torch.isnan(ops.dequantize8(codes, sf, 70)).any(0)
    assert bad.nonzero().flatten().tolist() == [0, 17, 38, 69]
    got = ops.weight_grad(d_y, codes, sf, 70, dtype=torch.float32)
    assert torch.isnan(got[:, bad]).all() and torch.equal(got[:, ~bad], clean[:, ~bad])
    r = ops.sort_tokens(torch.tensor([[0], [1], [1]], dtype=torch.int32, device="cuda"), 3)
    codes, sf = ops.quantize8(whole(3, r.rows, 70).cuda())
    d_y = whole(4, r.rows, N).bfloat16().cuda()
    want = ops.weight_grad(d_y, codes, sf, 70, r)
    padding = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    padding[r.slot.flatten().long()] = False
    codes[padding] = 0x7F
    assert torch.equal(ops.weight_grad(d_y, codes, sf, 70, r), want)


def long_rows(n):
    """n > 16384 values of d_y whose sum with x = 1 shows in fp32 and in bf16 whether an accumulator took more than its rows.
    The first 16384 sum up to 2^24 + 2^16, half way between two bf16 values, each partial sum exact; of those behind, 16 (one
    MMA's) make 1, half of the accumulator's last place there: dropped if they are added to it one MMA at a time, and exact in
    sums of their own."""
    v = torch.full((n,), 2.0 ** -4)
    v[:16384] = 2.0 ** 10
    v[:64] = 2.0 ** 11
    return v, 2.0 ** 24 + 2.0 ** 16 + (n - 16384) / 16


@pytest.mark.parametrize("N,C", [(1792, 1536), (1024, 2560), (1793, 1535), (1024, 2559)])
def test_accumulators_of_long_dense_sums(ops, N, C):
    """40 tiles and more, so that no sum is split into parts: x decoded first and by the converters, results by TMA and row
    by row."""
    v, total = long_rows(40_000)
    d_y = v.cuda().bfloat16()[:, None].repeat(1, N)
    codes, sf = ops.quantize8(torch.ones(len(v), C, device="cuda"))
    for dtype in (torch.float32, torch.bfloat16):
        got = ops.weight_grad(d_y, codes, sf, C, dtype=dtype)
        assert torch.equal(got, torch.full_like(got, total)), dtype          # bf16: up from half way


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("K", [1, 2])
def test_accumulators_of_an_expert_that_takes_nearly_all(ops, K, by_token):
    """One of 64 experts has 40000 rows (K = 2: every token names it twice), two others a few, the average is 640 (1250)."""
    T = 40_000 // K
    idx = torch.full((T + 5, K), 7, dtype=torch.int32)
    idx[T:] = torch.tensor([0, 0, 63, 0, 63], dtype=torch.int32)[:, None]
    r = ops.sort_tokens(idx.cuda(), 64)
    v, total = long_rows(T * K)
    d_y = torch.full((r.rows, 72), float("nan"))
    rows = torch.arange(T * K) + r.blk_off[7].item() * r.block_m
    few = torch.ones(r.rows, dtype=torch.bool)
    few[rows] = False
    d_y[few & (r.src.cpu() >= 0)] = 2.0
    d_y[rows] = v[:, None]
    codes, sf = ops.quantize8(torch.ones(T + 5 if by_token else r.rows, 100, device="cuda"))
    for dtype in (torch.float32, torch.bfloat16):
        got = ops.weight_grad(d_y.bfloat16().cuda(), codes, sf, 100, r, by_token, dtype)
        want = torch.zeros_like(got)
        want[0], want[7], want[63] = 6.0 * K, total, 4.0 * K
        assert torch.equal(got, want), dtype
    assert ops.sync_status() == (0, 0)


@pytest.mark.parametrize("N,C", [(2048, 2560), (1024, 5000)])
def test_long_sums_of_one_sign(ops, N, C):
    """20000 rows of values that round, 80 tiles, no parts: bf16 results from two accumulators, fp32 from 20."""
    g = torch.Generator(device="cuda").manual_seed(N)
    d_y = torch.rand(20_000, N, device="cuda", generator=g).bfloat16()
    codes, sf = ops.quantize8(torch.rand(20_000, C, device="cuda", generator=g))
    want = d_y[:, ::31].double().t() @ ops.dequantize8(codes, sf, C, torch.float32)[:, ::31].double()
    # an MMA's 16 products and its accumulator lose less than a place (2 U) each: 64 MMAs an accumulator in fp32, 1024 in
    # bf16; then the accumulators' additions and (bf16) the rounding
    for dtype, off in ((torch.float32, (64 * 17 * 2 + 20) * U), (torch.bfloat16, (1024 * 17 * 2 + 2) * U + 2.0 ** -8)):
        got = ops.weight_grad(d_y, codes, sf, C, dtype=dtype)[::31, ::31].double()
        assert ((got - want).abs() <= off * want).all(), dtype


@pytest.mark.parametrize("N", [(1 << 30) - 3, 1 << 30])
def test_the_widest_d_y_on_no_boundary(ops, N):
    """A row of 2 GB that is copied to 16-byte boundaries first: its bytes pass 31 bits."""
    d_y = torch.empty(N + 1, dtype=torch.bfloat16, device="cuda").random_(-3, 4)[1:].view(1, N)
    codes, sf = ops.quantize8(torch.full((1, 1), 2.0, device="cuda"))
    got = ops.weight_grad(d_y, codes, sf, 1)
    assert ops.sync_status() == (0, 0) and torch.equal(got, 2 * d_y.view(N, 1))


def test_long_sums_on_two_streams_and_in_graphs(ops):
    """Each call's sums of several accumulators are its own: at once on two streams, captured and replayed with new inputs,
    and from rows of d_y on no boundary."""
    v, total = long_rows(20_000)
    wide = v.cuda().bfloat16()[:, None].repeat(1, 2050)
    codes, sf = ops.quantize8(torch.ones(len(v), 2560, device="cuda"))
    calls = [(wide[:, 1:1025], total), (2 * wide[:, :2048], 2 * total)]
    want = [torch.full((d.shape[1], 2560), t, device="cuda").bfloat16() for d, t in calls]
    for _ in range(3):
        streams = [torch.cuda.Stream() for _ in calls]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                torch.cuda._sleep(2_000_000)
        got = [ops.weight_grad(d, codes, sf, 2560, stream=s) for (d, _), s in zip(calls, streams)]
        for s in streams:
            s.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    graphs = []
    for d, _ in calls:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ops.weight_grad(d, codes, sf, 2560)
        graphs.append((g, out))
    for scale in (1, 4):
        wide.copy_(scale * v[:, None])
        calls[1][0].copy_(2 * wide[:, :2048])
        for (g, out), w in zip(graphs, want):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, scale * w)
    assert ops.sync_status() == (0, 0)


@pytest.mark.parametrize("N", [1024, 2048])
def test_a_stage_that_never_comes_in_a_long_sum(ops, monkeypatch, N):
    import moe_expert_forward_gb300 as M
    real = M.lib()

    class Short:
        def __getattr__(self, name):
            return getattr(real, name)

        def mm_moe_weight_grad(self, *a):
            return real.mm_moe_weight_grad(*a[:19], 50, 1, a[21])
    d_y = torch.ones(20_000, N, device="cuda", dtype=torch.bfloat16)
    codes, sf = ops.quantize8(torch.ones(20_000, 2560, device="cuda"))
    want = ops.weight_grad(d_y, codes, sf, 2560)
    assert (want == torch.tensor(20_000.0).bfloat16().item()).all() and ops.sync_status() == (0, 0)
    monkeypatch.setattr(ops, "lib", lambda: Short())
    ops.weight_grad(d_y, codes, sf, 2560)
    code, where = ops.sync_status()
    assert code == M.MM_MOE_ERR_TIMEOUT and 181 <= where <= 191
    monkeypatch.setattr(ops, "lib", lambda: real)
    assert torch.equal(ops.weight_grad(d_y, codes, sf, 2560), want) and ops.sync_status() == (0, 0)

"""Operators where offsets pass 32 bits, and the products' bounded waits."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def test_rows_beyond_four_gigabytes(ops):
    """320,000 pool rows of 14 KB: the last rows sit past 2^32 bytes."""
    T, K, E, H = 40000, 8, 16, 7168
    g = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(K, 1).indices.int().contiguous()
    r = ops.sort_tokens(idx, E)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    rows = ops.permute(x, r)
    assert rows.numel() * 2 > 2 ** 32 and int(r.slot.max()) > 2 ** 32 // (2 * H)
    picked = torch.randint(0, T, (500,), generator=g, device="cuda")
    last = torch.nonzero(r.slot == r.slot.max())[0, 0]
    picked[0] = last
    for k in range(K):
        assert torch.equal(rows[r.slot[picked, k].long()], x[picked])
    pad = torch.ones(r.rows, dtype=torch.bool, device="cuda")
    pad[r.slot.flatten().long()] = False
    assert not rows[pad].any()
    w = torch.rand(T, K, generator=g, device="cuda")
    y = ops.unpermute(rows, r, w)
    want = x[picked].double() * w[picked].double().sum(1, keepdim=True)
    assert ((y[picked].double() - want).abs() <= 2.0 ** -8 * 1.01 * want.abs() + 2.0 ** -20 * x[picked].abs()).all()
    d_rows, d_w = ops.unpermute_backward(x, rows, r, w)
    for k in range(K):
        want = (w[picked, k, None] * x[picked].float()).bfloat16()
        assert torch.equal(d_rows[r.slot[picked, k].long()], want)
    dots = x[picked].double().square().sum(1, keepdim=True).expand(-1, K)
    assert ((d_w[picked].double() - dots).abs() <= 1e-4 * dots).all()


def test_quantise_beyond_four_gigaelements(ops):
    R, C = 1_060_000, 4096
    x = torch.empty(R, C, device="cuda", dtype=torch.bfloat16)
    for r in range(0, R, 100_000):
        x[r:r + 100_000].normal_()
    codes, sf = ops.mx_quantize(x)
    assert codes.numel() > 2 ** 31
    back = ops.mx_dequantize(codes, sf, C)
    for at in (0, 524_288, 1_048_570, R - 7):
        c, s = ops.mx_quantize(x[at:at + 7].contiguous())
        assert torch.equal(codes[at:at + 7], c) and torch.equal(sf[at:at + 7], s)
        assert torch.equal(back[at:at + 7], ops.mx_dequantize(c, s, C))


@pytest.mark.parametrize("C", [64, 4096])
def test_linear_output_beyond_four_gigabytes(ops, C):
    T, N = 600_000, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    wt = ops.mx_weights(torch.randint(0, 256, (N, C // 2), generator=g, device="cuda", dtype=torch.uint8),
                        torch.randint(119, 123, (N, C // 32), generator=g, device="cuda", dtype=torch.uint8))
    x = torch.randn(T, C, generator=g, device="cuda", dtype=torch.bfloat16)
    y = ops.mx_linear(x, wt)
    for at in (0, 2 ** 32 // (2 * N) - 8, T - 130):
        a, b = y[at:at + 130], ops.mx_linear(x[at:at + 130].contiguous(), wt)
        if C == 64:                                       # one step: every path adds the same exact products
            assert torch.equal(a, b)
        else:                                             # sums in another order, rounded to bf16 once
            assert ((a.double() - b.double()).abs() <= 2.0 ** -7 * b.double().abs() + 2.0 ** -12 * b.double().std()).all()


@pytest.mark.parametrize("T,N,C,routed", [(300, 300, 1024, False), (64, 256, 2048, False), (6000, 2600, 512, False), (6000, 2600, 4096, False),
                                          (200, 300, 512, True)])
def test_a_stage_that_never_comes(ops, T, N, C, routed):
    """Every tile form (one CTA a tile, a split contraction, pairs, routed) gives up after its limit, says where, and
    leaves the GPU in order."""
    import moe_expert_forward_gb300 as M
    E = 4 if routed else 1
    wt = ops.mx_weights(torch.zeros(E, N, C // 2, dtype=torch.uint8, device="cuda"),
                        torch.full((E, N, C // 32), 127, dtype=torch.uint8, device="cuda"))
    r = None
    if routed:
        r = ops.sort_tokens(torch.arange(T, device="cuda", dtype=torch.int32).remainder(E).view(T, 1).contiguous(), E, 128)
    rows = r.rows if routed else T
    codes, sf = ops.mx_quantize(torch.ones(T, C, device="cuda"), routing=r, chunks=True)
    out = torch.zeros(rows, N, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    cnt, blk = (r._cnt, r._blk) if routed else (None, None)
    torch.cuda.synchronize()
    began = time.monotonic()
    code = M.mm_moe_mx_product(codes.data_ptr(), sf.data_ptr(), rows, C, wt.codes.data_ptr(), wt.sfp.data_ptr(), E, N,
                               cnt, blk, 0, out.data_ptr(), N, status.data_ptr(), 50, 1,
                               torch.cuda.current_stream().cuda_stream)
    assert code == M.MM_MOE_OK
    torch.cuda.synchronize()
    assert time.monotonic() - began < 5
    assert int(status[0]) == M.MM_MOE_ERR_TIMEOUT and 161 <= int(status[1]) <= 178
    ops.mx_product(codes, sf, wt, routing=r, out=out, dtype=torch.float32, status=status.zero_())
    assert int(status[0]) == 0 and not out.any()

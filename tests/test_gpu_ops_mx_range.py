"""4-bit linears at both ends of the types' range: x and the weights' scales far from one, results in between."""
import pytest
import torch

from test_gpu_ops_mx import DT, close, plain_quantise, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def case(T, N, C, power, sf0, dt):
    g = torch.Generator().manual_seed(T + N)
    codes = torch.randint(0, 256, (1, N, C // 2), generator=g, dtype=torch.uint8)
    sf = torch.randint(sf0, sf0 + 4, (1, N, C // 32), generator=g, dtype=torch.uint8)
    x = (torch.randn(T, C, generator=g) * 2.0 ** power).to(DT[dt])
    assert torch.isfinite(x).all()
    return codes, sf, x


# x of 2^power through scales of 2^(sf0 - 127) and up: every result lies between 2^-40 and 2^110
@pytest.mark.parametrize("power,sf0", [(118, 60), (124, 87), (118, 0), (60, 1), (-30, 230), (-30, 251), (0, 220)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,C", [(1, 130, 4128), (2, 17, 512), (4, 64, 1056), (5, 64, 1056), (200, 300, 544)])
def test_large_and_small_factors(ops, T, N, C, power, sf0, dt):
    codes, sf, x = case(T, N, C, power, sf0, dt)
    y = ops.mx_linear(x.cuda(), ops.mx_weights(codes.cuda(), sf.cuda()))
    assert torch.isfinite(y).all()
    w = values(codes[0], sf[0], C)
    close(y, plain_quantise(x.double().numpy())[0], w, dt)


@pytest.mark.parametrize("T", [1, 3])
def test_few_routed_pairs(ops, T):
    codes, sf, x = case(T, 40, 1056, 122, 70, "f32")
    codes, sf = codes.repeat(3, 1, 1), sf.repeat(3, 1, 1)
    idx = torch.arange(2, dtype=torch.int32).repeat(T, 1).contiguous()
    r = ops.sort_tokens(idx.cuda(), 3, 128)
    y = ops.mx_linear(x.cuda(), ops.mx_weights(codes.cuda(), sf.cuda()), routing=r)
    q, w = plain_quantise(x.double().numpy())[0], values(codes[0], sf[0], 1056)
    for k in range(2):
        close(y[r.slot[:, k].long()], q, w, "f32")


@pytest.mark.parametrize("T", [1, 5])
def test_full_blocks_of_the_largest_values(ops, T):
    """6 * 2^120 everywhere times 6 * 2^-10 everywhere: 64 products of 36 * 2^110, below the largest fp32."""
    codes = torch.full((1, 8, 32), 0x77, dtype=torch.uint8)
    sf = torch.full((1, 8, 2), 117, dtype=torch.uint8)
    x = torch.full((T, 64), 6 * 2.0 ** 120)
    y = ops.mx_linear(x.cuda(), ops.mx_weights(codes.cuda(), sf.cuda()))
    assert (y.double().cpu() == 64 * 36 * 2.0 ** 110).all()

"""The router's weights and gradients relative to each value, however far it lies below the largest, and rows
whose largest logit is infinite; and every form that the number of rows and experts chooses with a bias."""
import numpy as np
import pytest
import torch

from test_gpu_ops_route import DT, plain, plain_gradient

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


def far_rows(T, E, dt, seed):
    """The largest logit 0, the others 8 to 84 below it in steps of 1/2: exact in every type, and so are the differences."""
    g = torch.Generator().manual_seed(seed)
    x = -torch.randint(16, 169, (T, E), generator=g).float() / 2
    x[:, 3] = 0
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [5, 16384])
def test_softmax_weights_far_below_the_largest(ops, dt, renorm, T):
    """Half units in the last place of fp32: 4 for the exponential (2 whole ones), 12 for at most 12 additions in a sum
    that the largest term, exactly one, dominates, 1 for the division; the sum's other terms add less than 1."""
    x = far_rows(T, 64, dt, T)
    idx, w = ops.route(x.cuda(), 8, renorm=renorm)
    some = slice(0, 200)
    r_idx, r_w, _ = plain(x[some].double().numpy(), 8, None, "softmax", renorm, 1.0)
    assert np.array_equal(idx[some].cpu().numpy(), r_idx)
    err = np.abs(w[some].double().cpu().numpy() - r_w) / r_w
    assert err.max() <= 18 * HALF, err.max() / HALF


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [5, 16384])
def test_softmax_gradient_far_below_the_largest(ops, renorm, T):
    """Incoming gradients of one sign, so that no sum cancels but the chosen logits': the others' relative error is that
    of a weight (17 half units) and of the sum over the chosen (17, 8 products and 3 additions), two products more."""
    x = far_rows(T, 64, "f32", T + 1)
    g = 1 + torch.rand(T, 8, generator=torch.Generator().manual_seed(2))
    idx, _ = ops.route(x.cuda(), 8, renorm=renorm)
    d = ops.route_backward(x.cuda(), idx, g.cuda(), renorm=renorm)
    some = slice(0, 200)
    x64 = x[some].double().numpy()
    r_idx, _, p = plain(x64, 8, None, "softmax", renorm, 1.0)
    ref = plain_gradient(x64, r_idx, g[some].double().numpy(), p, "softmax", renorm, 1.0)
    got = d[some].double().cpu().numpy()
    other = np.ones(ref.shape, bool)
    other[np.arange(len(ref))[:, None], r_idx] = False
    if renorm:
        assert (got[other] == 0).all()
    else:
        err = np.abs(got - ref)[other] / np.abs(ref)[other]
        assert err.max() <= 48 * HALF, err.max() / HALF


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [1, 16384])
def test_no_choice_has_weight_zero_beside_an_infinite_logit(ops, dt, renorm, T):
    x = torch.full((T, 16), -float("inf"), dtype=DT[dt])
    x[:, 5] = float("inf")
    idx, w = ops.route(x.cuda(), 4, renorm=renorm)
    assert (idx.cpu() == torch.tensor([5, -1, -1, -1])).all()
    assert torch.isnan(w[:, 0]).all() and (w[:, 1:] == 0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,K", [(16383, 64, 6), (16384, 64, 6), (32767, 128, 4), (32768, 128, 4), (16384, 160, 8),
                                   (40960, 160, 8), (65536, 162, 2), (65536, 256, 8)])
def test_bias_on_both_sides_of_the_row_rule(ops, T, E, K, dt):
    """The rows' choices and weights are those of the same rows in a small batch, which takes a warp a row; a sum of at
    most 8 scores in another order moves a weight by a few half units of 1."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn(T, E, generator=g, device="cuda").to(DT[dt])
    bias = torch.randn(E, generator=g, device="cuda")
    idx, w = ops.route(x, K, bias=bias, score="sigmoid")
    for at in (0, T // 2, T - 100):
        i, v = ops.route(x[at:at + 100], K, bias=bias, score="sigmoid")
        assert torch.equal(idx[at:at + 100], i)
        assert (w[at:at + 100] - v).abs().max() <= 16 * HALF

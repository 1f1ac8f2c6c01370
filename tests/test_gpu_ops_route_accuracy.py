"""The router's weights of rows whose largest logit is infinite."""
import pytest
import torch

from test_gpu_ops_route import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    return ops


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T", [1, 16384])
def test_no_choice_has_weight_zero_beside_an_infinite_logit(ops, dt, renorm, T):
    x = torch.full((T, 16), -float("inf"), dtype=DT[dt])
    x[:, 5] = float("inf")
    idx, w = ops.route(x.cuda(), 4, renorm=renorm)
    assert (idx.cpu() == torch.tensor([5, -1, -1, -1])).all()
    assert torch.isnan(w[:, 0]).all() and (w[:, 1:] == 0).all()

"""The operators together: the example's layer, served and trained."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from moe_expert_forward_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("routed_layer", os.path.join(ROOT, "examples", "routed_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("sizes", [(512, 1024, 512, 32, 4), (1, 256, 128, 8, 2), (77, 384, 256, 5, 5)])
def test_layer(example, sizes):
    names = ("--tokens", "--hidden", "--inner", "--experts", "--topk")
    found = example.main([str(v) for pair in zip(names, sizes) for v in pair])
    # e2m1 keeps 1 mantissa bit: uniform relative rounding within 1/4 .. 1/6 of a value, about 0.1 of the norm for a
    # Gaussian tensor; three such roundings (x, weights, inner), each through a product, add up to below 0.3.
    assert found["4-bit layer against fp32 weights"] < 0.35
    # only the activations' formats differ: x and the inner values in 4 bits, not 8
    assert found["4-bit layer against the fused layer"] < 0.25
    # bf16 products and roundings of 2^-8 each
    assert found["bf16 layer against autograd"] < 0.015
    assert found["gradient of x against autograd"] < 0.015
    assert found["gradient of the logits against autograd"] < 0.02

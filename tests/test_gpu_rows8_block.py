"""The operators together: a layer's training step with activations kept in 8 bits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from moe_expert_forward_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("trained_block", os.path.join(ROOT, "examples", "trained_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("sizes", [(512, 1024, 512, 16, 4), (1, 256, 128, 8, 2), (77, 384, 200, 5, 5), (300, 200, 72, 7, 1)])
def test_block(example, sizes):
    names = ("--tokens", "--hidden", "--inner", "--experts", "--topk")
    found = example.main([str(v) for pair in zip(names, sizes) for v in pair])
    # bf16 products and roundings of 2^-8 each on the way
    assert found["output against autograd"] < 0.015
    # gate and up, or a weight's own input, come from 8 bits: e4m3 rounds a value by up to 2^-4, uniformly about 2^-4 / sqrt(3)
    # = 0.036 at the low end of a binade and half of it at the high end, so about 0.027 of a tensor's norm, and gradients that
    # pass through gate and up hold three such factors at most
    for name in ("x", "norm weight", "logits", "first weights", "second weights"):
        assert found[f"gradient of {name} against autograd"] < 0.08, name
    # the same gradients with autograd run on the values that were kept: only bf16 is left
    for name in ("x", "norm weight", "logits", "first weights", "second weights"):
        assert found[f"gradient of {name} at the kept values"] < 0.02, name

"""What the operators' kernels must keep to where no run on a healthy GPU shows a breach: read from their source."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_expert_forward_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_the_cluster_barrier_takes_lanes_one_by_one():
    """Its callers (the sort, the split product) reach it from code that lanes of a warp leave at different times; the
    .aligned form is undefined there."""
    body = re.search(r"void cluster_barrier\(\) \{(.*?)\n\}", source("cluster.cuh"), re.S).group(1)
    assert re.findall(r"barrier\.cluster\.(\w+)", body) == ["arrive", "wait"] and ".aligned" not in body

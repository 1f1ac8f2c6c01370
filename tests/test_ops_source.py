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


def test_the_epilogues_wait_as_warps():
    """In the epilogue warps of both products a wait's answer is the whole warp's: lanes that left it one by one, some
    of them giving up, would meet the .aligned tensor memory loads and the shuffles after it without the others."""
    for name in ("mx_linear.cu", "mx_linear_pair.cu"):
        epilogue = source(name).split("----- epilogue", 1)[1]
        assert "mbar_wait_warp(" in epilogue
        assert not re.search(r"mbar_wait(_cluster|_drain)?\(", epilogue.split("__syncthreads")[0])
    body = re.search(r"bool mbar_wait_warp\(.*?\n\}", source("mx_linear.cuh"), re.S).group(0)
    assert "__all_sync(0xffffffffu, mbar_wait(" in body

"""What the kernels on rows in 8 bits must keep to where no run on a healthy GPU shows a breach: read from their source."""
import re

from test_ops_source import source


def test_the_epilogue_waits_as_warps():
    """A wait's answer is the whole warp's: lanes that left it one by one, some of them giving up, would meet the .aligned
    tensor memory loads after it without the others."""
    epilogue = source("weight_grad.cu").split("----- epilogue", 1)[1].split("__syncthreads")[0]
    assert "mbar_wait_warp(" in epilogue and not re.search(r"mbar_wait(_cluster|_drain)?\(", epilogue)


def test_every_wait_of_a_ring_is_bounded():
    """mbarrier waits go through the helpers that give up after a time; nothing spins on its own."""
    for name in ("norm.cu", "weight_grad.cu", "rows8.cuh", "quant8.cu", "swiglu.cu"):
        text = source(name)
        assert "try_wait" not in text and "test_wait" not in text and not re.search(r"while\s*\(\s*(true|1)\s*\)", text), name


def test_the_binding_has_the_kernels_constants():
    """Sizes of scratch are computed in both places."""
    from moe_expert_forward_gb300 import ops
    text = source("weight_grad.cu")
    found = {n: int(re.search(rf"constexpr int [^;]*\b{n} = (\d+)", text).group(1))
             for n in ("kTile", "kRowsPerStage", "kSplitPairs", "kMostParts", "kDecodeTiles")}
    assert (ops.GRAD_TILE, ops.GRAD_STAGE, ops.GRAD_PAIRS, ops.GRAD_PARTS, ops.GRAD_DECODE) == tuple(found.values())
    assert re.search(r"kLongTerms = 1 << (\d+)", text).group(1) == str(ops.GRAD_LONG.bit_length() - 1)
    sms = int(re.search(r"kNormSms = (\d+)", source("internal.h")).group(1))
    assert ops.NORM_CTAS == 2 * sms


def test_the_binding_has_the_accumulators_rows():
    from moe_expert_forward_gb300 import ops
    assert re.search(r"kLongSegment = (\d+)", source("weight_grad.cu")).group(1) == str(ops.GRAD_SEGMENT)

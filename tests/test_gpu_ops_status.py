"""A product's wait that runs out is reported where the call kept no status word of its own."""
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture
def ops():
    from moe_expert_forward_gb300 import build
    build.build()
    from moe_expert_forward_gb300 import ops
    ops.sync_status()              # what other tests let run out
    return ops


class Short:
    """The library, its products with a limit of 50 ms and one stage of each CTA left unloaded."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def mm_moe_mx_product(self, *a):
        return self.lib.mm_moe_mx_product(*a[:14], 50, 1, a[16])


# one CTA a tile, a split contraction, pairs, routed
@pytest.mark.parametrize("T,N,C,routed", [(300, 300, 1024, False), (64, 256, 2048, False), (6000, 2600, 4096, False),
                                          (200, 300, 512, True)])
def test_default_calls_report_a_wait_that_ran_out(ops, monkeypatch, T, N, C, routed):
    import moe_expert_forward_gb300 as M
    E = 4 if routed else 1
    w = ops.mx_weights(torch.full((E, N, C // 2), 0x22, dtype=torch.uint8, device="cuda"),
                       torch.full((E, N, C // 32), 127, dtype=torch.uint8, device="cuda"))
    idx = torch.arange(T, device="cuda", dtype=torch.int32).remainder(E).view(T, 1).contiguous()
    r = ops.sort_tokens(idx, E, 128) if routed else None
    x = torch.ones(T, C, device="cuda")
    codes, sf = ops.mx_quantize(x, routing=r, chunks=True)
    want = ops.mx_product(codes, sf, w, routing=r, dtype=torch.float32)
    assert ops.sync_status() == (0, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    real = M.lib()
    monkeypatch.setattr(ops, "lib", lambda: Short(real))
    for stream in (None, s):
        ops.mx_product(codes, sf, w, routing=r, dtype=torch.float32, stream=stream)
        ops.mx_linear(x, w, routing=r, stream=stream)        # a call that works after it does not hide it
        s.synchronize()
        code, where = ops.sync_status()
        assert code == M.MM_MOE_ERR_TIMEOUT and 161 <= where <= 178
        assert ops.sync_status() == (0, 0)                   # reported once
    monkeypatch.setattr(ops, "lib", lambda: real)
    live = slice(None) if r is None else r.slot[:, 0].long()
    assert torch.equal(ops.mx_product(codes, sf, w, routing=r, dtype=torch.float32)[live], want[live])
    assert (want[live] == C).all() and ops.sync_status() == (0, 0)


def test_the_first_product_of_a_process_may_be_captured():
    """The record's address is looked up by the first call, which a capture allows."""
    code = ("import torch\n"
            "from moe_expert_forward_gb300 import ops\n"
            "w = ops.mx_weights(torch.full((300, 512), 0x22, dtype=torch.uint8, device='cuda'),\n"
            "                   torch.full((300, 32), 127, dtype=torch.uint8, device='cuda'))\n"
            "x, out, ws = torch.ones(64, 1024, device='cuda'), torch.zeros(64, 300, device='cuda'), "
            "ops.mx_linear_workspace(64, 1024)\n"
            "torch.cuda.synchronize()\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n"
            "    ops.mx_linear(x, w, out=out, workspace=ws)\n"
            "g.replay()\n"
            "assert ops.sync_status() == (0, 0) and (out == 1024).all()\n")
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)

"""Routings and weights that are not the current device's are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_host_memory_is_refused():
    from moe_expert_forward_gb300 import MMError, build, ops
    build.build()
    T, K, E, H = 6, 2, 4, 64
    rows = ops.pool_rows(T, K, E, 128)
    r = ops.Routing(T, K, E, 128, rows, "cpu", 0)
    x, pool, w = torch.ones(T, H, device="cuda"), torch.ones(rows, H, device="cuda"), torch.ones(T, K, device="cuda")
    codes, sf = ops.mx_quantize(torch.ones(E * 32, H, device="cuda"))
    experts = ops.mx_weights(codes.view(E, 32, H // 2), sf.view(E, 32, H // 32))
    one = ops.mx_weights(codes, sf)
    chunked = ops.mx_quantize(x, chunks=True)
    for call in (lambda: ops.permute(x, r), lambda: ops.unpermute(pool, r, w), lambda: ops.permute_backward(pool, r),
                 lambda: ops.unpermute_backward(x, pool, r, w), lambda: ops.mx_quantize(x, routing=r),
                 lambda: ops.mx_linear(x, experts, routing=r),
                 lambda: ops.mx_linear(x, one._replace(codes=one.codes.cpu())),
                 lambda: ops.mx_product(*chunked, one._replace(sfp=one.sfp.cpu()))):
        with pytest.raises(MMError):
            call()
    torch.cuda.synchronize()

"""Argument checks of the operators on rows in 8 bits: refused on the host, before any device call."""
import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from moe_expert_forward_gb300 import build
    build.build()
    import moe_expert_forward_gb300 as M
    return M


A = 1 << 20          # an address that is never read: every call here is refused or empty
LONG = 1 << 30


def refused(M, call, cases):
    for kw in cases:
        assert call(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw


def test_quantize(M):
    def q(x=A, dtype=0, stride=64, R=4, C=64, v=0, codes=A, sf=A):
        return M.mm_moe_rows_quantize(x, dtype, stride, R, C, v, codes, sf, None)

    def back(codes=A, sf=A, R=4, C=64, v=0, dtype=1, out=A, stride=64):
        return M.mm_moe_rows_dequantize(codes, sf, R, C, v, dtype, out, stride, None)
    both = [dict(R=-1), dict(C=0), dict(C=LONG + 1, stride=LONG + 1), dict(v=2), dict(v=-1), dict(dtype=3), dict(dtype=-1),
            dict(stride=63), dict(codes=None), dict(codes=A + 8), dict(sf=None), dict(v=1, sf=A + 2)]
    refused(M, q, both + [dict(x=None), dict(x=A + 2)])
    refused(M, back, both + [dict(out=None), dict(out=A + 1)])
    assert q(R=0, x=None, codes=None, sf=None) == M.MM_MOE_OK
    assert back(R=0, out=None, codes=None, sf=None) == M.MM_MOE_OK


def test_norm(M):
    def norm(x=A, dtype=1, xs=64, res=A, rs=64, w=A, wd=1, T=4, H=64, eps=1e-6, h=A, y=A, v=0, codes=A, sf=A, rstd=A):
        return M.mm_moe_rms_norm(x, dtype, xs, res, rs, w, wd, T, H, eps, h, y, v, codes, sf, rstd, None)
    refused(M, norm, [dict(x=None), dict(x=A + 1), dict(dtype=3), dict(xs=63), dict(rs=63), dict(res=None), dict(h=None),
                      dict(h=A + 1), dict(w=None), dict(wd=2), dict(wd=0, w=A + 2), dict(T=-1), dict(H=0), dict(H=LONG + 1, xs=LONG + 1),
                      dict(eps=-1.0), dict(eps=float("nan")), dict(y=A + 1), dict(v=5), dict(codes=None), dict(sf=None),
                      dict(codes=A + 4), dict(v=1, sf=A + 2), dict(rstd=None), dict(rstd=A + 2)])
    assert norm(T=0, x=None, w=None, rstd=None) == M.MM_MOE_OK
    need = M.mm_moe_rms_norm_scratch_size(4, 64)

    def back(dy=A, dtype=1, ys=64, h=A, hs=64, w=A, wd=1, rstd=A, dh=A, ds=64, T=4, H=64, dx=A, dw=A, scr=A, n=need):
        return M.mm_moe_rms_norm_backward(dy, dtype, ys, h, hs, w, wd, rstd, dh, ds, T, H, dx, dw, scr, n, None)
    refused(M, back, [dict(dy=None), dict(dy=A + 1), dict(dtype=4), dict(ys=63), dict(h=None), dict(h=A + 1), dict(hs=63),
                      dict(w=None), dict(wd=2), dict(rstd=None), dict(rstd=A + 1), dict(dh=A + 1), dict(ds=63), dict(T=-1),
                      dict(H=0), dict(dx=None), dict(dx=A + 1), dict(dw=None), dict(dw=A + 2), dict(scr=None),
                      dict(scr=A + 4)])
    assert back(n=need - 1) == M.MM_MOE_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(M.MMError):
        M.mm_moe_rms_norm_scratch_size(-1, 64)


def test_swiglu(M):
    n = 8 + 4 * 15
    pool = dict(T=4, K=2, E=4, bm=16, slot=A, src=A, blk=A)

    def f(h=A, dtype=1, hs=128, rows=n, I=64, T=0, K=0, E=0, bm=0, slot=None, src=None, blk=None, w=None, a=A, codes=A, sf=A,
          kept=A, ksf=A):
        return M.mm_moe_swiglu(h, dtype, hs, rows, I, T, K, E, bm, slot, src, blk, w, a, codes, sf, kept, ksf, None)

    def b(da=A, dtype=1, ds=64, kept=A, ksf=A, rows=n, I=64, T=0, K=0, E=0, bm=0, slot=None, src=None, blk=None, w=None, dh=A,
          dw=None):
        return M.mm_moe_swiglu_backward(da, dtype, ds, kept, ksf, rows, I, T, K, E, bm, slot, src, blk, w, dh, dw, None)
    both = [dict(dtype=3), dict(rows=-1), dict(I=0), dict(I=LONG), dict(w=A), dict(slot=A), dict(src=A), dict(blk=A),
            dict(kept=None), dict(ksf=None), dict(kept=A + 8)]
    both += [dict(pool, **kw) for kw in (dict(slot=None), dict(src=None), dict(blk=None), dict(slot=A + 2), dict(src=A + 1),
                                         dict(T=-1), dict(K=0), dict(K=17, E=20), dict(K=5), dict(E=0), dict(E=1025),
                                         dict(bm=8), dict(bm=24), dict(bm=272), dict(rows=n - 1), dict(w=A + 2))]
    refused(M, f, both + [dict(h=None), dict(h=A + 1), dict(hs=127), dict(a=A + 1), dict(codes=None), dict(sf=None),
                          dict(a=None, codes=None, sf=None, kept=None, ksf=None)])
    refused(M, b, both + [dict(da=None), dict(da=A + 1), dict(ds=63), dict(dh=None), dict(dh=A + 1), dict(kept=None, ksf=None),
                          dict(dw=A), dict(pool, dw=A + 2)])
    assert f(rows=0, h=None) == M.MM_MOE_OK and b(rows=0, da=None, dh=None) == M.MM_MOE_OK


def test_weight_grad(M):
    n = 8 + 4 * 15

    def g(dy=A, ds=64, rows=n, N=64, codes=A, sf=A, C=64, T=4, K=2, E=4, bm=16, cnt=A, src=A, blk=A, tok=0, dtype=1, out=A,
          scr=None, n_scr=0):
        return M.mm_moe_weight_grad(dy, ds, rows, N, codes, sf, C, T, K, E, bm, cnt, src, blk, tok, dtype, out, scr, n_scr, 0, 0,
                                    None)
    dense = dict(cnt=None, src=None, blk=None)
    refused(M, g, [dict(dy=None), dict(dy=A + 1), dict(ds=63), dict(rows=-1), dict(N=0), dict(N=LONG + 1, ds=LONG + 1),
                   dict(codes=None), dict(codes=A + 8), dict(sf=None), dict(C=0), dict(C=LONG + 1), dict(T=-1), dict(K=0),
                   dict(K=5), dict(E=0), dict(E=1025), dict(bm=8), dict(bm=20), dict(cnt=None), dict(src=None),
                   dict(blk=None), dict(cnt=A + 2), dict(rows=n - 1), dict(dtype=2), dict(dtype=-1), dict(out=None),
                   dict(out=A + 1), dict(dtype=0, out=A + 2), dict(dense, tok=1), dict(N=1 << 29, ds=1 << 29),
                   dict(dense, N=1 << 20, ds=1 << 20, C=1 << 30), dict(ds=65), dict(dy=A + 2), dict(ds=65, scr=A + 8, n_scr=1 << 20)])
    need = M.mm_moe_weight_grad_scratch_size(A, 65, n, 64, A, 64, 4, 2, 4, 0)
    assert need == 16 * 8 * n + 4 * n and M.mm_moe_weight_grad_scratch_size(A, 64, n, 64, A, 128, 4, 2, 4, 0) == 0
    assert g(ds=65, scr=A, n_scr=need - 1) == M.MM_MOE_ERR_WORKSPACE_TOO_SMALL
    assert g(tok=1, scr=A, n_scr=2 * 64 * n - 1) == M.MM_MOE_ERR_WORKSPACE_TOO_SMALL
    assert g(tok=1, scr=A + 16, n_scr=2 * 64 * n) == M.MM_MOE_ERR_INVALID_ARG          # stored 32 bytes at a time
    # the router's gradient: 16 tiles, four parts of each
    assert M.mm_moe_weight_grad_scratch_size(A, 256, 8192, 256, A, 4096, 0, 0, 0, 0) == 4 * 256 * 4096 * 4
    for bad in ((A, 63, n, 64, A, 64, 4, 2, 4, 0), (A, 64, -1, 64, A, 64, 4, 2, 4, 0), (A, 64, n, 0, A, 64, 4, 2, 4, 0),
                (A, 64, n, 64, A, 0, 4, 2, 4, 0), (A, 64, n, 64, A, 64, -1, 2, 4, 0), (A, 64, n, 64, A, 64, 4, 17, 4, 0),
                (A, 64, n, 64, A, 64, 4, 0, 4, 0), (A, 64, n, 64, A, 64, 0, 0, 0, 1)):
        with pytest.raises(M.MMError):
            M.mm_moe_weight_grad_scratch_size(*bad)


def test_binding_sizes_agree_with_the_library(M):
    from moe_expert_forward_gb300 import ops
    for T in (0, 1, 7, 303, 304, 305, 1217, 2432, 2433, 100000):
        for H in (1, 16, 17, 512, 513, 1001, 1024, 1025, 4096, 7168, 8192, 8193, 16384, 16400, 100000):
            assert M.mm_moe_rms_norm_scratch_size(T, H) == ops._norm_scratch(T, H), (T, H)
    for at in (A, A + 2, A + 8, A + 16):
        for pitch, N in ((64, 64), (64, 63), (65, 64), (72, 65), (1, 1), (8, 1), (5000, 4096), (5001, 5000)):
            for sf, C in ((A, 128), (A, 129), (A, 96), (A + 1, 256), (A + 4, 1024)):
                for rows in (77, 5000, 100000, 1 << 18, (1 << 18) + 1):
                    for T, K, E, by_token in ((0, 0, 0, False), (2000, 2, 3, False), (2000, 2, 3, True), (50000, 6, 9, True)):
                        args = (at, pitch, rows, N, sf, C, T, K, E, by_token)
                        assert M.mm_moe_weight_grad_scratch_size(*args) == ops._grad_scratch(*args), args


# ------------------------------------------------------------------ tensor forms, with a stand-in for the library
from test_ops_binding import CURRENT, SIDE, Elsewhere, stand  # noqa: E402,F401


def outputs(stream):
    from moe_expert_forward_gb300 import ops
    x, w = torch.ones(6, 64), torch.ones(64)
    r = ops.sort_tokens(torch.ones(6, 2, dtype=torch.int32), 4, 16, stream=stream)
    h, topk_w = torch.ones(r.rows, 64), torch.ones(6, 2)
    codes, sf = ops.quantize8(x, stream=stream)
    f8 = ops.quantize8(x, "f8", stream=stream)
    n = ops.rms_norm(x, w, x, quant="mx", stream=stream)
    f = ops.swiglu(h, r, topk_w, quant=True, keep=True, stream=stream)
    made = [codes, sf, *f8, ops.dequantize8(codes, sf, 64, stream=stream), *n,
            *ops.rms_norm_backward(x, n.h, w, n.rstd, x, stream=stream), *f,
            *ops.swiglu_backward(torch.ones(r.rows, 32), f.kept, f.kept_sf, r, topk_w, stream=stream),
            ops.weight_grad(torch.ones(r.rows, 8, dtype=torch.bfloat16), codes, sf, 64, r, True, stream=stream)]
    return made


def test_results_are_the_launch_streams_and_marked_for_the_current_one(stand):  # noqa: F811
    for stream, owner in ((None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE)):
        stand.shared.clear()
        made = outputs(stream)
        pointers = [t.data_ptr() for t in made]
        assert len(made) == 20 and [stand.stream_of(p) for p in pointers] == [owner] * 20
        marked = [p for p, on in stand.shared if on == CURRENT]
        assert set(pointers) <= set(marked) if owner == SIDE else not marked
        scratch = stand.args("mm_moe_rms_norm_backward")
        assert stand.stream_of(scratch[14]) == owner and scratch[16] == owner


def test_tensor_forms_refuse(M, stand):  # noqa: F811
    from moe_expert_forward_gb300 import ops
    x, w, bf = torch.ones(6, 64), torch.ones(64), torch.bfloat16
    r = ops.sort_tokens(torch.ones(6, 2, dtype=torch.int32), 4, 16)
    h, topk_w, d_a = torch.ones(r.rows, 64), torch.ones(6, 2), torch.ones(r.rows, 32)
    codes, sf = ops.quantize8(x)
    f8 = ops.quantize8(x, "f8")
    n = ops.rms_norm(x, w)
    f = ops.swiglu(h, keep=True)
    d_y = torch.ones(r.rows, 8, dtype=bf)
    far = torch.ones(6, 64).as_subclass(Elsewhere)
    there = ops.sort_tokens(torch.ones(6, 2, dtype=torch.int32), 4, 16)
    there._buf = there._buf.as_subclass(Elsewhere)
    before = len(stand.calls)
    calls = [
        lambda: ops.quantize8(x, "e5m2"), lambda: ops.quantize8(x[:, :0]), lambda: ops.quantize8(x.int()),
        lambda: ops.quantize8(x[0]), lambda: ops.quantize8(x.t()), lambda: ops.quantize8(far),
        lambda: ops.dequantize8(codes, sf, 65), lambda: ops.dequantize8(codes, sf, 0), lambda: ops.dequantize8(codes, f8[1], 64),
        lambda: ops.dequantize8(codes[:, ::2], sf, 32), lambda: ops.dequantize8(codes, sf, 64, torch.float64),
        lambda: ops.dequantize8(codes[0], sf, 64), lambda: ops.dequantize8(codes.as_subclass(Elsewhere), sf, 64),
        lambda: ops.rms_norm(x, w[:63]), lambda: ops.rms_norm(x, w.double()), lambda: ops.rms_norm(x.to(bf), w.half()),
        lambda: ops.rms_norm(x, None), lambda: ops.rms_norm(x, w, x[:5]), lambda: ops.rms_norm(x, w, x.to(bf)),
        lambda: ops.rms_norm(x, w, quant="e4m3"), lambda: ops.rms_norm(x[:, :0], w[:0]), lambda: ops.rms_norm(x, w, far),
        lambda: ops.rms_norm(x, w.as_subclass(Elsewhere)),
        lambda: ops.rms_norm_backward(x, x[:5], w, n.rstd), lambda: ops.rms_norm_backward(x, x, w, n.rstd[:5]),
        lambda: ops.rms_norm_backward(x, x, w, n.rstd, x.to(bf)), lambda: ops.rms_norm_backward(x, None, w, n.rstd),
        lambda: ops.rms_norm_backward(x, x.to(bf), w, n.rstd), lambda: ops.rms_norm_backward(x, x, w, n.rstd.double()),
        lambda: ops.rms_norm_backward(x, far, w, n.rstd),
        lambda: ops.swiglu(h[:, :63]), lambda: ops.swiglu(h[:, :0]), lambda: ops.swiglu(h, rows=False),
        lambda: ops.swiglu(h, None, topk_w), lambda: ops.swiglu(h[1:], r), lambda: ops.swiglu(h, r, topk_w[:5]),
        lambda: ops.swiglu(h, r, topk_w.double()), lambda: ops.swiglu(h, there),
        lambda: ops.swiglu_backward(d_a, f.kept[1:], f.kept_sf), lambda: ops.swiglu_backward(d_a, f.kept, f.kept_sf.int()),
        lambda: ops.swiglu_backward(d_a[:, :31], f.kept[:, :, ::2], f.kept_sf),
        lambda: ops.swiglu_backward(d_a, f.kept, f.kept_sf, None, topk_w), lambda: ops.swiglu_backward(d_a, None, None),
        lambda: ops.swiglu_backward(d_a, f.kept, f.kept_sf, there),
        lambda: ops.weight_grad(d_y.float(), codes, sf, 64, r, True), lambda: ops.weight_grad(d_y, codes, sf, 64, r),
        lambda: ops.weight_grad(d_y[:6], *f8, 64), lambda: ops.weight_grad(d_y[:6], codes, sf, 64, None, True),
        lambda: ops.weight_grad(d_y[:5], codes, sf, 64), lambda: ops.weight_grad(d_y[:6], codes, sf, 96),
        lambda: ops.weight_grad(d_y[:6], codes, sf, 64, dtype=torch.float16),
        lambda: ops.weight_grad(d_y[:6, :0], codes, sf, 64), lambda: ops.weight_grad(d_y, codes, sf, 64, there, True)]
    for i, call in enumerate(calls):
        with pytest.raises(M.MMError):
            call()
            pytest.fail(f"call {i} was taken")
    assert len(stand.calls) == before


def test_tensors_that_require_grad_are_refused_where_a_gradient_would_be_lost(M, stand):  # noqa: F811
    from moe_expert_forward_gb300 import ops
    x, w = torch.ones(6, 64), torch.ones(64)
    need, need_w = x.clone().requires_grad_(), w.clone().requires_grad_()
    r = ops.sort_tokens(torch.ones(6, 2, dtype=torch.int32), 4, 16)
    h, topk_w = torch.ones(r.rows, 64), torch.ones(6, 2).requires_grad_()
    for call in (lambda: ops.rms_norm(need, w), lambda: ops.rms_norm(x, need_w), lambda: ops.rms_norm(x, w, need),
                 lambda: ops.swiglu(need), lambda: ops.swiglu(h, r, topk_w)):
        before = len(stand.calls)
        with pytest.raises(M.MMError, match="requires grad"):
            call()
        assert len(stand.calls) == before
        with torch.no_grad():
            call()
        assert len(stand.calls) == before + 1
    # no gradient passes through these: rounding to 8 bits, and gradients themselves
    codes, sf = ops.quantize8(need)
    ops.rms_norm_backward(need, x, need_w, torch.ones(6))
    ops.weight_grad(torch.ones(6, 8, dtype=torch.bfloat16).requires_grad_(), codes, sf, 64)


def test_scratch_of_long_sums(M):
    """Tiles of fp32 sums, one a pair of CTAs, wherever one sum may pass 16384 rows: dense, or of one expert that takes every
    pair; not where the sums are in parts."""
    from moe_expert_forward_gb300 import ops
    tile = 256 * 256 * 4
    for rows, N, C, T, K, E, want in ((16384, 1024, 2560, 0, 0, 0, 0), (16385, 1024, 2560, 0, 0, 0, 76 * tile),
                                      (17000, 256, 256, 2048, 8, 64, 0), (17000, 256, 256, 2049, 8, 64, 76 * tile),
                                      (17000, 256, 256, 2049, 8, 39, 76 * tile), (20000, 8, 128, 20000, 1, 1, 16 * 8 * 128 * 4)):
        args = (A, N, rows, N, A, C, T, K, E, 0)
        assert M.mm_moe_weight_grad_scratch_size(*args) == ops._grad_scratch(*args) == want, args

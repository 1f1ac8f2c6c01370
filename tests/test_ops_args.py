"""Argument checks of the operators' C entry points: refused on the host, before
any device call, so they run without a GPU."""
import pytest


@pytest.fixture(scope="module")
def M():
    from moe_expert_forward_gb300 import build
    build.build()
    import moe_expert_forward_gb300 as M
    return M


A = 1 << 20          # an address that is never read: every call here is refused or empty


def test_route(M):
    def call(logits=A, dtype=0, stride=8, T=4, E=8, K=2, bias=None, score=0, idx=A, w=A):
        return M.mm_moe_route(logits, dtype, stride, T, E, K, bias, score, 1, 1.0, idx, w, None)
    bad = [dict(logits=None), dict(logits=A + 2), dict(dtype=3), dict(stride=7), dict(T=-1), dict(E=0), dict(E=1025, stride=1025),
           dict(K=0), dict(K=9), dict(K=17, E=32, stride=32), dict(score=2), dict(bias=A), dict(idx=None), dict(w=None),
           dict(w=A + 1), dict(T=2 ** 31 - 1, K=2)]
    for kw in bad:
        assert call(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    assert call(T=0, logits=None, idx=None, w=None) == M.MM_MOE_OK


def test_route_backward(M):
    def call(logits=A, idx=A, g=A, T=4, d=A, d_stride=8, **kw):
        return M.mm_moe_route_backward(logits, kw.get("dtype", 1), 8, idx, g, T, 8, 2, 0, 1, 1.0, d, d_stride, None)
    for kw in (dict(logits=None), dict(idx=None), dict(g=None), dict(d=None), dict(d=A + 1), dict(d_stride=7), dict(dtype=-1)):
        assert call(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    assert call(T=0, logits=None, idx=None, g=None, d=None) == M.MM_MOE_OK


def test_sort(M):
    def sort(idx=A, T=4, K=2, E=4, bm=16, cnt=A, blk=A, slot=A, src=A, cap=8 + 4 * 15, scr=None, n=0, status=A):
        return M.mm_moe_sort(idx, T, K, E, bm, cnt, blk, slot, src, cap, scr, n, status, None)
    for kw in (dict(idx=None), dict(T=-1), dict(K=0), dict(K=5), dict(E=0), dict(E=1025), dict(bm=8), dict(bm=20),
               dict(cnt=None), dict(blk=None), dict(slot=None), dict(src=None), dict(cap=67), dict(status=None),
               dict(T=1 << 20, cap=1 << 24)):                       # two launches need scratch
        assert sort(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    need = M.mm_moe_sort_scratch_size(1 << 20, 2, 4)
    assert need > 0 and M.mm_moe_sort_scratch_size(4, 2, 4) == 0
    assert sort(T=1 << 20, cap=1 << 24, scr=A, n=need - 1) == M.MM_MOE_ERR_WORKSPACE_TOO_SMALL


def test_rows(M):
    def permute(x=A, dtype=0, stride=8, T=4, H=8, K=2, E=4, bm=16, slot=A, src=A, blk=A, rows=A, n=8 + 4 * 15):
        return M.mm_moe_permute(x, dtype, stride, T, H, K, E, bm, slot, src, blk, rows, n, None)

    def back(d=A, dtype=0, stride=8, rows=A, T=4, H=8, K=2, E=4, bm=16, src=A, d_rows=A, n=8 + 4 * 15, d_w=A):
        return M.mm_moe_unpermute_backward(d, dtype, stride, rows, T, H, K, E, bm, A, src, A, A, d_rows, n, d_w, None)

    def unpermute(rows=A, dtype=0, n=68, T=4, H=8, K=2, slot=A, out=A, stride=8):
        return M.mm_moe_unpermute(rows, dtype, n, T, H, K, slot, None, out, stride, None)
    for kw in (dict(x=None), dict(x=A + 2), dict(dtype=9), dict(stride=7), dict(T=-1), dict(H=0), dict(K=0), dict(K=5),
               dict(bm=8), dict(bm=272), dict(bm=20), dict(slot=None), dict(src=None), dict(blk=None), dict(rows=None),
               dict(n=8 + 4 * 15 - 1), dict(n=-1)):
        assert permute(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    for kw in (dict(d=None), dict(stride=7), dict(rows=None), dict(src=None), dict(d_rows=None), dict(n=60), dict(dtype=3)):
        assert back(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    for kw in (dict(rows=None), dict(slot=None), dict(out=None), dict(out=A + 1), dict(stride=7), dict(H=0), dict(K=17)):
        assert unpermute(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    assert unpermute(T=0, rows=None, slot=None, out=None) == M.MM_MOE_OK
    assert permute(T=0, n=0, x=None, slot=None, src=None, blk=None, rows=None) == M.MM_MOE_OK


def test_quantise(M):
    def q(x=A, dtype=0, stride=64, R=4, C=64, slot=None, K=1, n=4, codes=A, sf=A, chunks=1):
        return M.mm_moe_mx_quantize(x, dtype, stride, R, C, slot, K, n, codes, sf, chunks, None)
    for kw in (dict(x=None), dict(dtype=3), dict(stride=63), dict(R=-1), dict(C=0), dict(codes=None), dict(codes=A + 4),
               dict(sf=None), dict(sf=A + 4), dict(slot=A, K=0), dict(slot=A, K=17), dict(slot=A, n=-1)):
        assert q(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    assert q(R=0, x=None, codes=None, sf=None) == M.MM_MOE_OK
    assert M.mm_moe_mx_dequantize(None, A, 4, 64, 1, A, 64, None) == M.MM_MOE_ERR_INVALID_ARG
    assert M.mm_moe_mx_dequantize(A, A, 4, 64, 1, A, 63, None) == M.MM_MOE_ERR_INVALID_ARG
    assert M.mm_moe_mx_prepare(A, 2000, 8, 64, A, None) == M.MM_MOE_ERR_INVALID_ARG
    assert M.mm_moe_mx_prepare(None, 2, 8, 64, A, None) == M.MM_MOE_ERR_INVALID_ARG
    with pytest.raises(M.MMError):
        M.mm_moe_mx_scale_size(-1, 64)


def test_product(M):
    def p(codes=A, sf=A, rows=128, C=64, w=A, w_sf=A, E=1, N=8, cnt=None, blk=None, dtype=1, out=A, stride=8, status=A):
        return M.mm_moe_mx_product(codes, sf, rows, C, w, w_sf, E, N, cnt, blk, dtype, out, stride, status, 0, 0, None)
    for kw in (dict(codes=None), dict(codes=A + 8), dict(sf=None), dict(rows=-1), dict(C=48), dict(C=0), dict(w=None),
               dict(w=A + 8), dict(w_sf=None), dict(E=2), dict(N=0), dict(cnt=A), dict(blk=A), dict(dtype=4),
               dict(out=None), dict(out=A + 1), dict(stride=7), dict(status=None), dict(rows=100, cnt=A, blk=A)):
        assert p(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    assert p(rows=0, codes=None, sf=None, out=None, status=None) == M.MM_MOE_OK


def test_linear(M):
    need = M.mm_moe_mx_linear_workspace(8, 64, 8, 0, 8)

    def lin(x=A, dtype=1, stride=64, T=8, C=64, w=A, E=1, N=8, slot=None, K=0, cnt=None, blk=None, n=8, out=A, ws=A,
            size=need):
        return M.mm_moe_mx_linear(x, dtype, stride, T, C, w, A, E, N, slot, K, cnt, blk, n, out, N, ws, size, 0, None)
    for kw in (dict(x=None), dict(x=A + 1), dict(dtype=7), dict(stride=63), dict(T=-1, n=-1), dict(C=63), dict(w=None),
               dict(E=2), dict(slot=A), dict(cnt=A, blk=A), dict(n=5), dict(out=None), dict(ws=None), dict(ws=A + 16),
               dict(slot=A, K=2, cnt=A, blk=A, E=4, n=128),              # a pool too small for any routing
               dict(slot=A, K=0, cnt=A, blk=A, E=4, n=1024)):
        assert lin(**kw) == M.MM_MOE_ERR_INVALID_ARG, kw
    assert lin(size=need - 1) == M.MM_MOE_ERR_WORKSPACE_TOO_SMALL
    assert lin(T=4, n=4, size=8) == M.MM_MOE_ERR_WORKSPACE_TOO_SMALL      # given, it holds a status word
    assert lin(T=4, n=4, x=None, ws=None, size=0) == M.MM_MOE_ERR_INVALID_ARG
    for bad in ((4, 100, 8, 0, 4), (4, 64, 8, 0, 5), (-1, 64, 8, 0, -1), (4, 64, 8, 17, 512), (4, 64, 0, 0, 4)):
        with pytest.raises(M.MMError):
            M.mm_moe_mx_linear_workspace(*bad)


def test_words_on_no_boundary_and_rows_of_any_length(M):
    odd = A + 2                                     # an int32 or fp32 array there would fault on the device
    bad = M.MM_MOE_ERR_INVALID_ARG
    long = 1 << 30                                  # the longest row

    def sort(idx=A, cnt=A, blk=A, slot=A, src=A, status=A):
        return M.mm_moe_sort(idx, 4, 2, 4, 16, cnt, blk, slot, src, 8 + 4 * 15, None, 0, status, None)
    for name in ("idx", "cnt", "blk", "slot", "src", "status"):
        assert sort(**{name: odd}) == bad, name

    def permute(H=8, slot=A, src=A, blk=A):
        return M.mm_moe_permute(A, 1, H, 4, H, 2, 4, 16, slot, src, blk, A, 8 + 4 * 15, None)

    def unpermute(H=8, slot=A, w=A):
        return M.mm_moe_unpermute(A, 1, 68, 4, H, 2, slot, w, A, H, None)

    def back(H=8, slot=A, src=A, blk=A, w=A, d_w=A):
        return M.mm_moe_unpermute_backward(A, 1, H, A, 4, H, 2, 4, 16, slot, src, blk, w, A, 8 + 4 * 15, d_w, None)
    for f, names in ((permute, ("slot", "src", "blk")), (unpermute, ("slot", "w")),
                     (back, ("slot", "src", "blk", "w", "d_w"))):
        for name in names:
            assert f(**{name: odd}) == bad, (f.__name__, name)
        assert f(H=long + 1) == bad, f.__name__
    assert M.mm_moe_mx_quantize(A, 1, 64, 4, 64, odd, 1, 128, A, A, 1, None) == bad

    def product(cnt=A, blk=A, status=A):
        return M.mm_moe_mx_product(A, A, 128, 64, A, A, 4, 8, cnt, blk, 1, A, 8, status, 0, 0, None)

    def linear(slot=A, cnt=A, blk=A):
        return M.mm_moe_mx_linear(A, 1, 64, 8, 64, A, A, 4, 8, slot, 2, cnt, blk, 1024, A, 8, A, 1 << 20, 0, None)
    for name in ("cnt", "blk", "status"):
        assert product(**{name: odd}) == bad, name
    for name in ("slot", "cnt", "blk"):
        assert linear(**{name: odd}) == bad, name


def test_binding_sizes_agree_with_the_library(M):
    from moe_expert_forward_gb300 import ops
    for rows, C in ((1, 32), (129, 96), (1000, 4096)):
        assert M.mm_moe_mx_scale_size(rows, C) == ops._scale_bytes(rows, C)
    for T in (0, 1, 1000, 24576, 24577, 100000):
        for K, E in ((1, 1), (2, 60), (8, 1024)):
            assert M.mm_moe_sort_scratch_size(T, K, E) == ops._sort_scratch(T, K, E), (T, K, E)
    for T in (0, 1, 2, 3, 4, 5, 100):
        for K in (0, 1, 3, 4, 8):
            for C in (32, 4096, 36384, 65536, 145632, 200000 // 32 * 32):
                for N in (1, 300, 2048, 4096, 8192, 16384):
                    rows = T if K == 0 else ops.pool_rows(T, K, 16, 128)
                    want = 0 if ops._few(T, C, N, K) else ops._linear_bytes(rows, C)
                    assert M.mm_moe_mx_linear_workspace(T, C, N, K, rows) == want, (T, K, C, N)

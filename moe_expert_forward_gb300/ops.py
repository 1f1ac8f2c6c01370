"""Operators around the expert layer, on torch tensors.

  route, route_backward         a router's top-k with its weights, and the gradient
  sort_tokens                   the routing of a batch: every pair's pool row
  permute, permute_backward     tokens into rows sorted by expert, and the gradient
  unpermute, unpermute_backward rows back to tokens, weighted, and the gradients
  mx_quantize, mx_dequantize    rows into 4-bit e2m1 with a UE8M0 scale per 32, and back
  mx_weights, mx_product, mx_linear
                                products of 4-bit operands: dense, or each expert's
                                rows with its matrix
  sync_status                   whether a device wait of a product has run out

Argument marshalling and checks only; the arithmetic is in the CUDA library,
whose C entry points (include/mm_moe.h) define each operator.  Every function
enqueues on `stream` (default: the current stream) of the current device and
returns at once.  What a call allocates is `stream`'s memory; its results are
also marked as used on the stream that is current at the call (7 us a tensor on the
host; `with torch.cuda.stream(s):` around calls makes s the current stream and needs
none of it).  Other uses of a tensor on a stream that it was not allocated on are
the caller's to order and to keep alive.

Nothing here is recorded by autograd: the *_backward calls give the gradients, for
example from a torch.autograd.Function.  So while grad mode is on, the calls whose
result a gradient would flow through refuse tensors that require one; detach them,
or call under torch.no_grad().
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import (MM_MOE_ERR_INVALID_ARG, MM_MOE_SCORE_SIGMOID, MM_MOE_SCORE_SOFTMAX, MMError, _check, lib,
               mm_moe_ops_status)

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCORES = {"softmax": MM_MOE_SCORE_SOFTMAX, "sigmoid": MM_MOE_SCORE_SIGMOID}
PRODUCT_BLOCK = 128      # rows of a routed block the 4-bit product reads


class Routing:
    """Where every (token, k) pair of a batch sits in a pool sorted by expert.

    T, K, E, block_m: of the batch; rows: pool rows that any routing of these sizes
    fits.  The tensors are views of one buffer:
      cnt      int32 [E]      rows of each expert
      blk_off  int32 [E + 1]  first block of each expert
      slot     int32 [T, K]   pool row of each pair, -1 where masked
      src      int32 [rows]   pair of each pool row, -1 on padding (undefined past the last block)
      status   int32 [4]      [0] = MM_MOE_ERR_BAD_ROUTING where topk_idx held other ids
    """
    __slots__ = ("T", "K", "E", "block_m", "rows", "_buf", "_status", "_cnt", "_blk", "_slot", "_src")

    def __init__(self, T: int, K: int, E: int, block_m: int, rows: int, device, scratch_ints: int, stream=None):
        self.T, self.K, self.E, self.block_m, self.rows = T, K, E, block_m, rows
        self._buf = _result(stream, 5 + 2 * E + T * K + rows + scratch_ints, torch.int32, device)
        self._status = p = self._buf.data_ptr()      # addresses, for the calls
        self._cnt = p + 16
        self._blk = p + 16 + 4 * E
        self._slot = p = p + 20 + 8 * E
        self._src = p + 4 * T * K

    @property
    def status(self):
        return self._buf.as_strided((4,), (1,), 0)

    @property
    def cnt(self):
        return self._buf.as_strided((self.E,), (1,), 4)

    @property
    def blk_off(self):
        return self._buf.as_strided((self.E + 1,), (1,), 4 + self.E)

    @property
    def slot(self):
        return self._buf.as_strided((self.T, self.K), (self.K, 1), 5 + 2 * self.E)

    @property
    def src(self):
        return self._buf.as_strided((self.rows,), (1,), 5 + 2 * self.E + self.T * self.K)


class MxWeights(NamedTuple):
    """4-bit matrices with their scales in the product's order."""
    codes: torch.Tensor    # u8 [E, N, C/2]
    sfp: torch.Tensor
    E: int
    N: int
    C: int


def _bad(what: str, why: str):
    raise MMError(MM_MOE_ERR_INVALID_ARG, f"{what}: {why}")


_device = torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # absent in builds of torch without CUDA


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_streams = {}            # torch's objects of streams by device and number; making one takes 2 us


def _torch_stream(device: int, ptr: int, make):
    key = (device, ptr)
    if key not in _streams:
        _streams[key] = make()
    return _streams[key]


def _new(stream, shape, dtype, device, zero=False, shared=False):
    """A tensor (uninitialised, or zeroed in `stream`'s order) for a call on `stream`, of that stream's memory: what the
    current stream frees and takes again would otherwise meet kernels that `stream` still runs.  shared: marked as used
    on the current stream too.  (torch.cuda.stream as a context would do; it takes about 15 us, a whole call 10.)"""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    ptr, dev = _stream(stream), _device()
    current = _raw_stream(dev)
    if ptr == current:
        return make(shape, dtype=dtype, device=device)
    here = _torch_stream(dev, current, torch.cuda.current_stream)
    # stream 0 has no external form
    there = _torch_stream(dev, ptr, lambda: torch.cuda.ExternalStream(ptr) if ptr else torch.cuda.default_stream())
    torch.cuda.set_stream(there)
    try:
        t = make(shape, dtype=dtype, device=device)
    finally:
        torch.cuda.set_stream(here)
    if shared:
        t.record_stream(here)
    return t


def _result(stream, shape, dtype, device):
    """What a call on `stream` returns: memory that no work queued on the current stream still uses, and that is not
    taken again before the work which the current stream has been given when it is freed."""
    return _new(stream, shape, dtype, device, shared=True)


def _here(t, what: str, name: str):
    """A tensor on the current CUDA device."""
    if not isinstance(t, torch.Tensor) or t.get_device() != _device():
        _bad(what, f"{name} must be a tensor on the current CUDA device")


def _no_grad(what: str, *tensors):
    """A result without a gradient is no answer to a tensor that requires one."""
    if torch.is_grad_enabled():
        for t in tensors:
            if getattr(t, "requires_grad", False):     # what is no tensor is refused by the checks after this
                _bad(what, "a tensor requires grad, and autograd does not see this call: detach it, or call under "
                           "torch.no_grad() (gradients: the *_backward calls)")


def _routing_here(r: Routing, what: str):
    """The calls pass a routing's addresses on, so it has to be the current device's."""
    _here(r._buf, what, "routing")


def _rows(t, what: str, name: str, cols: Optional[int] = None, dtype=None) -> int:
    """dtype code of a 2-D tensor with unit column stride and rows that do not overlap."""
    _here(t, what, name)
    code = _DTYPES.get(t.dtype)
    if code is None or (dtype is not None and t.dtype != dtype):
        _bad(what, f"{name} must be {dtype or 'float32, bfloat16 or float16'}, got {t.dtype}")
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols):
        _bad(what, f"{name} must be [rows, {'columns' if cols is None else cols}], got {tuple(t.shape)}")
    if not t.is_contiguous():
        R, C = t.shape
        if (C > 1 and t.stride(1) != 1) or (R > 1 and t.stride(0) < C):
            _bad(what, f"{name} must have contiguous columns and rows that do not overlap, got {tuple(t.shape)} "
                       f"strides {t.stride()}")
    return code


def _pitch(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _whole(t, what: str, name: str, shape, dtype):
    """A contiguous tensor of exactly this shape and type."""
    _here(t, what, name)
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _bad(what, f"{name} must be contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)} "
                   f"strides {t.stride()}")
    return t.data_ptr()


# ------------------------------------------------------------------ router
def route(logits, k: int, bias=None, score: str = "softmax", renorm: bool = True, scale: float = 1.0, stream=None):
    """Top-k experts and weights of logits [T, E]: (topk_idx int32 [T, k], topk_w fp32 [T, k]).

    The k largest logits, or with bias (fp32 [E], sigmoid only) the k largest
    sigmoid(logit) + bias; equal keys by ascending expert; -inf and NaN never (index
    -1, weight 0).  Weights: scale times the softmax over all experts, or the
    sigmoid, of the chosen logits, divided by their sum where renorm."""
    code = _rows(logits, "route", "logits")
    _no_grad("route", logits, bias)
    T, E = logits.shape
    if score not in _SCORES:
        _bad("route", f"score must be one of {sorted(_SCORES)}, got {score!r}")
    bp = None if bias is None else _whole(bias, "route", "bias", (E,), torch.float32)
    idx = _result(stream, (T, k), torch.int32, logits.device)
    w = _result(stream, (T, k), torch.float32, logits.device)
    _check(lib().mm_moe_route(logits.data_ptr(), code, _pitch(logits), T, E, k, bp, _SCORES[score], renorm, scale,
                              idx.data_ptr(), w.data_ptr(), _stream(stream)), "mm_moe_route")
    return idx, w


def route_backward(logits, topk_idx, d_topk_w, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
                   stream=None):
    """Gradient of route's weights with respect to the logits: [T, E] in the logits' type."""
    code = _rows(logits, "route_backward", "logits")
    T, E = logits.shape
    if score not in _SCORES:
        _bad("route_backward", f"score must be one of {sorted(_SCORES)}, got {score!r}")
    k = topk_idx.shape[-1]
    ip = _whole(topk_idx, "route_backward", "topk_idx", (T, k), torch.int32)
    dp = _whole(d_topk_w, "route_backward", "d_topk_w", (T, k), torch.float32)
    d = _result(stream, (T, E), logits.dtype, logits.device)
    _check(lib().mm_moe_route_backward(logits.data_ptr(), code, _pitch(logits), ip, dp, T, E, k, _SCORES[score], renorm,
                                       scale, d.data_ptr(), E, _stream(stream)), "mm_moe_route_backward")
    return d


# ------------------------------------------------------------------ tokens by expert
def pool_rows(T: int, K: int, E: int, block_m: int) -> int:
    """Rows of a pool that any routing of these sizes fits: whole blocks."""
    pairs = T * K
    return -(-(pairs + min(pairs, E) * (block_m - 1)) // block_m) * block_m


SORT_ONE_LAUNCH = 3 << 16     # pairs up to which mm_moe_sort needs no scratch (mm_moe_sort_scratch_size)


def _sort_scratch(T: int, K: int, E: int) -> int:
    return 0 if T * K <= SORT_ONE_LAUNCH else 4 * 256 * E


def sort_tokens(topk_idx, E: int, block_m: int = 16, stream=None) -> Routing:
    """The routing of topk_idx (int32 [T, K], -1 masked): pairs in ascending order
    inside each expert, every expert's rows padded to whole blocks of block_m (16 to
    256, a multiple of 16; 128 for the 4-bit product)."""
    if topk_idx.dim() != 2:
        _bad("sort_tokens", f"topk_idx must be [T, K], got {tuple(topk_idx.shape)}")
    T, K = topk_idx.shape
    ip = _whole(topk_idx, "sort_tokens", "topk_idx", (T, K), torch.int32)
    if block_m < 1 or E < 1:
        _bad("sort_tokens", f"block_m must be 16 to 256 and E at least 1, got {block_m} and {E}")
    scratch = _sort_scratch(T, K, E)
    rows = pool_rows(T, K, E, block_m)
    r = Routing(T, K, E, block_m, rows, topk_idx.device, scratch // 4, stream)
    _check(lib().mm_moe_sort(ip, T, K, E, block_m, r._cnt, r._blk, r._slot, r._src, rows, r._src + 4 * rows, scratch,
                             r._status, _stream(stream)), "mm_moe_sort")
    return r


def permute(x, routing: Routing, stream=None):
    """Tokens x [T, H] at their pool rows: [routing.rows, H], zero on padding."""
    code = _rows(x, "permute", "x")
    _no_grad("permute", x)
    r = routing
    _routing_here(r, "permute")
    T, H = x.shape
    if T != r.T:
        _bad("permute", f"x has {T} tokens, the routing {r.T}")
    rows = _result(stream, (r.rows, H), x.dtype, x.device)
    _check(lib().mm_moe_permute(x.data_ptr(), code, _pitch(x), T, H, r.K, r.E, r.block_m, r._slot,
                                r._src, r._blk, rows.data_ptr(), r.rows, _stream(stream)),
           "mm_moe_permute")
    return rows


def unpermute(rows, routing: Routing, topk_w=None, stream=None):
    """Pool rows [routing.rows, H] back to tokens [T, H]: the sum of each token's
    rows times topk_w (fp32 [T, K]; None: ones), masked slots left out."""
    _no_grad("unpermute", rows, topk_w)
    return _unpermute(rows, routing, topk_w, stream)


def _unpermute(rows, r: Routing, topk_w, stream):
    code = _rows(rows, "unpermute", "rows")
    _routing_here(r, "unpermute")
    H = rows.shape[1]
    if rows.shape[0] != r.rows or not rows.is_contiguous():
        _bad("unpermute", f"rows must be contiguous [{r.rows}, H], got {tuple(rows.shape)}")
    wp = None if topk_w is None else _whole(topk_w, "unpermute", "topk_w", (r.T, r.K), torch.float32)
    out = _result(stream, (r.T, H), rows.dtype, rows.device)
    _check(lib().mm_moe_unpermute(rows.data_ptr(), code, r.rows, r.T, H, r.K, r._slot, wp, out.data_ptr(), H,
                                  _stream(stream)), "mm_moe_unpermute")
    return out


def permute_backward(d_rows, routing: Routing, stream=None):
    """Gradient of permute: the sum of the gradients of each token's rows, [T, H]."""
    return _unpermute(d_rows, routing, None, stream)


def unpermute_backward(d_out, rows, routing: Routing, topk_w=None, stream=None):
    """Gradients of unpermute: (d_rows [routing.rows, H], zero on padding, and d_topk_w
    fp32 [T, K]; without topk_w the second is None and rows is not read)."""
    code = _rows(d_out, "unpermute_backward", "d_out")
    r = routing
    _routing_here(r, "unpermute_backward")
    T, H = d_out.shape
    if T != r.T:
        _bad("unpermute_backward", f"d_out has {T} tokens, the routing {r.T}")
    wp = rp = d_w = None
    if topk_w is not None:
        wp = _whole(topk_w, "unpermute_backward", "topk_w", (T, r.K), torch.float32)
        rp = _whole(rows, "unpermute_backward", "rows", (r.rows, H), d_out.dtype)
        d_w = _result(stream, (T, r.K), torch.float32, d_out.device)
    d_rows = _result(stream, (r.rows, H), d_out.dtype, d_out.device)
    _check(lib().mm_moe_unpermute_backward(d_out.data_ptr(), code, _pitch(d_out), rp, T, H, r.K, r.E, r.block_m,
                                           r._slot, r._src, r._blk, wp,
                                           d_rows.data_ptr(), r.rows, None if d_w is None else d_w.data_ptr(),
                                           _stream(stream)), "mm_moe_unpermute_backward")
    return d_rows, d_w


# ------------------------------------------------------------------ 4-bit
def _scale_bytes(rows: int, C: int) -> int:
    return -(-rows // 128) * (2 * -(-C // 256)) * 512


def mx_quantize(x, routing: Optional[Routing] = None, chunks: bool = False, stream=None):
    """Rows x [R, C] into 4 bits: (codes u8 [rows, 16 ceil(C/32)], scales u8).

    Scales are [rows, ceil(C/32)], the layout of the layer's weight scales, or with
    chunks the flat buffer mx_product reads.  With a routing the rows are its pool's,
    every token's row written to its slots (other rows undefined)."""
    code = _rows(x, "mx_quantize", "x")
    R, C = x.shape
    if C < 1:
        _bad("mx_quantize", "x has no columns")
    rows, slot, K = R, None, 1
    if routing is not None:
        _routing_here(routing, "mx_quantize")
        if routing.T != R:
            _bad("mx_quantize", f"x has {R} tokens, the routing {routing.T}")
        rows, slot, K = routing.rows, routing._slot, routing.K
    nb = -(-C // 32)
    codes = _result(stream, (rows, 16 * nb), torch.uint8, x.device)
    sf = _result(stream, _scale_bytes(rows, C) if chunks else (rows, nb), torch.uint8, x.device)
    _check(lib().mm_moe_mx_quantize(x.data_ptr(), code, _pitch(x), R, C, slot, K, rows, codes.data_ptr(),
                                    sf.data_ptr(), chunks, _stream(stream)), "mm_moe_mx_quantize")
    return codes, sf


def mx_dequantize(codes, sf, C: int, dtype=torch.bfloat16, stream=None):
    """The values of codes [R, 16 ceil(C/32)] with scales [R, ceil(C/32)]: [R, C] (bf16
    and fp32 hold them exactly)."""
    nb = -(-C // 32)
    R = codes.shape[0]
    cp = _whole(codes, "mx_dequantize", "codes", (R, 16 * nb), torch.uint8)
    sp = _whole(sf, "mx_dequantize", "sf", (R, nb), torch.uint8)
    if dtype not in _DTYPES:
        _bad("mx_dequantize", f"dtype must be float32, bfloat16 or float16, got {dtype}")
    out = _result(stream, (R, C), dtype, codes.device)
    _check(lib().mm_moe_mx_dequantize(cp, sp, R, C, _DTYPES[dtype], out.data_ptr(), C, _stream(stream)),
           "mm_moe_mx_dequantize")
    return out


def mx_weights(codes, sf, stream=None) -> MxWeights:
    """4-bit matrices codes u8 [E, N, C/2] (or [N, C/2]) with scales u8 [E, N, C/32],
    the scales laid out once for the product.  The codes are used as they are."""
    if codes.dim() == 2 and sf.dim() == 2:
        codes, sf = codes[None], sf[None]
    if codes.dim() != 3 or codes.shape[2] % 16 or codes.numel() == 0:
        _bad("mx_weights", f"codes must be [E, N, C/2] with C a multiple of 32, got {tuple(codes.shape)}")
    E, N, C = codes.shape[0], codes.shape[1], codes.shape[2] * 2
    _whole(codes, "mx_weights", "codes", (E, N, C // 2), torch.uint8)
    sp = _whole(sf, "mx_weights", "sf", (E, N, C // 32), torch.uint8)
    sfp = _result(stream, E * _scale_bytes(N, C), torch.uint8, codes.device)
    _check(lib().mm_moe_mx_prepare(sp, E, N, C, sfp.data_ptr(), _stream(stream)), "mm_moe_mx_prepare")
    return MxWeights(codes, sfp, E, N, C)


def _product_args(what: str, weights: MxWeights, routing: Optional[Routing], rows: int, dtype, device, out,
                  stream):
    """(out, cnt, blk_off) after the checks mx_product and mx_linear share."""
    _here(weights.codes, what, "weights.codes")
    _here(weights.sfp, what, "weights.sfp")
    if routing is None:
        if weights.E != 1:
            _bad(what, f"weights of {weights.E} experts need a routing")
        cnt = blk = None
    else:
        _routing_here(routing, what)
        if routing.block_m != PRODUCT_BLOCK or routing.E != weights.E:
            _bad(what, f"the routing must have blocks of {PRODUCT_BLOCK} and {weights.E} experts, got "
                       f"{routing.block_m} and {routing.E}")
        cnt, blk = routing._cnt, routing._blk
    if out is None:
        out = _result(stream, (rows, weights.N), dtype, device)
    else:
        _rows(out, what, "out", weights.N, dtype)
        if out.shape[0] != rows:
            _bad(what, f"out must have {rows} rows, got {out.shape[0]}")
    return out, cnt, blk


def mx_product(codes, sf, weights: MxWeights, routing: Optional[Routing] = None, out=None, dtype=torch.bfloat16,
               status=None, stream=None):
    """Product of 4-bit rows (mx_quantize with chunks) and weights: [rows, N].

    Dense with one matrix; with a routing (block_m = 128) every expert's rows take
    its matrix and rows of padding are left as they are.  A device wait that runs out
    leaves the result undefined and is reported by sync_status, and in status (int32
    [4] zeroed by the caller) where that is given."""
    rows = codes.shape[0]
    cp = _whole(codes, "mx_product", "codes", (rows, weights.C // 2), torch.uint8)
    sp = _whole(sf, "mx_product", "sf", (_scale_bytes(rows, weights.C),), torch.uint8)
    if dtype not in _DTYPES:
        _bad("mx_product", f"dtype must be float32, bfloat16 or float16, got {dtype}")
    if routing is not None and routing.rows != rows:
        _bad("mx_product", f"codes have {rows} rows, the routing's pool {routing.rows}")
    out, cnt, blk = _product_args("mx_product", weights, routing, rows, dtype, codes.device, out, stream)
    if status is None:
        status = _new(stream, 4, torch.int32, codes.device, zero=True)
    st = _whole(status, "mx_product", "status", (4,), torch.int32)
    _check(lib().mm_moe_mx_product(cp, sp, rows, weights.C, weights.codes.data_ptr(), weights.sfp.data_ptr(), weights.E,
                                   weights.N, cnt, blk, _DTYPES[dtype], out.data_ptr(), _pitch(out), st, 0, 0,
                                   _stream(stream)), "mm_moe_mx_product")
    return out


FEW_TOKENS, FEW_PAIRS, FEW_WORK, FEW_BYTES = 4, 16, 1 << 26, 160 * 1024   # mm_moe_mx_linear_workspace's rule


def mx_linear_workspace(num_rows: int, C: int, device="cuda"):
    """A workspace of mx_linear for num_rows rows (T, or a routing's rows)."""
    return torch.empty(_linear_bytes(num_rows, C), dtype=torch.uint8, device=device)


def _linear_bytes(rows: int, C: int) -> int:
    return (256 + rows * (C // 2) + 255) // 256 * 256 + _scale_bytes(rows, C)


def _few(T: int, C: int, N: int, K: int) -> bool:
    """Whether mx_linear of these sizes needs no workspace (K = 0: dense)."""
    rows = T * K if K else 1 if T < 2 else 2 if T == 2 else 4
    if (rows > FEW_PAIRS) if K else (T > FEW_TOKENS):
        return False
    return rows * N <= FEW_WORK // C and (1 if K else rows) * (C // 32) * 36 <= FEW_BYTES


def mx_linear(x, weights: MxWeights, routing: Optional[Routing] = None, out=None, workspace=None, stream=None):
    """x [T, C] through 4-bit weights: x quantised to 4 bits, then the product, in x's type.

    A few tokens (up to FEW_TOKENS, or FEW_PAIRS routed pairs) run in one launch without
    a workspace.  Dense: [T, N].  With a routing (block_m = 128): [routing.rows, N], every token's
    row through its experts' matrices, rows of padding left as they are.  A device
    wait that runs out leaves the result undefined and is reported by sync_status, and by
    the package's sync_status(workspace) where the workspace is the caller's
    (mx_linear_workspace)."""
    code = _rows(x, "mx_linear", "x", weights.C)
    _no_grad("mx_linear", x)
    T, C = x.shape
    rows, slot, K = T, None, 0
    if routing is not None:
        if routing.T != T:
            _bad("mx_linear", f"x has {T} tokens, the routing {routing.T}")
        rows, slot, K = routing.rows, routing._slot, routing.K
    out, cnt, blk = _product_args("mx_linear", weights, routing, rows, x.dtype, x.device, out, stream)
    ws, ws_bytes = None, 0
    if workspace is not None or not _few(T, C, weights.N, K):
        if workspace is None:
            workspace = _new(stream, _linear_bytes(rows, C), torch.uint8, x.device)
        else:
            _here(workspace, "mx_linear", "workspace")
            if not workspace.is_contiguous():
                _bad("mx_linear", "workspace must be contiguous")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(lib().mm_moe_mx_linear(x.data_ptr(), code, _pitch(x), T, C, weights.codes.data_ptr(),
                                  weights.sfp.data_ptr(), weights.E, weights.N, slot, K, cnt, blk, rows,
                                  out.data_ptr(), _pitch(out), ws, ws_bytes, 0, _stream(stream)), "mm_moe_mx_linear")
    return out


def sync_status(stream=None):
    """Waits for `stream`; (code, where) of the first device wait of a product that ran out on this device since the
    last report, on any stream: MM_MOE_ERR_TIMEOUT and its site, or (0, 0)."""
    return mm_moe_ops_status(_stream(stream))

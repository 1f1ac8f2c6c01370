// C ABI of the operators around the expert layer: argument checks, then the
// launchers of route.cu, rows.cu, mx_quant.cu and mx_linear.cu.
#include "mx_linear.h"
#include "rowtypes.cuh"

using namespace mm;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
// int32 and fp32 arrays; null counts
template <typename... P>
bool words(const P*... p) { return (... && aligned(p, 4)); }

int done(cudaError_t e) { return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ERR_CUDA; }

bool device_ok() { return dev_info().cc_major == 10 && dev_info().cc_minor == 3; }

constexpr int64_t kMaxPairs = int64_t(1) << 30;
constexpr int kMaxCols = 1 << 30;                           // column indices are int32, with room for a granule
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;      // row indices are int32

int check_route(const void* logits, int dtype, int64_t stride, int T, int E, int K, int score) {
  if (T < 0 || E < 1 || E > kMaxE || K < 1 || K > kMaxK || K > E || !dtype_known(dtype)) return MM_MOE_ERR_INVALID_ARG;
  if (score != MM_MOE_SCORE_SOFTMAX && score != MM_MOE_SCORE_SIGMOID) return MM_MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * K > kMaxPairs || stride < E) return MM_MOE_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !aligned(logits, dtype_size(dtype)))) return MM_MOE_ERR_INVALID_ARG;
  return MM_MOE_OK;
}

// the pool of T*K pairs over E experts in blocks of block_m rows fits num_rows
int check_rows(int dtype, int T, int H, int K, int64_t num_rows) {
  if (!dtype_known(dtype) || T < 0 || H < 1 || H > kMaxCols || K < 1 || K > kMaxK || num_rows < 0 || num_rows > kMaxRows)
    return MM_MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * K > kMaxPairs) return MM_MOE_ERR_INVALID_ARG;
  return MM_MOE_OK;
}
int check_pool(int T, int K, int E, int block_m, int64_t num_rows) {
  if (E < 1 || E > kMaxE || K > E || block_m < 16 || block_m > 256 || block_m % 16) return MM_MOE_ERR_INVALID_ARG;
  const int64_t pairs = static_cast<int64_t>(T) * K;
  const int64_t live = pairs < E ? pairs : E;
  return num_rows < pairs + live * (block_m - 1) ? MM_MOE_ERR_INVALID_ARG : MM_MOE_OK;
}

// codes, scales and weights of a product; nothing on the device is touched
int check_product(int64_t rows, int C, const void* w, const void* w_sfp, int E, int N, bool routed, int dtype,
                  const void* out, int64_t out_stride) {
  if (rows < 0 || rows > kMaxRows || C < 32 || C % 32 || N < 1 || E < 1 || E > kMaxE || !dtype_known(dtype))
    return MM_MOE_ERR_INVALID_ARG;
  if ((!routed && E != 1) || (routed && rows % 128)) return MM_MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(E) * N > kMaxRows || C > kMaxCols || out_stride < N) return MM_MOE_ERR_INVALID_ARG;
  if (((rows + 127) / 128) * ((static_cast<int64_t>(N) + 63) / 64) > (int64_t(1) << 30)) return MM_MOE_ERR_INVALID_ARG;
  if (!w || !w_sfp || !aligned(w, 16) || !aligned(w_sfp, 16)) return MM_MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!out || !aligned(out, dtype_size(dtype)))) return MM_MOE_ERR_INVALID_ARG;
  return MM_MOE_OK;
}

uint64_t timeout_ns(unsigned ms) { return static_cast<uint64_t>(ms ? ms : 2000) * 1000000ull; }

struct LinearLayout {
  size_t codes, sf, total;
};
LinearLayout linear_layout(int64_t num_rows, int C) {
  LinearLayout L;
  L.codes = 256;
  L.sf = (L.codes + static_cast<size_t>(num_rows) * (C / 2) + 255) / 256 * 256;
  L.total = L.sf + mx_sf_bytes(num_rows, C);
  return L;
}

}  // namespace

extern "C" {

int mm_moe_route(const void* logits, int dtype, int64_t row_stride, int T, int E, int K, const float* bias, int score,
                 int renorm, float scale, int32_t* topk_idx, float* topk_w, void* stream) {
  if (int r = check_route(logits, dtype, row_stride, T, E, K, score)) return r;
  if (bias && (score != MM_MOE_SCORE_SIGMOID || !words(bias))) return MM_MOE_ERR_INVALID_ARG;
  if (T == 0) return MM_MOE_OK;
  if (!topk_idx || !topk_w || !words(topk_idx, topk_w)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const RouteArgs a{logits, dtype, row_stride, T, E, K, bias, score, renorm != 0, scale, topk_idx, topk_w};
  return done(launch_route(a, static_cast<cudaStream_t>(stream)));
}

int mm_moe_route_backward(const void* logits, int dtype, int64_t row_stride, const int32_t* topk_idx,
                          const float* d_topk_w, int T, int E, int K, int score, int renorm, float scale,
                          void* d_logits, int64_t d_row_stride, void* stream) {
  if (int r = check_route(logits, dtype, row_stride, T, E, K, score)) return r;
  if (d_row_stride < E) return MM_MOE_ERR_INVALID_ARG;
  if (T == 0) return MM_MOE_OK;
  if (!topk_idx || !d_topk_w || !d_logits || !words(topk_idx, d_topk_w) ||
      !aligned(d_logits, dtype_size(dtype)))
    return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const RouteArgs a{logits, dtype, row_stride, T, E, K, nullptr, score, renorm != 0, scale, nullptr, nullptr};
  return done(launch_route_backward(a, topk_idx, d_topk_w, d_logits, d_row_stride, static_cast<cudaStream_t>(stream)));
}

int mm_moe_sort_scratch_size(int T, int K, int E, size_t* bytes) {
  if (!bytes || T < 0 || K < 1 || K > kMaxK || E < 1 || E > kMaxE || K > E) return MM_MOE_ERR_INVALID_ARG;
  const int64_t pairs = static_cast<int64_t>(T) * K;
  if (pairs > kMaxPairs) return MM_MOE_ERR_INVALID_ARG;
  *bytes = sort_in_one_launch(pairs) ? 0 : sizeof(int32_t) * static_cast<size_t>(kDispatchMaxCtas) * E;
  return MM_MOE_OK;
}

int mm_moe_sort(const int32_t* topk_idx, int T, int K, int E, int block_m, int32_t* cnt, int32_t* blk_off,
                int32_t* slot, int32_t* src, int64_t src_capacity, void* scratch, size_t scratch_bytes,
                int32_t* status, void* stream) {
  size_t need = 0;
  if (int r = mm_moe_sort_scratch_size(T, K, E, &need)) return r;
  if (int r = check_pool(T, K, E, block_m, src_capacity)) return r;
  if (!cnt || !blk_off || !status || (T > 0 && (!topk_idx || !slot || !src))) return MM_MOE_ERR_INVALID_ARG;
  if (!words(topk_idx, cnt, blk_off, slot, src, status)) return MM_MOE_ERR_INVALID_ARG;
  if (need && (!scratch || !words(scratch))) return MM_MOE_ERR_INVALID_ARG;
  if (scratch_bytes < need) return MM_MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  return done(launch_sort(topk_idx, T, K, E, block_m, cnt, blk_off, slot, src, status, static_cast<int32_t*>(scratch),
                          static_cast<int64_t>(scratch_bytes / 4), static_cast<cudaStream_t>(stream)));
}

int mm_moe_permute(const void* x, int dtype, int64_t row_stride, int T, int H, int K, int E, int block_m,
                   const int32_t* slot, const int32_t* src, const int32_t* blk_off, void* rows, int64_t num_rows,
                   void* stream) {
  if (int r = check_rows(dtype, T, H, K, num_rows)) return r;
  if (int r = check_pool(T, K, E, block_m, num_rows)) return r;
  if (row_stride < H) return MM_MOE_ERR_INVALID_ARG;
  if (num_rows == 0) return MM_MOE_OK;
  const int es = dtype_size(dtype);
  if (!rows || !src || !blk_off || (T > 0 && (!x || !slot))) return MM_MOE_ERR_INVALID_ARG;
  if (!aligned(x, es) || !aligned(rows, es) || !words(slot, src, blk_off)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const RowsArgs a{dtype, T, H, K, E, block_m, num_rows, slot, src, blk_off};
  return done(launch_permute(a, x, row_stride, rows, static_cast<cudaStream_t>(stream)));
}

int mm_moe_unpermute(const void* rows, int dtype, int64_t num_rows, int T, int H, int K, const int32_t* slot,
                     const float* w, void* out, int64_t out_stride, void* stream) {
  if (int r = check_rows(dtype, T, H, K, num_rows)) return r;
  if (out_stride < H) return MM_MOE_ERR_INVALID_ARG;
  if (T == 0) return MM_MOE_OK;
  const int es = dtype_size(dtype);
  if (!rows || !slot || !out || !aligned(rows, es) || !aligned(out, es) || !words(slot, w)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const RowsArgs a{dtype, T, H, K, 0, 0, num_rows, slot, nullptr, nullptr};
  return done(launch_unpermute(a, rows, w, out, out_stride, static_cast<cudaStream_t>(stream)));
}

int mm_moe_unpermute_backward(const void* d_out, int dtype, int64_t d_stride, const void* rows, int T, int H, int K,
                              int E, int block_m, const int32_t* slot, const int32_t* src, const int32_t* blk_off,
                              const float* w, void* d_rows, int64_t num_rows, float* d_w, void* stream) {
  if (int r = check_rows(dtype, T, H, K, num_rows)) return r;
  if (int r = check_pool(T, K, E, block_m, num_rows)) return r;
  if (d_stride < H) return MM_MOE_ERR_INVALID_ARG;
  if (num_rows == 0) return MM_MOE_OK;
  const int es = dtype_size(dtype);
  if (!d_rows || !src || !blk_off || (T > 0 && (!d_out || !slot)) || (T > 0 && d_w && !rows))
    return MM_MOE_ERR_INVALID_ARG;
  if (!aligned(d_out, es) || !aligned(d_rows, es) || !aligned(rows, es) || !words(slot, src, blk_off, w, d_w))
    return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const RowsArgs a{dtype, T, H, K, E, block_m, num_rows, slot, src, blk_off};
  return done(launch_unpermute_backward(a, d_out, d_stride, rows, w, d_rows, d_w, static_cast<cudaStream_t>(stream)));
}

int mm_moe_mx_scale_size(int64_t rows, int C, size_t* bytes) {
  if (!bytes || rows < 0 || rows > kMaxRows || C < 1 || C > kMaxCols) return MM_MOE_ERR_INVALID_ARG;
  *bytes = mx_sf_bytes(rows, C);
  return MM_MOE_OK;
}

int mm_moe_mx_quantize(const void* x, int dtype, int64_t row_stride, int64_t R, int C, const int32_t* slot, int K,
                       int64_t num_rows, void* codes, void* sf, int chunks, void* stream) {
  if (!dtype_known(dtype) || R < 0 || R > kMaxRows || C < 1 || C > kMaxCols || row_stride < C)
    return MM_MOE_ERR_INVALID_ARG;
  if (slot && (!words(slot) || K < 1 || K > kMaxK || num_rows < 0 || num_rows > kMaxRows || R * K > kMaxPairs))
    return MM_MOE_ERR_INVALID_ARG;
  if (R == 0) return MM_MOE_OK;
  if (!x || !codes || !sf || !aligned(x, dtype_size(dtype)) || !aligned(codes, 16) || (chunks && !aligned(sf, 16)))
    return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const MxQuantArgs a{x, dtype, row_stride, R, C, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(sf), chunks != 0,
                      slot, K, num_rows, nullptr};
  return done(launch_mx_quantize(a, static_cast<cudaStream_t>(stream)));
}

int mm_moe_mx_dequantize(const void* codes, const void* sf, int64_t R, int C, int dtype, void* out, int64_t out_stride,
                         void* stream) {
  if (!dtype_known(dtype) || R < 0 || R > kMaxRows || C < 1 || C > kMaxCols || out_stride < C)
    return MM_MOE_ERR_INVALID_ARG;
  if (R == 0) return MM_MOE_OK;
  if (!codes || !sf || !out || !aligned(codes, 16) || !aligned(out, dtype_size(dtype))) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  return done(launch_mx_dequantize(static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(sf), R, C, dtype,
                                   out, out_stride, static_cast<cudaStream_t>(stream)));
}

int mm_moe_mx_prepare(const void* sf, int E, int N, int C, void* sfp, void* stream) {
  if (!sf || !sfp || !aligned(sfp, 16) || E < 1 || E > kMaxE || N < 1 || C < 1 || C > kMaxCols ||
      static_cast<int64_t>(E) * N > kMaxRows)
    return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  return done(launch_mx_prepare(static_cast<const uint8_t*>(sf), E, N, C, static_cast<uint8_t*>(sfp),
                                static_cast<cudaStream_t>(stream)));
}

int mm_moe_mx_product(const void* codes, const void* sf, int64_t rows, int C, const void* w, const void* w_sfp, int E,
                      int N, const int32_t* cnt, const int32_t* blk_off, int dtype, void* out, int64_t out_stride,
                      int32_t* status, unsigned timeout_ms, int debug_flags, void* stream) {
  if (!cnt != !blk_off) return MM_MOE_ERR_INVALID_ARG;
  if (int r = check_product(rows, C, w, w_sfp, E, N, blk_off != nullptr, dtype, out, out_stride)) return r;
  if (rows == 0) return MM_MOE_OK;
  if (!codes || !sf || !status || !aligned(codes, 16) || !aligned(sf, 16) || !words(status, cnt, blk_off))
    return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const MxProductArgs a{static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(sf), rows, C,
                        static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(w_sfp), E, N, cnt, blk_off, dtype,
                        out, out_stride, status, timeout_ns(timeout_ms), false, (debug_flags & 1) != 0};
  return done(launch_mx_product(a, static_cast<cudaStream_t>(stream)));
}

int mm_moe_mx_linear_workspace(int T, int C, int N, int K, int64_t num_rows, size_t* bytes) {
  if (!bytes || T < 0 || N < 1 || K < 0 || K > kMaxK || num_rows < 0 || num_rows > kMaxRows || C < 32 || C % 32 || C > kMaxCols)
    return MM_MOE_ERR_INVALID_ARG;
  if (K == 0 && num_rows != T) return MM_MOE_ERR_INVALID_ARG;
  *bytes = mx_few_rows(T, C, N, K) ? 0 : linear_layout(num_rows, C).total;
  return MM_MOE_OK;
}

int mm_moe_mx_linear(const void* x, int dtype, int64_t row_stride, int T, int C, const void* w, const void* w_sfp,
                     int E, int N, const int32_t* slot, int K, const int32_t* cnt, const int32_t* blk_off,
                     int64_t num_rows, void* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
                     unsigned timeout_ms, void* stream) {
  const bool routed = slot != nullptr;
  if (T < 0 || row_stride < C || !cnt != !slot || !blk_off != !slot || (!routed && num_rows != T) ||
      !words(slot, cnt, blk_off))
    return MM_MOE_ERR_INVALID_ARG;
  if (int r = check_product(num_rows, C, w, w_sfp, E, N, routed, dtype, out, out_stride)) return r;
  if (routed) {
    if (K < 1 || K > kMaxK || static_cast<int64_t>(T) * K > kMaxPairs) return MM_MOE_ERR_INVALID_ARG;
    if (int r = check_pool(T, K, E, 128, num_rows)) return r;
  }
  const LinearLayout L = linear_layout(num_rows, C);
  const bool few = mx_few_rows(T, C, N, routed ? K : 0);
  if ((!few && !workspace) || !aligned(workspace, 256)) return MM_MOE_ERR_INVALID_ARG;
  if (workspace_bytes < (few ? (workspace ? 16 : 0) : L.total)) return MM_MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)   // nothing to compute; leave a clean status word for mm_moe_sync_status
    return workspace ? done(cudaMemsetAsync(workspace, 0, 16, s)) : MM_MOE_OK;
  if (!x || !aligned(x, dtype_size(dtype))) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  const MxQuantArgs q{x, dtype, row_stride, T, C, ws + L.codes, ws + L.sf, 1, slot, K, num_rows, status};
  const MxProductArgs p{ws + L.codes, ws + L.sf, num_rows, C, static_cast<const uint8_t*>(w),
                        static_cast<const uint8_t*>(w_sfp), E, N, cnt, blk_off, dtype, out, out_stride, status,
                        timeout_ns(timeout_ms), true, false};
  if (few) return done(launch_mx_few(q, p, s));
  cudaError_t e = launch_mx_quantize(q, s);
  if (e != cudaSuccess) return done(e);
  return done(launch_mx_product(p, s));
}

int mm_moe_ops_status(void* stream, int* where) {
  if (where) *where = 0;
  int32_t* record = nullptr;
  if (mx_report(&record) != cudaSuccess) return MM_MOE_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t h[4] = {0, 0, 0, 0};
  if (cudaMemcpyAsync(h, record, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return MM_MOE_ERR_CUDA;
  if (h[0] == 0) return MM_MOE_OK;
  if (cudaMemsetAsync(record, 0, sizeof(h), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return MM_MOE_ERR_CUDA;
  if (where) *where = h[1];
  return h[0];
}

}  // extern "C"

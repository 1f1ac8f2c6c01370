// C ABI of the operators on rows in 8 bits: argument checks, then the launchers of
// quant8.cu, norm.cu, swiglu.cu and weight_grad.cu.
#include "internal.h"
#include "rowtypes.cuh"

using namespace mm;

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
template <typename... P>
bool words(const P*... p) { return (... && aligned(p, 4)); }
int done(cudaError_t e) { return e == cudaSuccess ? MM_MOE_OK : MM_MOE_ERR_CUDA; }
bool device_ok() { return dev_info().cc_major == 10 && dev_info().cc_minor == 3; }

constexpr int64_t kMaxPairs = int64_t(1) << 30;
constexpr int kMaxCols = 1 << 30;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 256;

bool variant_known(int v) { return v == MM_MOE_VARIANT_MX || v == MM_MOE_VARIANT_F8; }
bool rows_known(int dtype, int64_t rows, int cols) {
  return dtype_known(dtype) && rows >= 0 && rows <= kMaxRows && cols >= 1 && cols <= kMaxCols;
}
// rows of one sum of a weight gradient: all (E = 0: dense), or an expert's on average
int64_t terms_of(int64_t rows, int T, int K, int E) { return E ? static_cast<int64_t>(T) * K / E : rows; }
// and at most: one expert may take every pair
int64_t longest_of(int64_t rows, int T, int K, int E) { return E ? static_cast<int64_t>(T) * K : rows; }
// codes and scales of rows, both or neither
bool held_ok(const void* codes, const void* sf, int variant) {
  if (!codes || !sf) return !codes && !sf;
  return variant_known(variant) && aligned(codes, 16) && (variant == MM_MOE_VARIANT_MX || words(sf));
}

// A routing's arrays, all or none; the pool of T*K pairs over E experts fits `rows`.
int check_routing(int64_t rows, int T, int K, int E, int block_m, const int32_t* slot, const int32_t* src,
                  const int32_t* blk_off) {
  if (!slot != !src || !slot != !blk_off) return MM_MOE_ERR_INVALID_ARG;
  if (!slot) return MM_MOE_OK;
  if (!words(slot, src, blk_off) || T < 0 || K < 1 || K > kMaxK || E < 1 || E > kMaxE || K > E || block_m < 16 ||
      block_m > 256 || block_m % 16)
    return MM_MOE_ERR_INVALID_ARG;
  const int64_t pairs = static_cast<int64_t>(T) * K;
  if (pairs > kMaxPairs || rows < pairs + (pairs < E ? pairs : E) * (block_m - 1)) return MM_MOE_ERR_INVALID_ARG;
  return MM_MOE_OK;
}

}  // namespace

extern "C" {

int mm_moe_rows_quantize(const void* x, int dtype, int64_t row_stride, int64_t R, int C, int variant, void* codes,
                         void* sf, void* stream) {
  if (!rows_known(dtype, R, C) || row_stride < C || !variant_known(variant)) return MM_MOE_ERR_INVALID_ARG;
  if (R == 0) return MM_MOE_OK;
  if (!x || !codes || !aligned(x, dtype_size(dtype)) || !held_ok(codes, sf, variant)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  return done(launch_quantize8(x, dtype, row_stride, R, C, variant, codes, sf, static_cast<cudaStream_t>(stream)));
}

int mm_moe_rows_dequantize(const void* codes, const void* sf, int64_t R, int C, int variant, int dtype, void* out,
                           int64_t out_stride, void* stream) {
  if (!rows_known(dtype, R, C) || out_stride < C || !variant_known(variant)) return MM_MOE_ERR_INVALID_ARG;
  if (R == 0) return MM_MOE_OK;
  if (!out || !codes || !aligned(out, dtype_size(dtype)) || !held_ok(codes, sf, variant)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  return done(launch_dequantize8(codes, sf, R, C, variant, dtype, out, out_stride, static_cast<cudaStream_t>(stream)));
}

int mm_moe_rms_norm(const void* x, int dtype, int64_t x_stride, const void* residual, int64_t residual_stride,
                    const void* weight, int weight_dtype, int64_t T, int H, float eps, void* h, void* y, int variant,
                    void* codes, void* sf, float* rstd, void* stream) {
  if (!rows_known(dtype, T, H) || x_stride < H || (weight_dtype != dtype && weight_dtype != MM_MOE_DTYPE_F32) ||
      !(eps >= 0.f) || (residual && residual_stride < H) || !residual != !h || !held_ok(codes, sf, variant))
    return MM_MOE_ERR_INVALID_ARG;
  if (T == 0) return MM_MOE_OK;
  const size_t es = dtype_size(dtype);
  if (!x || !weight || !rstd || !aligned(x, es) || !aligned(residual, es) || !aligned(h, es) || !aligned(y, es) ||
      !aligned(weight, dtype_size(weight_dtype)) || !words(rstd))
    return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const NormLaunch n{x, dtype, x_stride, residual, residual_stride, weight, weight_dtype, T, H, eps, h, y, variant,
                     codes, sf, rstd};
  return done(launch_rms_norm(n, static_cast<cudaStream_t>(stream)));
}

int mm_moe_rms_norm_scratch_size(int64_t T, int H, size_t* bytes) {
  if (!bytes || T < 0 || T > kMaxRows || H < 1 || H > kMaxCols) return MM_MOE_ERR_INVALID_ARG;
  *bytes = norm_scratch_bytes(T, H);
  return MM_MOE_OK;
}

int mm_moe_rms_norm_backward(const void* d_y, int dtype, int64_t d_y_stride, const void* h, int64_t h_stride,
                             const void* weight, int weight_dtype, const float* rstd, const void* d_h,
                             int64_t d_h_stride, int64_t T, int H, void* d_x, float* d_weight, void* scratch,
                             size_t scratch_bytes, void* stream) {
  if (!rows_known(dtype, T, H) || d_y_stride < H || h_stride < H || (d_h && d_h_stride < H) ||
      (weight_dtype != dtype && weight_dtype != MM_MOE_DTYPE_F32) || !d_weight || !words(d_weight))
    return MM_MOE_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  if (T > 0) {
    if (!d_y || !h || !weight || !rstd || !d_x || !scratch || !aligned(d_y, es) || !aligned(h, es) ||
        !aligned(d_h, es) || !aligned(d_x, es) || !aligned(weight, dtype_size(weight_dtype)) || !words(rstd) ||
        !aligned(scratch, 16))
      return MM_MOE_ERR_INVALID_ARG;
    if (scratch_bytes < norm_scratch_bytes(T, H)) return MM_MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const NormBackLaunch n{d_y, dtype, d_y_stride, h, h_stride, weight, weight_dtype, rstd, d_h, d_h_stride, T, H, d_x,
                         d_weight, scratch};
  return done(launch_rms_norm_backward(n, static_cast<cudaStream_t>(stream)));
}

int mm_moe_swiglu(const void* h, int dtype, int64_t h_stride, int64_t rows, int I, int T, int K, int E, int block_m,
                  const int32_t* slot, const int32_t* src, const int32_t* blk_off, const float* w, void* a,
                  void* codes, void* sf, void* kept, void* kept_sf, void* stream) {
  if (!rows_known(dtype, rows, I) || I > kMaxCols / 2 || h_stride < 2 * static_cast<int64_t>(I) || (w && !slot) ||
      !held_ok(codes, sf, MM_MOE_VARIANT_MX) || !held_ok(kept, kept_sf, MM_MOE_VARIANT_MX))
    return MM_MOE_ERR_INVALID_ARG;
  if (int r = check_routing(rows, T, K, E, block_m, slot, src, blk_off)) return r;
  if (rows == 0) return MM_MOE_OK;
  const size_t es = dtype_size(dtype);
  if (!h || !aligned(h, es) || !aligned(a, es) || !words(w) || (!a && !codes && !kept)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const SwigluRows r{rows, I, slot, src, blk_off, E, block_m, static_cast<int64_t>(T) * K};
  return done(launch_swiglu(r, dtype, h, h_stride, w, a, codes, sf, kept, kept_sf, static_cast<cudaStream_t>(stream)));
}

int mm_moe_swiglu_backward(const void* d_a, int dtype, int64_t d_stride, const void* kept, const void* kept_sf,
                           int64_t rows, int I, int T, int K, int E, int block_m, const int32_t* slot,
                           const int32_t* src, const int32_t* blk_off, const float* w, void* d_h, float* d_w,
                           void* stream) {
  if (!rows_known(dtype, rows, I) || I > kMaxCols / 2 || d_stride < I || (w && !slot) || (d_w && !slot) ||
      !held_ok(kept, kept_sf, MM_MOE_VARIANT_MX))
    return MM_MOE_ERR_INVALID_ARG;
  if (int r = check_routing(rows, T, K, E, block_m, slot, src, blk_off)) return r;
  if (rows == 0) return MM_MOE_OK;
  const size_t es = dtype_size(dtype);
  if (!d_a || !kept || !d_h || !aligned(d_a, es) || !aligned(d_h, es) || !words(w, d_w)) return MM_MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  const SwigluRows r{rows, I, slot, src, blk_off, E, block_m, static_cast<int64_t>(T) * K};
  return done(launch_swiglu_backward(r, dtype, d_a, d_stride, kept, kept_sf, w, d_h, d_w,
                                     static_cast<cudaStream_t>(stream)));
}

int mm_moe_weight_grad_scratch_size(const void* d_y, int64_t d_stride, int64_t rows, int N, const void* sf, int C,
                                    int T, int K, int E, int by_token, size_t* bytes) {
  if (!bytes || rows < 0 || rows > kMaxRows || N < 1 || N > kMaxCols || d_stride < N || C < 1 || C > kMaxCols || T < 0 ||
      K < 0 || K > kMaxK || E < 0 || E > kMaxE || !K != !E || (by_token && !E))
    return MM_MOE_ERR_INVALID_ARG;
  *bytes = weight_grad_scratch_bytes(d_y, d_stride, rows, N, sf, C, by_token != 0, E ? E : 1, terms_of(rows, T, K, E),
                                     longest_of(rows, T, K, E));
  return MM_MOE_OK;
}

int mm_moe_weight_grad(const void* d_y, int64_t d_stride, int64_t rows, int N, const void* codes, const void* sf, int C,
                       int T, int K, int E, int block_m, const int32_t* cnt, const int32_t* src,
                       const int32_t* blk_off, int by_token, int dtype, void* out, void* scratch, size_t scratch_bytes,
                       unsigned timeout_ms, int debug_flags, void* stream) {
  if (rows < 0 || rows > kMaxRows || N < 1 || N > kMaxCols || C < 1 || C > kMaxCols || d_stride < N ||
      (dtype != MM_MOE_DTYPE_F32 && dtype != MM_MOE_DTYPE_BF16) || !cnt != !src || (by_token && !cnt))
    return MM_MOE_ERR_INVALID_ARG;
  if (int r = check_routing(rows, T, K, cnt ? E : 1, block_m, cnt, src, blk_off)) return r;
  if (!cnt) E = 1;
  if (static_cast<int64_t>(E) * N > kMaxRows || weight_grad_tasks(E, N, C) > (int64_t(1) << 30))
    return MM_MOE_ERR_INVALID_ARG;
  if (!out || !aligned(out, dtype_size(dtype))) return MM_MOE_ERR_INVALID_ARG;
  if (rows > 0 && !(cnt && T == 0) && (!d_y || !codes || !aligned(d_y, 2) || !held_ok(codes, sf, MM_MOE_VARIANT_MX)))
    return MM_MOE_ERR_INVALID_ARG;
  const int64_t terms = terms_of(rows, T, K, cnt ? E : 0), longest = longest_of(rows, T, K, cnt ? E : 0);
  const size_t need = weight_grad_scratch_bytes(d_y, d_stride, rows, N, sf, C, by_token != 0, E, terms, longest);
  if (need && (!scratch || !aligned(scratch, 32))) return MM_MOE_ERR_INVALID_ARG;
  if (scratch_bytes < need) return MM_MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!device_ok()) return MM_MOE_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0 || (cnt && T == 0))            // sums of nothing
    return done(cudaMemsetAsync(out, 0, static_cast<size_t>(E) * N * C * dtype_size(dtype), s));
  const WeightGradLaunch p{d_y, d_stride, rows, N, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(sf),
                           C, cnt, blk_off, src, by_token != 0, K, E, block_m,
                           terms, longest, dtype, out, scratch,
                           static_cast<uint64_t>(timeout_ms ? timeout_ms : 2000) * 1000000ull, (debug_flags & 1) != 0};
  return done(launch_weight_grad(p, s));
}

}  // extern "C"

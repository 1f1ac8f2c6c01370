// Declarations of the 4-bit quantiser and product (mx_quant.cu, mx_linear.cu).
#pragma once

#include "internal.h"

namespace mm {

// 128-wide scale chunks along a contraction of C elements; an even number, so
// that the two chunks of a 256-wide stage are always there.
__host__ __device__ __forceinline__ int mx_chunks(int C) { return (C + 255) / 256 * 2; }

// Byte offset of the 4-byte scale word of row r and 128-wide chunk kb, in a
// region laid out [128-row block][KB chunks][512]: the order one
// tcgen05.cp.32x128b.warpx4 reads (16-byte line r % 32, word (r % 128) / 32).
__host__ __device__ __forceinline__ size_t mx_sf_word(int64_t r, int kb, int KB) {
  return (static_cast<size_t>(r >> 7) * KB + kb) * kSFChunk + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

inline size_t mx_sf_bytes(int64_t rows, int C) {
  return static_cast<size_t>((rows + 127) / 128) * mx_chunks(C) * kSFChunk;
}

struct MxQuantArgs {
  const void* x;
  int dtype;
  int64_t stride;            // elements between rows of x
  int64_t R;
  int C;
  uint8_t* codes;            // [rows, ceil(C / 32) * 16 bytes]
  uint8_t* sf;               // [rows, ceil(C / 32)], or chunks
  int chunks;
  const int32_t* slot;       // row r goes to rows slot[r * K + k] (null: to row r)
  int K;
  int64_t num_rows;
  int32_t* status;           // four words to clear, or null
};
cudaError_t launch_mx_quantize(const MxQuantArgs& a, cudaStream_t s);
cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* sf, int64_t R, int C, int dtype, void* out,
                                 int64_t out_stride, cudaStream_t s);
cudaError_t launch_mx_prepare(const uint8_t* sf, int E, int N, int C, uint8_t* out, cudaStream_t s);

struct MxProductArgs {
  const uint8_t* codes;      // activations [rows, C / 2], scales in chunks
  const uint8_t* sf;
  int64_t rows;              // rows of `codes` and `out`
  int C;                     // contraction, a multiple of 32
  const uint8_t* w;          // [E, N, C / 2] and its prepared scales
  const uint8_t* w_sf;
  int E, N;
  const int32_t* cnt;        // per expert: rows and first 128-row block (null: one expert, all rows)
  const int32_t* blk_off;
  int dtype;                 // of out
  void* out;
  int64_t out_stride;
  int32_t* status;
  uint64_t timeout_ns;
  bool after_quantize;       // launched programmatically behind the quantiser
  bool unreachable;          // the last stage of each CTA's last task is never loaded (a test of the bounded waits)
  int32_t* report = nullptr; // mx_report's record, filled in by launch_mx_product
};
// Device address of the current device's record of waits that ran out in any product: four words, zero until one did.
cudaError_t mx_report(int32_t** record);
cudaError_t launch_mx_product(const MxProductArgs& a, cudaStream_t s);
// on CTA pairs: two 128-row blocks a task
cudaError_t launch_mx_product_pair(const MxProductArgs& a, cudaStream_t s);

// Both steps of a linear in one launch for a few rows (mx_few.cu).
constexpr int kMxFewTokens = 4;      // rows of a dense linear
constexpr int kMxFewPairs = 16;      // (token, k) pairs of a routed one
constexpr int64_t kMxFewWork = int64_t(1) << 26;   // rows * N * C
constexpr int kMxFewSmem = 160 * 1024;
bool mx_few_rows(int T, int C, int N, int K);   // K = 0: dense
cudaError_t launch_mx_few(const MxQuantArgs& q, const MxProductArgs& p, cudaStream_t s);

}  // namespace mm

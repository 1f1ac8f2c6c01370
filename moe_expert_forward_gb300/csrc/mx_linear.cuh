// Device pieces shared by the 4-bit products (mx_linear.cu, mx_linear_pair.cu).
#pragma once

#include "mx_linear.h"
#include "ptx.cuh"
#include "rowtypes.cuh"

namespace mm {

constexpr int kMxRows = 128;                     // rows of a block
constexpr int kMxStageK = 256;                   // contraction elements per stage
constexpr int kMxStageBytes = kMxStageK / 2;     // of one row's codes: one 128-byte swizzle atom
constexpr int kMxTileBytes = kMxRows * kMxStageBytes;
constexpr int kMxSfBytes = 2 * kSFChunk;         // the two scale chunks of 128 rows and one stage

struct MxArgs {
  int rows, C, E, N;
  int KS, KB;                // 256-wide stages, scale chunks along the contraction
  int NB, NT;                // 128-row scale blocks and weight tiles of one expert
  int nblk;                  // row blocks of a dense product
  const uint8_t* sf;
  const uint8_t* w_sf;
  const int* cnt;
  const int* blk_off;
  char* out;
  int64_t out_pitch;         // bytes
  int lines;                 // out and its rows are 32-byte aligned
  int wait_prior;            // launched programmatically: activations come from the kernel before
  int unreachable;           // leave the last stage of the CTA's last task out
  int* status;
  int* report;
  uint64_t timeout_ns;
};

// Instruction descriptor of kind::mxf4: A and B e2m1 (1) in [9:7] and [11:10],
// both K-major, N >> 3 in [22:17], UE8M0 scales (bit 23), M >> 7 in [28:27];
// the scale bytes a 64-wide MMA takes from each 32-bit word: 0 (bytes 0, 1) or 2
// (bytes 2, 3) in [30:29] for A and [5:4] for B.
__host__ __device__ constexpr uint32_t idesc_mxf4(int n, int m, int half) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 7) << 27) | (static_cast<uint32_t>(2 * half) << 29) |
         (static_cast<uint32_t>(2 * half) << 4);
}

// The last i < n with a[i] <= v; a[0] <= v.
__device__ __forceinline__ int last_not_above(const int* a, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// mbar_wait by a whole warp, of one answer for all of its lanes: each lane's own may differ where an abort or the limit
// meets the barrier's completion, and what follows (loads from tensor memory, shuffles) takes all lanes or none.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, const Status& st, volatile int* abort,
                                               int where) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, st, abort, where));
}

// mbar_wait_drain, and on its limit the CTA's flag raised.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity, const Status& st, volatile int* abort,
                                           int where) {
  if (!mbar_wait_drain(bar, parity, st, where)) *abort = 1;
}

// One thread of a CTA at its end: a wait that ran out goes into the library's record too, which is there to be read
// when the call's own status word no longer is. The first one stays.
__device__ __forceinline__ void note_given_up(const MxArgs& a, volatile int* abort) {
  if (*abort && atomicCAS(a.report, 0, MM_MOE_ERR_TIMEOUT) == 0) a.report[1] = *(volatile int*)(a.status + 1);
}

// Two accumulators as one 32-bit word of 16-bit elements.
template <typename T>
__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b) {
  Vec<T, 2> h;
  h.v[0] = from_float<T>(__uint_as_float(a));
  h.v[1] = from_float<T>(__uint_as_float(b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Exchanges 32-byte pieces among each 4 lanes: lane j's piece i becomes piece j of what lane i held.
__device__ __forceinline__ void transpose4(uint32_t (&w)[32], int lane) {
#pragma unroll
  for (int step = 1; step <= 2; step *= 2) {
    const bool up = (lane & step) != 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & step) continue;                    // pieces i and i + step change places with lane ^ step
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t& lo = w[8 * i + c];
        uint32_t& hi = w[8 * (i + step) + c];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, step);
        if (up) lo = got; else hi = got;
      }
    }
  }
}

// Word i of lane j becomes word j of lane i.
__device__ __forceinline__ void transpose32(uint32_t (&w)[32], int lane) {
#pragma unroll
  for (int step = 1; step <= 16; step *= 2) {
    const bool up = (lane & step) != 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i & step) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + step], step);
      if (up) w[i] = got; else w[i + step] = got;
    }
  }
}

// A warp's 32 rows of accumulator columns [col, col + kCols) of TMEM, lane = row, stored from `out` on (row 0, first
// column) `pitch` bytes a row: the first `rows` rows and the first `cols` columns. `release` is called as soon as the
// accumulator has been read: with kLines 16-bit results are packed into registers first and stored after it, others are
// stored 32 or 64 columns at a time and it follows the last read.
//
// kLines: `out` and its rows are 32-byte aligned. 16-bit results change lanes so that an instruction stores whole
// 128-byte lines of 8 rows instead of 32 bytes of 32 rows (8192x7168x4096: 87 us, 90 without).
// Otherwise the warp transposes 32 words and stores one row at a time, consecutive lanes consecutive words, as words
// where rows are 4-byte aligned (8192x4096x4095 bf16: 309 us with a row per lane).
template <typename T, int kCols, bool kLines, typename F>
__device__ __forceinline__ void store_accumulator(uint32_t col, char* out, int64_t pitch, int rows, int cols,
                                                  int lane, F release) {
  // 64 columns as 32 words of two 16-bit elements
  auto load64 = [&](int c, uint32_t (&w)[32]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(col + c + 32 * h, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) w[16 * h + i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
  };
  if constexpr (sizeof(T) == 2 && kLines) {
    uint32_t w[kCols / 64][32];
#pragma unroll
    for (int h = 0; h < kCols / 64; ++h) load64(64 * h, w[h]);
    release();
    T* p = reinterpret_cast<T*>(out + lane * pitch);
#pragma unroll
    for (int h = 0; h < kCols / 64; ++h) {
      if (cols >= 64 * (h + 1)) {
        transpose4(w[h], lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (lane & ~3) + i;
          if (r < rows)
            st_global_v8(reinterpret_cast<float*>(out + r * pitch + h * 128 + (lane & 3) * 32), w[h] + 8 * i);
        }
      } else if (lane < rows) {                  // the last columns: 32 bytes of a row, then element by element
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          if (cols >= 64 * h + c + 16) {
            st_global_v8(reinterpret_cast<float*>(p + 64 * h + c), w[h] + c / 2);
          } else {
#pragma unroll
            for (int i = c / 2; i < c / 2 + 8; ++i) {
              const Vec<T, 2> e = *reinterpret_cast<const Vec<T, 2>*>(&w[h][i]);
              if (64 * h + 2 * i < cols) p[64 * h + 2 * i] = e.v[0];
              if (64 * h + 2 * i + 1 < cols) p[64 * h + 2 * i + 1] = e.v[1];
            }
          }
        }
      }
    }
  } else if constexpr (sizeof(T) == 2) {
    const bool words = ((reinterpret_cast<uintptr_t>(out) | static_cast<uintptr_t>(pitch)) & 3) == 0;
#pragma unroll 1
    for (int c = 0; c < kCols; c += 64) {
      uint32_t w[32];
      load64(c, w);
      if (c + 64 == kCols) release();
      if (cols <= c) continue;
      transpose32(w, lane);
      const int left = cols - c - 2 * lane;      // columns from this lane's two on
      char* q = out + (c + 2 * lane) * 2;
      if (words && left >= 2) {
#pragma unroll
        for (int r = 0; r < 32; ++r, q += pitch)
          if (r < rows) *reinterpret_cast<uint32_t*>(q) = w[r];
      } else if (left >= 1) {
#pragma unroll
        for (int r = 0; r < 32; ++r, q += pitch)
          if (r < rows) {
            const Vec<T, 2> e = *reinterpret_cast<const Vec<T, 2>*>(&w[r]);
            reinterpret_cast<T*>(q)[0] = e.v[0];
            if (left >= 2) reinterpret_cast<T*>(q)[1] = e.v[1];
          }
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < kCols; c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(col + c, v);
      tmem_ld_wait();
      if (c + 32 == kCols) release();
      if (kLines && cols >= c + 32) {
        if (lane < rows) {
          float* p = reinterpret_cast<float*>(out + lane * pitch) + c;
#pragma unroll
          for (int i = 0; i < 32; i += 8) st_global_v8(p + i, v + i);
        }
      } else if (cols > c) {
        transpose32(v, lane);
        char* q = out + (c + lane) * 4;
        if (c + lane < cols) {
#pragma unroll
          for (int r = 0; r < 32; ++r, q += pitch)
            if (r < rows) *reinterpret_cast<uint32_t*>(q) = v[r];
        }
      }
    }
  }
}

// Arguments and tensor maps that do not depend on the kernel's tiles.
inline MxArgs mx_args(const MxProductArgs& p, int elem, int tile_n) {
  MxArgs a{};
  a.rows = static_cast<int>(p.rows);
  a.C = p.C; a.E = p.E; a.N = p.N;
  a.KB = mx_chunks(p.C); a.KS = a.KB / 2;
  a.NB = (p.N + 127) / 128; a.NT = (p.N + tile_n - 1) / tile_n;
  a.nblk = static_cast<int>((p.rows + kMxRows - 1) / kMxRows);
  a.sf = p.sf; a.w_sf = p.w_sf; a.cnt = p.cnt; a.blk_off = p.blk_off;
  a.out = static_cast<char*>(p.out);
  a.out_pitch = p.out_stride * static_cast<int64_t>(elem);
  a.lines = (reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(a.out_pitch)) % 32 == 0;
  a.wait_prior = p.after_quantize;
  a.unreachable = p.unreachable;
  a.status = p.status; a.report = p.report; a.timeout_ns = p.timeout_ns;
  return a;
}
// codes of `rows` rows as [rows, C/2] bytes in boxes of one stage x box_rows
inline CUresult mx_codes_map(CUtensorMap* m, const void* codes, int64_t rows, int C, int box_rows) {
  const uint64_t pitch = static_cast<uint64_t>(C) / 2;
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, pitch, static_cast<uint64_t>(rows), pitch,
                        kMxStageBytes, static_cast<uint32_t>(box_rows), CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace mm

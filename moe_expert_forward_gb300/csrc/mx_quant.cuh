// The 4-bit rule on 16 elements of a row (mx_quant.cu, mx_few.cu): amax, scale
// exponent and codes of e2m1 blocks of 32.
#pragma once

#include <cstring>
#include <type_traits>

#include "mx_linear.h"
#include "ptx.cuh"
#include "rowtypes.cuh"

namespace mm {

// 8 fp32 values -> 8 e2m1 codes, value 0 in the lowest nibble
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Bits of |x| of the largest element -> the block's exponent e; finite input only.
// amax = m * 2^ex, m in [0.5, 1); 6 = 0.75 * 2^3, so e = ex - 3 when m <= 0.75, else ex - 2.
// amax >= 1e-10 keeps e >= -36, and amax < 2^128 keeps e <= 126.
__device__ __forceinline__ int e2m1_exponent(uint32_t amax_bits) {
  const uint32_t b = max(amax_bits, __float_as_uint(1e-10f));
  return static_cast<int>(b >> 23) - 126 - 3 + ((b & 0x7FFFFF) > 0x400000 ? 1 : 0);
}

// Sixteen consecutive elements of a row as they sit in memory.
template <typename T>
struct Group {
  static constexpr int kWords = 16 * sizeof(T) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // elements c .. c+15 of `row`, zeros past C
  template <bool kVec>
  __device__ __forceinline__ void load(const T* __restrict__ row, int c, int C) {
    if (kVec) {                       // C is a multiple of 16, rows 32-byte aligned
      if (c < C) {
#pragma unroll
        for (int h = 0; h < kWords / 8; ++h)
          asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                       : "=r"(w[8 * h]), "=r"(w[8 * h + 1]), "=r"(w[8 * h + 2]), "=r"(w[8 * h + 3]),
                         "=r"(w[8 * h + 4]), "=r"(w[8 * h + 5]), "=r"(w[8 * h + 6]), "=r"(w[8 * h + 7])
                       : "l"(row + c + h * (32 / sizeof(T))));
      } else {
        clear();
      }
    } else {
      constexpr int N = 16 / sizeof(T);
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const int n = C - (c + h * N);               // elements from here on
        uint4 q = make_uint4(0, 0, 0, 0);
        if (n > 0) q = load16_any(row + c + h * N, (n < N ? n : N) * static_cast<int>(sizeof(T)));
        w[4 * h] = q.x; w[4 * h + 1] = q.y; w[4 * h + 2] = q.z; w[4 * h + 3] = q.w;
        if (n < N) {                                 // what lies past the row
          if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * h + i] = i < n ? w[4 * h + i] : 0u;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[4 * h + i] = 2 * i + 1 < n ? w[4 * h + i] : (2 * i < n ? w[4 * h + i] & 0xFFFFu : 0u);
          }
        }
      }
    }
  }
  // the largest |element| as fp32 bits; at least 0x7F800000 where one is not finite
  __device__ __forceinline__ uint32_t amax_bits() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
      // magnitudes of 16-bit floats order like their bits, NaN above infinity
      uint32_t hi = 0, lo = 0;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        hi = max(hi, w[i] & 0x7FFF0000u);
        lo = max(lo, w[i] & 0x00007FFFu);
      }
      const uint32_t m = max(hi >> 16, lo);
      if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
      else return m >= 0x7C00u ? 0x7F800000u : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(m))));
    }
  }
  __device__ __forceinline__ void floats(float (&f)[16]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 p = __half22float2(h);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
};

// Codes and scale byte of the block that this lane and its neighbour (lane ^ 1) hold, 16 elements each;
// every lane of the warp takes part. A block that is not finite: byte 255 and zero codes.
template <typename T>
__device__ __forceinline__ uint32_t quantize_group(const Group<T>& v, uint2& codes) {
  uint32_t am = v.amax_bits();
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  const bool bad = am >= 0x7F800000u;
  const int e = bad ? 128 : e2m1_exponent(am);
  const float scale = __uint_as_float(static_cast<uint32_t>(bad ? 0 : 127 - e) << 23);   // 2^-e
  float f[16];
  v.floats(f);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = f[i] * scale;
  codes = make_uint2(cvt_e2m1x8(f), cvt_e2m1x8(f + 8));
  if (bad) codes = make_uint2(0, 0);
  return static_cast<uint32_t>(e + 127);
}

// 2^(byte - 127); byte 255 is NaN
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : (byte ? byte << 23 : 0x00400000u));
}

}  // namespace mm

// Rows in 8 bits (quant8.cu, norm.cu, swiglu.cu): e4m3 codes in the two forms the
// layer's activations have.
//   MX  32 elements a block; e = the smallest integer with 448 * 2^e >= max(amax, 1e-10),
//       code = e4m3(x * 2^-e), scale byte e + 127
//   F8  128 elements a block; s = max(amax, 1e-10) / 448 in fp32 (IEEE division),
//       code = e4m3(fp32(x / s)) (IEEE division), scale s
// Codes round to nearest, ties to the even code. A block that holds a NaN or an
// infinity gets zero codes and a scale of NaN (MX: byte 255).
//
// A lane holds 16 consecutive elements of a row: 16 codes are one 16-byte access, and a
// block's other lanes (2 of MX, 8 of F8) are shuffles away.
#pragma once

#include "mx_quant.cuh"
#include "quant.cuh"

namespace mm {

constexpr int kMxBlock = 32, kF8Block = 128;
__host__ __device__ constexpr int block8(int variant) { return variant == MM_MOE_VARIANT_MX ? kMxBlock : kF8Block; }
// blocks of a row of C elements, and the 16-element groups that its codes fill
__host__ __device__ constexpr int blocks8(int C, int variant) { return (C + block8(variant) - 1) / block8(variant); }
__host__ __device__ constexpr int groups8(int C, int variant) { return blocks8(C, variant) * (block8(variant) / 16); }

// Bits of the largest |f|, at least 0x7F800000 where one is not finite.
__device__ __forceinline__ uint32_t amax_bits16(const float (&f)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

__device__ __forceinline__ uint4 pack_e4m3x16(const float (&f)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(cvt_e4m3x2(f[4 * i], f[4 * i + 1])) |
           (static_cast<uint32_t>(cvt_e4m3x2(f[4 * i + 2], f[4 * i + 3])) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of a lane's 16 elements and its block's scale (the byte, or the fp32 bits). am: the amax bits of those 16. Every
// lane of the warp takes part; a block starts at a lane that is a multiple of its lanes.
__device__ __forceinline__ uint4 encode_mx(const float (&f)[16], uint32_t am, uint32_t& scale) {
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  const bool bad = am >= 0x7F800000u;
  const int e = bad ? 0 : ue8m0_exponent_e4m3(__uint_as_float(am));
  const float by = exp2_neg(e);
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = f[i] * by;
  scale = bad ? 255u : static_cast<uint32_t>(e + 127);
  return bad ? make_uint4(0, 0, 0, 0) : pack_e4m3x16(v);
}
__device__ __forceinline__ uint4 encode_f8(const float (&f)[16], uint32_t am, uint32_t& scale) {
#pragma unroll
  for (int o = 1; o < 8; o *= 2) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
  const bool bad = am >= 0x7F800000u;
  const float s = __fdiv_rn(fmaxf(__uint_as_float(bad ? 0u : am), 1e-10f), 448.0f);
  // f times the reciprocal a little less and a little more (2^-20; it and the products round by 2^-24) has the IEEE
  // quotient between: where both round to the same codes those are its codes, and else, next to a border, the lane
  // divides. (8192x7168 with a division of every element 173 us.)
  const float inv = __frcp_rn(s), less = inv * (1.0f - 0x1p-20f), more = inv * (1.0f + 0x1p-20f);
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = f[i] * less;
  uint4 c = pack_e4m3x16(v);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = f[i] * more;
  const uint4 d = pack_e4m3x16(v);
  if (c.x != d.x || c.y != d.y || c.z != d.z || c.w != d.w) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fdiv_rn(f[i], s);
    c = pack_e4m3x16(v);
  }
  scale = bad ? 0x7FC00000u : __float_as_uint(s);
  return bad ? make_uint4(0, 0, 0, 0) : c;
}

// Codes and scales of rows; cols: code bytes of a row.
struct Out8 {
  int variant;
  uint8_t* codes;
  void* sf;
  int groups, blocks;        // of a row
};
// Group g of a row of codes and (its block's first lane) the scale. `live`: the group is one of the row's.
__device__ __forceinline__ void store_mx(const Out8& o, int64_t row, int g, bool live, const float (&f)[16], uint32_t am) {
  uint32_t scale;
  const uint4 c = encode_mx(f, am, scale);
  if (live) {
    reinterpret_cast<uint4*>(o.codes)[row * o.groups + g] = c;
    if ((g & 1) == 0) static_cast<uint8_t*>(o.sf)[row * o.blocks + (g >> 1)] = static_cast<uint8_t>(scale);
  }
}
__device__ __forceinline__ void store_f8(const Out8& o, int64_t row, int g, bool live, const float (&f)[16], uint32_t am) {
  uint32_t scale;
  const uint4 c = encode_f8(f, am, scale);
  if (live) {
    reinterpret_cast<uint4*>(o.codes)[row * o.groups + g] = c;
    if ((g & 7) == 0) static_cast<float*>(o.sf)[row * o.blocks + (g >> 3)] = __uint_as_float(scale);
  }
}
__device__ __forceinline__ void store8(const Out8& o, int64_t row, int g, bool live, const float (&f)[16], uint32_t am) {
  if (o.variant == MM_MOE_VARIANT_MX) store_mx(o, row, g, live, f, am);
  else store_f8(o, row, g, live, f, am);
}

// Four e4m3 codes of a word as fp32, exact.
__device__ __forceinline__ void decode_e4m3x4(uint32_t c, float* f) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
  __half2 h;
  memcpy(&h, &lo, 4);
  const float2 p = __half22float2(h);
  f[0] = p.x;
  f[1] = p.y;
  memcpy(&h, &hi, 4);
  const float2 q = __half22float2(h);
  f[2] = q.x;
  f[3] = q.y;
}
__device__ __forceinline__ void decode16(const uint4& c, float s, float (&f)[16]) {
  decode_e4m3x4(c.x, f);
  decode_e4m3x4(c.y, f + 4);
  decode_e4m3x4(c.z, f + 8);
  decode_e4m3x4(c.w, f + 12);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] *= s;
}

// Sixteen fp32 values rounded into T as they sit in memory.
template <typename T>
__device__ __forceinline__ void round16(const float (&f)[16], uint32_t (&w)[Group<T>::kWords]) {
  T v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = from_float<T>(f[i]);
  memcpy(w, v, sizeof(v));
}

// 16 bytes of shared memory from any even offset of a 16-byte aligned array on; the granule that holds the last of them
// exists.
__device__ __forceinline__ uint4 shared16_any(const void* array, int offset) {
  const int m = offset & 15;
  const uint4* g = reinterpret_cast<const uint4*>(static_cast<const char*>(array) + (offset - m));
  const uint4 lo = g[0];
  if (m == 0) return lo;
  const uint4 hi = g[1];
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = (m & 8) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = (m & 4) ? w[i + 1] : w[i];
  const uint32_t b = (m & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], b), __funnelshift_r(w[1], w[2], b), __funnelshift_r(w[2], w[3], b),
                    __funnelshift_r(w[3], w[4], b));
}

// Stores the 16-element groups of a warp, each of n (up to 16) elements from `at` on; all lanes take part.
//   kVec    whole groups on 32-byte boundaries: 32 bytes an instruction
//   else    anywhere, through shared memory (512 elements a warp): groups that follow each other by the 16-byte granules of
//           memory they cover, others so that consecutive lanes store consecutive elements
template <typename T, bool kVec>
__device__ __forceinline__ void store_groups(T* at, int n, const uint32_t (&w)[Group<T>::kWords], T* warp_smem) {
  if constexpr (kVec) {
    if (n > 0) {
#pragma unroll
      for (int h = 0; h < Group<T>::kWords / 8; ++h) st_global_v8(reinterpret_cast<float*>(at) + 8 * h, w + 8 * h);
    }
  } else {
    constexpr int kSize = sizeof(T), kWhole = 16 / kSize, kRun = 512;
    const int lane = threadIdx.x & 31;
    const unsigned long long p = reinterpret_cast<unsigned long long>(at), p0 = __shfl_sync(0xffffffffu, p, 0);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < Group<T>::kWords / 4; ++q)
      reinterpret_cast<uint4*>(warp_smem)[lane * (Group<T>::kWords / 4) + q] =
          make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    const bool run = __all_sync(0xffffffffu, n == 16 && p == p0 + static_cast<unsigned long long>(lane) * 16 * kSize);
    __syncwarp();
    if (run) {
      T* to = reinterpret_cast<T*>(p0);
      const int before = static_cast<int>(p0 & 15) / kSize;      // elements of the first granule that are not the run's
#pragma unroll
      for (int i = 0; i < kRun / kWhole / 32; ++i) {
        const int first = (i * 32 + lane) * kWhole - before;     // the granule's first element
        if (first >= 0) *reinterpret_cast<uint4*>(to + first) = shared16_any(warp_smem, first * kSize);
      }
      // what the run has of its first and of its last granule
      if (before && lane < kWhole - before) to[lane] = warp_smem[lane];
      if (lane < before) to[kRun - before + lane] = warp_smem[kRun - before + lane];
      return;
    }
    const int e = lane & 15;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = 2 * i + (lane >> 4);         // the lane whose group these 16 elements are
      T* q = reinterpret_cast<T*>(__shfl_sync(0xffffffffu, p, j));
      if (e < __shfl_sync(0xffffffffu, n, j)) q[e] = warp_smem[j * 16 + e];
    }
  }
}

// Whether rows of C elements at p, `pitch` bytes apart, are whole groups on 32-byte boundaries.
inline bool whole_groups(const void* p, int64_t pitch, int C) {
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(pitch)) % 32 == 0 && C % 16 == 0;
}

// Threads of a row of `groups` groups: a power of two from 32 to `most`, as few as hold it in `each` groups a thread.
inline int row_threads(int groups, int each, int most) {
  int p = 32;
  while (p < most && p * each < groups) p *= 2;
  return p;
}

}  // namespace mm

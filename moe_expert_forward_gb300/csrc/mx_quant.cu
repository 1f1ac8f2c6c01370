// Microscaled 4-bit rows: e2m1 codes (two per byte, the even column in the low
// nibble) with one UE8M0 scale byte per 32 elements.
//   e = the smallest integer with 6 * 2^e >= max(amax, 1e-10); scale byte e + 127;
//   code = e2m1(x * 2^-e), round to nearest, ties to the even code.
// A block that holds a NaN or an infinity gets the scale byte 255 (NaN) and
// zero codes, so everything computed from it is NaN.
//
// The quantiser is bound by its reads (R * C elements in, 17/32 byte per
// element out).  A lane takes 8 elements, four lanes a block: reads of 16 bytes
// a lane and code stores of 4 are contiguous over the warp, and a block's amax
// is two shuffles away.  kBatch octets' loads are in flight per thread.
#include "mx_linear.h"
#include "ptx.cuh"
#include "rowtypes.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;

// 8 fp32 values -> 8 e2m1 codes, value 0 in the lowest nibble
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
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

template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* __restrict__ row, int c, int C, float (&f)[8]) {
  if (kVec) {
    if (c < C) {
      if constexpr (sizeof(T) == 2) {
        const Vec<T, 8> v = *reinterpret_cast<const Vec<T, 8>*>(row + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_float(v.v[i]);
      } else {
        const Vec<T, 4> v0 = *reinterpret_cast<const Vec<T, 4>*>(row + c);
        const Vec<T, 4> v1 = *reinterpret_cast<const Vec<T, 4>*>(row + c + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = to_float(v0.v[i]);
          f[i + 4] = to_float(v1.v[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < C ? to_float(row[c + i]) : 0.f;
  }
}

// Octet o of row r, over all rows; thread i takes octets i, i + step, ...  A row
// has `opr` octets (a multiple of 4); step = d_row * opr + d_oct.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const MxQuantArgs a, int opr, int d_row, int d_oct) {
  pdl_trigger();                      // the product may set itself up meanwhile
  const T* x = static_cast<const T*>(a.x);
  if (a.status && blockIdx.x == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0;
  const int code_octs = (a.C + 31) / 32 * 4;          // octets a row of codes holds
  const int KB = mx_chunks(a.C);
  const int64_t total = a.R * opr;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  int64_t r = i0 / opr;
  int o = static_cast<int>(i0 - r * opr);
  // the last lanes of a warp may be past the end: they take part in the shuffles with zeros
  for (int64_t base = i0 - (threadIdx.x & 31); base < total; base += kBatch * step) {
    float f[kBatch][8];
    int64_t rr[kBatch];
    int oo[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      rr[u] = r;
      oo[u] = o;
      if (r < a.R) {
        load8<T, kVec>(x + r * a.stride, o * 8, a.C, f[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[u][i] = 0.f;
      }
      r += d_row;
      o += d_oct;
      if (o >= opr) {
        o -= opr;
        ++r;
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(f[u][i]) & 0x7FFFFFFFu);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const bool bad = am >= 0x7F800000u;
      const int e = bad ? 128 : e2m1_exponent(am);
      const float scale = __uint_as_float(bad ? 0u : static_cast<uint32_t>(127 - e) << 23);   // 2^-e
#pragma unroll
      for (int i = 0; i < 8; ++i) f[u][i] = bad ? 0.f : f[u][i] * scale;
      const uint32_t codes = cvt_e2m1x8(f[u]);
      if (rr[u] >= a.R) continue;
      const uint8_t sf = static_cast<uint8_t>(e + 127);
      const int K = a.slot ? a.K : 1;
      for (int k = 0; k < K; ++k) {
        int64_t d = rr[u];
        if (a.slot) {
          d = __ldg(a.slot + rr[u] * K + k);
          if (d < 0 || d >= a.num_rows) continue;
        }
        if (oo[u] < code_octs) *reinterpret_cast<uint32_t*>(a.codes + (d * code_octs + oo[u]) * 4) = codes;
        if ((oo[u] & 3) == 0) {
          const int b = oo[u] >> 2;
          if (a.chunks) a.sf[mx_sf_word(d, b >> 2, KB) + (b & 3)] = sf;
          else a.sf[d * (code_octs / 4) + b] = sf;
        }
      }
    }
  }
}

// Values of codes [R, ceil(C/32) * 16 bytes] with row-major scales.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int64_t R, int C,
                      T* __restrict__ out, int64_t out_stride) {
  const int octs = (C + 31) / 32 * 4;
  const int64_t total = R * octs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t r = i / octs;
    const int o = static_cast<int>(i - r * octs);
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    const uint32_t b = __ldg(sf + (i >> 2));
    const float scale = b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b ? b << 23 : 0x00400000u);
    T* d = out + r * out_stride + o * 8;
    Vec<T, 8> v;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      // sign, then the magnitude (2-bit exponent, 1-bit mantissa; 0 and 0.5 are its subnormals)
      const uint32_t n = (w >> (4 * q)) & 15u, ex = (n >> 1) & 3u, m = n & 1u;
      const float mag = ex ? __uint_as_float((ex + 126u) << 23 | m << 22) : 0.5f * m;
      v.v[q] = from_float<T>(scale * (n & 8u ? -mag : mag));
    }
    if (kVec && o * 8 + 8 <= C) {
      constexpr int N = 16 / sizeof(T);
#pragma unroll
      for (int h = 0; h < 8 / N; ++h)
        reinterpret_cast<Vec<T, N>*>(d)[h] = reinterpret_cast<const Vec<T, N>*>(&v)[h];
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (o * 8 + q < C) d[q] = v.v[q];
    }
  }
}

// Row-major scale bytes [E, N, ceil(C/32)] -> chunks [E][ceil(N/128)][mx_chunks(C)][512];
// one thread a 4-byte word, 127 (a scale of one) past N and past the last block.
__global__ void __launch_bounds__(kThreads)
    prepare_kernel(const uint8_t* __restrict__ sf, int E, int N, int C, uint8_t* __restrict__ out) {
  const int nb = (C + 31) / 32, KB = mx_chunks(C), rows = (N + 127) / 128 * 128;
  const int64_t total = static_cast<int64_t>(E) * rows * KB;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    // i counts words in the order of the output
    const int64_t chunk = i >> 7;
    const int w = static_cast<int>(i & 127);
    const int kb = static_cast<int>(chunk % KB);
    const int64_t rb = chunk / KB;                       // 128-row block, over all experts
    const int64_t e = rb / (rows / 128);
    const int n = static_cast<int>(rb - e * (rows / 128)) * 128 + (w >> 2) + (w & 3) * 32;
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = kb * 4 + j;
      const uint32_t byte = (n < N && b < nb) ? __ldg(sf + (e * N + n) * nb + b) : 127u;
      v |= byte << (8 * j);
    }
    reinterpret_cast<uint32_t*>(out)[i] = v;
  }
}

int blocks_for(int64_t threads, int per_sm) {
  int64_t b = (threads + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(dev_info().sms) * per_sm;
  return static_cast<int>(b < 1 ? 1 : (b > cap ? cap : b));
}

bool wide(const void* p, int64_t pitch_bytes) {
  return access_bytes(reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(pitch_bytes)) == 16;
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs& a, cudaStream_t s) {
  const int opr = a.chunks ? mx_chunks(a.C) * 16 : (a.C + 31) / 32 * 4;
  const int grid = blocks_for((a.R * opr + kBatch - 1) / kBatch, 8);
  const int64_t step = static_cast<int64_t>(grid) * kThreads;
  const int d_row = static_cast<int>(step / opr), d_oct = static_cast<int>(step % opr);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    if (wide(a.x, a.stride * sizeof(T)) && a.C % 8 == 0)
      quantize_kernel<T, true><<<grid, kThreads, 0, s>>>(a, opr, d_row, d_oct);
    else
      quantize_kernel<T, false><<<grid, kThreads, 0, s>>>(a, opr, d_row, d_oct);
    return cudaGetLastError();
  });
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* sf, int64_t R, int C, int dtype, void* out,
                                 int64_t out_stride, cudaStream_t s) {
  const int grid = blocks_for(R * ((C + 31) / 32 * 4), 16);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    if (wide(out, out_stride * sizeof(T)))
      dequantize_kernel<T, true><<<grid, kThreads, 0, s>>>(codes, sf, R, C, static_cast<T*>(out), out_stride);
    else
      dequantize_kernel<T, false><<<grid, kThreads, 0, s>>>(codes, sf, R, C, static_cast<T*>(out), out_stride);
    return cudaGetLastError();
  });
}

cudaError_t launch_mx_prepare(const uint8_t* sf, int E, int N, int C, uint8_t* out, cudaStream_t s) {
  const int64_t words = static_cast<int64_t>(E) * ((N + 127) / 128 * 128) * mx_chunks(C);
  prepare_kernel<<<blocks_for(words, 16), kThreads, 0, s>>>(sf, E, N, C, out);
  return cudaGetLastError();
}

}  // namespace mm

// Microscaled 4-bit rows: e2m1 codes (two per byte, the even column in the low
// nibble) with one UE8M0 scale byte per 32 elements.
//   e = the smallest integer with 6 * 2^e >= max(amax, 1e-10); scale byte e + 127;
//   code = e2m1(x * 2^-e), round to nearest, ties to the even code.
// A block that holds a NaN or an infinity gets the scale byte 255 (NaN) and
// zero codes, so everything computed from it is NaN.
//
// Both directions are bound by memory (R * C elements on one side, 17/32 byte per
// element on the other).  A lane takes 16 elements, two lanes a block: 16-bit
// rows are read and written 32 bytes a lane and codes 8, contiguous over the
// warp, and a block's amax is one shuffle away.  The amax is taken on the packed
// 16-bit words, and every thread steps its (row, group) pair instead of dividing.
#include "mx_quant.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 2;            // groups of 16 elements a thread has in flight

// The position of a thread in [rows][groups of 16], stepped by a fixed number of groups.
struct Walk {
  int64_t r;
  int g;
  __device__ __forceinline__ Walk(int64_t i, int groups) : r(i / groups), g(static_cast<int>(i - r * groups)) {}
  __device__ __forceinline__ void step(int d_row, int d_group, int groups) {
    r += d_row;
    g += d_group;
    if (g >= groups) {
      g -= groups;
      ++r;
    }
  }
};

// step = gridDim * kThreads groups = d_row rows and d_group groups; `groups` (of a row) is even.
template <typename T, bool kVec, bool kChunks, bool kSlots>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const MxQuantArgs a, int groups, int d_row, int d_group) {
  pdl_trigger();                      // the product may set itself up meanwhile
  const T* x = static_cast<const T*>(a.x);
  if (a.status && blockIdx.x == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0;
  const int code_groups = (a.C + 31) / 32 * 2;        // groups a row of codes holds
  const int KB = mx_chunks(a.C);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  Walk at(i0, groups);
  // a warp runs while any of its lanes has a row, so the shuffles see all of it
  while (__any_sync(0xffffffffu, at.r < a.R)) {
    Group<T> v[kBatch];
    int64_t rr[kBatch];
    int gg[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      rr[u] = at.r;
      gg[u] = at.g;
      if (at.r < a.R) v[u].template load<kVec>(x + at.r * a.stride, at.g * 16, a.C);
      else v[u].clear();
      at.step(d_row, d_group, groups);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint2 codes;
      const uint8_t sf = static_cast<uint8_t>(quantize_group(v[u], codes));
      if (rr[u] < a.R) {
        const int K = kSlots ? a.K : 1;
        for (int k = 0; k < K; ++k) {
          int64_t d = rr[u];
          if (kSlots) {
            d = __ldg(a.slot + rr[u] * K + k);
            if (d < 0 || d >= a.num_rows) continue;
          }
          if (!kChunks || gg[u] < code_groups) reinterpret_cast<uint2*>(a.codes)[d * code_groups + gg[u]] = codes;
          if ((gg[u] & 1) == 0) {
            const int b = gg[u] >> 1;
            if (kChunks) a.sf[mx_sf_word(d, b >> 2, KB) + (b & 3)] = sf;
            else a.sf[d * (code_groups / 2) + b] = sf;
          }
        }
      }
    }
  }
}

// Eight e2m1 codes times s.
__device__ __forceinline__ void decode8(uint32_t c, float s, float* f) {
  uint32_t h[4];                      // pairs of fp16, exact
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 p;
    memcpy(&p, &h[i], 4);
    const float2 v = __half22float2(p);
    f[2 * i] = v.x * s;
    f[2 * i + 1] = v.y * s;
  }
}

// Values of codes [R, ceil(C/32) * 16 bytes] with row-major scales; C a multiple of 16, rows of out 32-byte aligned.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int64_t R, int C,
                      T* __restrict__ out, int64_t out_stride, int groups, int d_row, int d_group) {
  const int nb = (C + 31) / 32;
  Walk at(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, groups);
  while (at.r < R) {
    uint2 w[kBatch];
    uint32_t b[kBatch];
    T* d[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      d[u] = nullptr;
      if (at.r < R) {
        w[u] = __ldg(reinterpret_cast<const uint2*>(codes + at.r * nb * 16) + at.g);
        b[u] = __ldg(sf + at.r * nb + (at.g >> 1));
        d[u] = out + at.r * out_stride + at.g * 16;
      }
      at.step(d_row, d_group, groups);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!d[u]) continue;
      const float s = ue8m0_value(b[u]);
      float f[16];
      decode8(w[u].x, s, f);
      decode8(w[u].y, s, f + 8);
      T v[16];
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = from_float<T>(f[q]);
      uint32_t o[Group<T>::kWords];
      memcpy(o, v, sizeof(v));
#pragma unroll
      for (int h = 0; h < Group<T>::kWords / 8; ++h) st_global_v8(reinterpret_cast<float*>(d[u]) + 8 * h, o + 8 * h);
    }
  }
}

// The same for rows of out on no 32-byte boundary: a lane takes a 16-byte granule of out (Granule), whose elements
// start anywhere in the codes' words and lie in up to two blocks. (With the form above and single elements stored,
// 32776x4095 bf16 took 670 us, 4096 columns 51.)
template <typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_any_kernel(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ sf, int64_t R, int C,
                          T* __restrict__ out, int64_t out_stride, int granules, int d_row, int d_granule) {
  constexpr int N = Granule<T>::kWhole;
  const int nb = (C + 31) / 32;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  for (Walk at(i0, granules); at.r < R; at.step(d_row, d_granule, granules)) {
    T* o = out + at.r * out_stride;
    const Granule<T> g(o, C, at.g);
    if (g.n <= 0) continue;
    const uint32_t* c = codes + at.r * nb * 4 + (g.first >> 3);
    const uint32_t lo = __ldg(c), hi = (g.first & 7) + g.n > 8 ? __ldg(c + 1) : 0u;
    const int b = g.first >> 5;
    const uint8_t* sr = sf + at.r * nb + b;
    const float s0 = ue8m0_value(__ldg(sr));
    const int split = 32 * (b + 1) - g.first;        // elements of the first block
    const float s1 = split < g.n ? ue8m0_value(__ldg(sr + 1)) : 0.f;
    float f[8];
    decode8(__funnelshift_r(lo, hi, (g.first & 7) * 4), 1.0f, f);
    Vec<T, N> v;
#pragma unroll
    for (int q = 0; q < N; ++q) v.v[q] = from_float<T>(f[q] * (q < split ? s0 : s1));
    g.store(o, v);
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

// Per SM: as many CTAs as one pass over the data takes. 65536x4096 bf16, into 4 bits and back: 97 and 98 us (6.7 TB/s),
// with 8 CTAs an SM that step through the data 104 and 114.
constexpr int kOnePass = 1 << 20;

int blocks_for(int64_t threads, int per_sm) {
  int64_t b = (threads + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(dev_info().sms) * per_sm;
  return static_cast<int>(b < 1 ? 1 : (b > cap ? cap : b));
}

// rows of whole 16-element groups on 32-byte boundaries
bool wide(const void* p, int64_t pitch_bytes, int C) {
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(pitch_bytes)) % 32 == 0 && C % 16 == 0;
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs& a, cudaStream_t s) {
  const int groups = a.chunks ? mx_chunks(a.C) * 8 : (a.C + 31) / 32 * 2;
  const int grid = blocks_for((a.R * groups + kBatch - 1) / kBatch, kOnePass);
  const int64_t step = static_cast<int64_t>(grid) * kThreads;
  const int d_row = static_cast<int>(step / groups), d_group = static_cast<int>(step % groups);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    auto go = [&](auto vec) {
      constexpr bool V = decltype(vec)::value;
      if (a.slot && a.chunks) quantize_kernel<T, V, true, true><<<grid, kThreads, 0, s>>>(a, groups, d_row, d_group);
      else if (a.slot) quantize_kernel<T, V, false, true><<<grid, kThreads, 0, s>>>(a, groups, d_row, d_group);
      else if (a.chunks) quantize_kernel<T, V, true, false><<<grid, kThreads, 0, s>>>(a, groups, d_row, d_group);
      else quantize_kernel<T, V, false, false><<<grid, kThreads, 0, s>>>(a, groups, d_row, d_group);
      return cudaGetLastError();
    };
    return wide(a.x, a.stride * sizeof(T), a.C) ? go(std::true_type{}) : go(std::false_type{});
  });
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* sf, int64_t R, int C, int dtype, void* out,
                                 int64_t out_stride, cudaStream_t s) {
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    T* o = static_cast<T*>(out);
    const bool vec = wide(out, out_stride * sizeof(T), C);
    const int parts = vec ? C / 16 : Granule<T>::most(C);          // of a row
    const int grid = blocks_for(vec ? (R * parts + kBatch - 1) / kBatch : R * parts, kOnePass);
    const int64_t step = static_cast<int64_t>(grid) * kThreads;
    const int d_row = static_cast<int>(step / parts), d_part = static_cast<int>(step % parts);
    if (vec)
      dequantize_kernel<T><<<grid, kThreads, 0, s>>>(codes, sf, R, C, o, out_stride, parts, d_row, d_part);
    else
      dequantize_any_kernel<T><<<grid, kThreads, 0, s>>>(reinterpret_cast<const uint32_t*>(codes), sf, R, C, o,
                                                         out_stride, parts, d_row, d_part);
    return cudaGetLastError();
  });
}

cudaError_t launch_mx_prepare(const uint8_t* sf, int E, int N, int C, uint8_t* out, cudaStream_t s) {
  const int64_t words = static_cast<int64_t>(E) * ((N + 127) / 128 * 128) * mx_chunks(C);
  prepare_kernel<<<blocks_for(words, 16), kThreads, 0, s>>>(sf, E, N, C, out);
  return cudaGetLastError();
}

}  // namespace mm

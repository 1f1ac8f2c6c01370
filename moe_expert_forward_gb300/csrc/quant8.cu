// Rows of fp32, bf16 or fp16 into 8 bits and back (the two forms of rows8.cuh): what
// the layer takes as x and x_sf, and what a training step keeps of its activations.
//
// Bound by memory both ways: an element is read in its own type and written as one
// byte and a 32nd, or the reverse.  A lane takes 16 elements, and a warp's lanes
// follow each other through the rows.
//
// Measured: 65536x4096 bf16 into "mx" 126 us and back 120 (813 MB: 95 and 100 % of the copy rate), into "f8" 208 and back
// 119 (58 %: two conversions an element; fp32 206, 96 %), 4095 columns 167 and 153, "f8" 231 and 148.
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

// step = gridDim * kThreads groups = d_row rows and d_group groups. A row's groups are those its codes fill, so that
// blocks lie inside a warp.
// kBatch: groups a thread has in flight.
template <typename T, bool kVec, int kBatch>
__global__ void __launch_bounds__(kThreads)
    quantize8_kernel(const T* __restrict__ x, int64_t stride, int64_t R, int C, const Out8 out, int d_row, int d_group) {
  Walk at(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, out.groups);
  // a warp runs while any of its lanes has a row, so the shuffles see all of it
  while (__any_sync(0xffffffffu, at.r < R)) {
    Group<T> v[kBatch];
    int64_t rr[kBatch];
    int gg[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      rr[u] = at.r;
      gg[u] = at.g;
      if (at.r < R) v[u].template load<kVec>(x + at.r * stride, at.g * 16, C);
      else v[u].clear();
      at.step(d_row, d_group, out.groups);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      float f[16];
      v[u].floats(f);
      store8(out, rr[u], gg[u], rr[u] < R, f, v[u].amax_bits());
    }
  }
}

// `groups`: 16-element groups that hold one of a row's C elements.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    dequantize8_kernel(const Out8 in, int64_t R, int C, T* __restrict__ out, int64_t stride, int groups, int d_row,
                       int d_group) {
  __shared__ alignas(16) T s_run[kVec ? 1 : kWarps * 512];
  T* run = kVec ? s_run : s_run + (threadIdx.x >> 5) * 512;
  // a warp runs while any of its lanes has a row, so the shuffles see all of it
  for (Walk at(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, groups); __any_sync(0xffffffffu, at.r < R);
       at.step(d_row, d_group, groups)) {
    uint4 c = make_uint4(0, 0, 0, 0);
    float s = 0.f;
    T* d = out;
    int n = 0;
    if (at.r < R) {
      c = __ldg(reinterpret_cast<const uint4*>(in.codes) + at.r * in.groups + at.g);
      s = in.variant == MM_MOE_VARIANT_MX
              ? ue8m0_value(__ldg(static_cast<const uint8_t*>(in.sf) + at.r * in.blocks + (at.g >> 1)))
              : __ldg(static_cast<const float*>(in.sf) + at.r * in.blocks + (at.g >> 3));
      d = out + at.r * stride + at.g * 16;
      n = min(16, C - at.g * 16);
    }
    float f[16];
    decode16(c, s, f);
    uint32_t w[Group<T>::kWords];
    round16<T>(f, w);
    store_groups<T, kVec>(d, n, w, run);
  }
}

// CTAs of one pass over `threads` threads
int grid_for(int64_t threads) {
  const int64_t b = (threads + kThreads - 1) / kThreads, most = int64_t(1) << 28;
  return static_cast<int>(b < 1 ? 1 : (b > most ? most : b));
}

}  // namespace

cudaError_t launch_quantize8(const void* x, int dtype, int64_t stride, int64_t R, int C, int variant, void* codes,
                             void* sf, cudaStream_t s) {
  const Out8 o{variant, static_cast<uint8_t*>(codes), sf, groups8(C, variant), blocks8(C, variant)};
  // Groups a thread: four of rows on 32-byte boundaries where they are more than 2^22, else one (65536x4096 bf16 132 us for
  // 143 with one, 136 with two; 65536x4095 205 for 172; 33x1001 9.6 for 7.4).
  const bool vec = whole_groups(x, stride * dtype_size(dtype), C);
  const int batch = vec && R * o.groups > (int64_t(1) << 22) ? 4 : 1;
  const int grid = grid_for((R * o.groups + batch - 1) / batch);
  const int64_t step = static_cast<int64_t>(grid) * kThreads;
  const int d_row = static_cast<int>(step / o.groups), d_group = static_cast<int>(step % o.groups);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* p = static_cast<const T*>(x);
    if (batch == 4) quantize8_kernel<T, true, 4><<<grid, kThreads, 0, s>>>(p, stride, R, C, o, d_row, d_group);
    else if (vec) quantize8_kernel<T, true, 1><<<grid, kThreads, 0, s>>>(p, stride, R, C, o, d_row, d_group);
    else quantize8_kernel<T, false, 1><<<grid, kThreads, 0, s>>>(p, stride, R, C, o, d_row, d_group);
    return cudaGetLastError();
  });
}

cudaError_t launch_dequantize8(const void* codes, const void* sf, int64_t R, int C, int variant, int dtype, void* out,
                               int64_t stride, cudaStream_t s) {
  const Out8 in{variant, static_cast<uint8_t*>(const_cast<void*>(codes)), const_cast<void*>(sf), groups8(C, variant),
                blocks8(C, variant)};
  const int groups = (C + 15) / 16;
  const int grid = grid_for(R * groups);
  const int64_t step = static_cast<int64_t>(grid) * kThreads;
  const int d_row = static_cast<int>(step / groups), d_group = static_cast<int>(step % groups);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    T* p = static_cast<T*>(out);
    if (whole_groups(out, stride * sizeof(T), C))
      dequantize8_kernel<T, true><<<grid, kThreads, 0, s>>>(in, R, C, p, stride, groups, d_row, d_group);
    else
      dequantize8_kernel<T, false><<<grid, kThreads, 0, s>>>(in, R, C, p, stride, groups, d_row, d_group);
    return cudaGetLastError();
  });
}

}  // namespace mm

// The activation between the experts' two products, on rows [gate | up], and its
// gradients from gate and up kept in 8 bits (MX, each half in blocks of its own).
//   a = gate s up w,  s = 1 / (1 + exp(-gate)),  w the weight of the row's pair (or 1)
//   d_gate = d_a w up s (1 + gate (1 - s)),  d_up = d_a w gate s,
//   d_w[pair] = sum over the row of d_a gate s up
// With a routing, rows that hold no pair are padding: every output is zero there and
// no input is read.  The router's weight is applied here, as in the fused layer, so
// that training need not keep the experts' outputs for the weights' gradient.
//
// Memory bounds both (forward: 4 bytes an element of a read and 2 written in 16 bits,
// and 2 1/16 where kept; back: 2 and 2 1/16 read, 4 written).  A row has a group of
// threads, 16 columns a lane and step, and everything about an element stays in its
// lane but a block's amax and the row's dot.
//
// 16-bit rows take the fast exponential and reciprocal (within 2^-20, under a
// hundredth of the rounding of the result); fp32 rows expf and the IEEE division.
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kMx = MM_MOE_VARIANT_MX;

template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 4) return __fdiv_rn(1.0f, 1.0f + expf(-g));
  else return rcp_approx(1.0f + __expf(-g));
}

// The pair of a pool row, or -1 where the row is padding. Without a routing a row is its own.
__device__ __forceinline__ int64_t pair_of(const SwigluRows& r, int64_t row) {
  if (row >= r.rows) return -1;
  if (!r.src) return row;
  if (row >= static_cast<int64_t>(__ldg(r.blk_off + r.E)) * r.block_m) return -1;
  return __ldg(r.src + row);
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_kernel(const SwigluRows r, const T* __restrict__ h, int64_t stride, const float* __restrict__ w,
                  T* __restrict__ a, const Out8 q, const Out8 kept, int P) {
  __shared__ alignas(16) T s_run[kVec ? 1 : kThreads / 32 * 512];
  T* run = kVec ? s_run : s_run + (threadIdx.x >> 5) * 512;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / P) + threadIdx.x / P;
  const int l = threadIdx.x % P, I = r.I;
  const int64_t pair = pair_of(r, row);
  const float weight = pair >= 0 ? (w ? __ldg(w + pair) : 1.f) : 0.f;
  const T* hr = h + (pair >= 0 ? row : 0) * stride;
  const int groups = blocks8(I, kMx) * 2;
  const bool in = row < r.rows;
  for (int g = l; g - (l & 31) < groups; g += P) {
    Group<T> vg, vu;
    if (pair >= 0 && g * 16 < I) {
      vg.template load<kVec>(hr, g * 16, I);
      vu.template load<kVec>(hr + I, g * 16, I);
    } else {
      vg.clear();
      vu.clear();
    }
    float gate[16], up[16];
    vg.floats(gate);
    vu.floats(up);
    if (kept.codes) {                            // gate and up as blocks of one row of both
      store8(kept, row * 2, g, in && g < groups, gate, vg.amax_bits());
      store8(kept, row * 2 + 1, g, in && g < groups, up, vu.amax_bits());
    }
    float f[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = gate[i] * sigmoid<T>(gate[i]) * up[i] * weight;
    if (pair < 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] = 0.f;
    if (q.codes) {
      float z[16];                               // past the row: zeros, also where the weight is not finite
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = g * 16 + i < I ? f[i] : 0.f;
      store8(q, row, g, in && g < groups, z, amax_bits16(z));
    }
    if (a) {
      uint32_t o[Group<T>::kWords];
      round16<T>(f, o);
      store_groups<T, kVec>(a + row * I + g * 16, in ? min(16, I - g * 16) : 0, o, run);
    }
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const SwigluRows r, const T* __restrict__ d_a, int64_t stride, const Out8 kept,
                           const float* __restrict__ w, T* __restrict__ d_h, float* __restrict__ d_w, int P) {
  __shared__ float s_part[kThreads / 32];
  __shared__ alignas(16) T s_run[kVec ? 1 : kThreads / 32 * 512];
  T* run = kVec ? s_run : s_run + (threadIdx.x >> 5) * 512;
  // pairs that no row holds: masked slots
  if (d_w)
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; p < r.pairs;
         p += static_cast<int64_t>(gridDim.x) * kThreads)
      if (__ldg(r.slot + p) < 0) d_w[p] = 0.f;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / P) + threadIdx.x / P;
  const int l = threadIdx.x % P, I = r.I;
  const int64_t pair = pair_of(r, row);
  const float weight = pair >= 0 ? (w ? __ldg(w + pair) : 1.f) : 0.f;
  const bool in = row < r.rows;
  const T* dr = d_a + (pair >= 0 ? row : 0) * stride;
  const uint4* codes = reinterpret_cast<const uint4*>(kept.codes) + (pair >= 0 ? row : 0) * 2 * kept.groups;
  const uint8_t* sf = static_cast<const uint8_t*>(kept.sf) + (pair >= 0 ? row : 0) * 2 * kept.blocks;
  const int groups = (I + 15) / 16;
  float dot = 0.f;
  for (int g = l; g - (l & 31) < groups; g += P) {
    float og[16], ou[16];
    if (pair >= 0 && g < groups) {
      Group<T> vd;
      vd.template load<kVec>(dr, g * 16, I);
      float gate[16], up[16], d[16];
      const uint4 cg = __ldg(codes + g), cu = __ldg(codes + kept.groups + g);
      decode16(cg, ue8m0_value(__ldg(sf + (g >> 1))), gate);
      decode16(cu, ue8m0_value(__ldg(sf + kept.blocks + (g >> 1))), up);
      vd.floats(d);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float s = sigmoid<T>(gate[i]);
        const float silu = gate[i] * s;
        if (g * 16 + i < I) dot = fmaf(d[i] * silu, up[i], dot);
        const float dw = d[i] * weight;
        og[i] = dw * up[i] * (s * (1.0f + gate[i] * (1.0f - s)));
        ou[i] = dw * silu;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) og[i] = ou[i] = 0.f;
    }
    uint32_t o[Group<T>::kWords];
    T* at = d_h + row * 2 * I + g * 16;
    const int n = in ? min(16, I - g * 16) : 0;
    round16<T>(og, o);
    store_groups<T, kVec>(at, n, o, run);
    round16<T>(ou, o);
    store_groups<T, kVec>(at + I, n, o, run);
  }
  if (!d_w) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
  if (P > 32) {
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = dot;
    __syncthreads();
    dot = 0.f;
    if (l == 0)
      for (int i = 0; i < P / 32; ++i) dot += s_part[threadIdx.x / 32 + i];
  }
  if (l == 0 && pair >= 0) d_w[pair] = dot;
}

Out8 kept_rows(void* codes, void* sf, int I) {
  return Out8{kMx, static_cast<uint8_t*>(codes), sf, groups8(I, kMx), blocks8(I, kMx)};
}

}  // namespace

cudaError_t launch_swiglu(const SwigluRows& r, int dtype, const void* h, int64_t stride, const float* w, void* a,
                          void* codes, void* sf, void* kept, void* kept_sf, cudaStream_t s) {
  const int elem = dtype_size(dtype);
  const bool vec = whole_groups(h, stride * elem, r.I) && whole_groups(a, static_cast<int64_t>(r.I) * elem, r.I);
  const int P = row_threads(groups8(r.I, kMx), 1, kThreads);
  const unsigned grid = static_cast<unsigned>((r.rows + kThreads / P - 1) / (kThreads / P));
  const Out8 q = kept_rows(codes, sf, r.I), k = kept_rows(kept, kept_sf, r.I);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* p = static_cast<const T*>(h);
    T* o = static_cast<T*>(a);
    if (vec) swiglu_kernel<T, true><<<grid, kThreads, 0, s>>>(r, p, stride, w, o, q, k, P);
    else swiglu_kernel<T, false><<<grid, kThreads, 0, s>>>(r, p, stride, w, o, q, k, P);
    return cudaGetLastError();
  });
}

cudaError_t launch_swiglu_backward(const SwigluRows& r, int dtype, const void* d_a, int64_t stride, const void* kept,
                                   const void* kept_sf, const float* w, void* d_h, float* d_w, cudaStream_t s) {
  const int elem = dtype_size(dtype);
  const bool vec = whole_groups(d_a, stride * elem, r.I) && whole_groups(d_h, static_cast<int64_t>(r.I) * elem, r.I);
  const int P = row_threads((r.I + 15) / 16, 1, kThreads);
  const unsigned grid = static_cast<unsigned>((r.rows + kThreads / P - 1) / (kThreads / P));
  const Out8 k = kept_rows(const_cast<void*>(kept), const_cast<void*>(kept_sf), r.I);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* p = static_cast<const T*>(d_a);
    T* o = static_cast<T*>(d_h);
    if (vec) swiglu_backward_kernel<T, true><<<grid, kThreads, 0, s>>>(r, p, stride, k, w, o, d_w, P);
    else swiglu_backward_kernel<T, false><<<grid, kThreads, 0, s>>>(r, p, stride, k, w, o, d_w, P);
    return cudaGetLastError();
  });
}

}  // namespace mm

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
// and 2 1/16 where kept; back: 2 and 2 1/16 read, 4 written).  A CTA takes a few rows,
// looks their pairs and weights up at once, and then a lane takes 16 columns at a time;
// everything about an element stays in its lane but a block's amax and the row's dot.
// Two groups a lane in flight changed nothing: four CTAs an SM have the loads in flight.
//
// 16-bit rows take the fast exponential (ex2 of the rounded product of the gate and log2 e) and reciprocal, both without
// denormals: a third of the instructions. The sigmoid is then within 2^-21 + |gate| 2^-23.7 of its value below zero
// (2^-20 at -8, 2^-17 at -80; half of it and less above zero), under a hundredth of the rounding of a 16-bit result, and 0
// from -87.4 on, where it is below 2^-126. d_w has it too, in fp32, in terms whose gate and up are rounded to 2^-4. fp32 rows
// take expf and the IEEE division.
//
// Measured (one of the calls of a graph over 400 MB of inputs): 13248 pool rows (2048 tokens, top-6 of 64) of 2048 columns in
// bf16, kept in 8 bits, 39 us forward and 41 back, 79 and 77 % of the copy rate (31 us each; of 256 experts, 16128 rows, 44
// and 43 for 34.5), with a in 8 bits too 47 (76 %), in fp32 61 and 68 (89 and 80 %); 4093 rows of 2731 in fp16 26 and 29
// (rows on no 32-byte boundary: shifted from and into 16-byte granules; 2736 columns 18 and 20).
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kMx = MM_MOE_VARIANT_MX;

template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 4) return __fdiv_rn(1.0f, 1.0f + expf(-g));
  else {
    float e;                                     // exp(-g) as a power of two; what is below 2^-126 is 0
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    return rcp_approx(1.0f + e);
  }
}

constexpr int kMostRows = 64;        // of a CTA

// The CTA's rows: their pairs (-1: padding, or past the end) and weights. Without a routing a row is its own pair.
struct Rows {
  int64_t pair[kMostRows];
  float w[kMostRows];
};
__device__ __forceinline__ void look_up(Rows& s, const SwigluRows& r, const float* __restrict__ w, int64_t row0, int rows) {
  for (int i = threadIdx.x; i < rows; i += kThreads) {
    const int64_t row = row0 + i;
    int64_t pair = -1;
    if (row < r.rows) pair = !r.src ? row : row < static_cast<int64_t>(__ldg(r.blk_off + r.E)) * r.block_m ? __ldg(r.src + row) : -1;
    s.pair[i] = pair;
    s.w[i] = pair >= 0 ? (w ? __ldg(w + pair) : 1.f) : 0.f;
  }
  __syncthreads();
}

// `rows` rows of a CTA, as groups of 16 columns in a row; a row's groups are those its codes fill, an even number, so that
// blocks lie inside a warp.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 4)
    swiglu_kernel(const SwigluRows r, int rows, const T* __restrict__ h, int64_t stride, const float* __restrict__ w,
                  T* __restrict__ a, const Out8 q, const Out8 kept) {
  __shared__ Rows s_rows;
  __shared__ alignas(16) T s_run[kVec ? 1 : kThreads / 32 * 512];
  T* run = kVec ? s_run : s_run + (threadIdx.x >> 5) * 512;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows;
  look_up(s_rows, r, w, row0, rows);
  const int I = r.I, groups = kept.groups, items = rows * groups;
  for (int i = threadIdx.x; i - static_cast<int>(threadIdx.x & 31) < items; i += kThreads) {
    const int at = i / groups, g = i - at * groups;
    const int64_t row = row0 + at;
    const bool in = i < items && row < r.rows;
    const bool live = in && s_rows.pair[at] >= 0;
    Group<T> vg, vu;
    if (live && g * 16 < I) {
      const T* hr = h + row * stride;
      vg.template load<kVec>(hr, g * 16, I);
      vu.template load<kVec>(hr + I, g * 16, I);
    } else {
      vg.clear();
      vu.clear();
    }
    if (!__any_sync(0xffffffffu, live)) {        // padding: zeros, and the scale of zeros
      const uint8_t zero = static_cast<uint8_t>(ue8m0_exponent_e4m3(0.f) + 127);
      if (in && kept.codes) {
        reinterpret_cast<uint4*>(kept.codes)[row * 2 * groups + g] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint4*>(kept.codes)[(row * 2 + 1) * groups + g] = make_uint4(0, 0, 0, 0);
        static_cast<uint8_t*>(kept.sf)[(row * 2 + (g & 1)) * kept.blocks + (g >> 1)] = zero;
      }
      if (in && q.codes) {
        reinterpret_cast<uint4*>(q.codes)[row * groups + g] = make_uint4(0, 0, 0, 0);
        if ((g & 1) == 0) static_cast<uint8_t*>(q.sf)[row * q.blocks + (g >> 1)] = zero;
      }
      if (a) {
        uint32_t o[Group<T>::kWords];
#pragma unroll
        for (int c = 0; c < Group<T>::kWords; ++c) o[c] = 0;
        store_groups<T, kVec>(a + row * I + g * 16, in ? min(16, I - g * 16) : 0, o, run);
      }
      continue;
    }
    float gate[16], up[16];
    vg.floats(gate);
    vu.floats(up);
    if (kept.codes) {                            // gate and up as blocks of one row of both
      store_mx(kept, row * 2, g, in, gate, vg.amax_bits());
      store_mx(kept, row * 2 + 1, g, in, up, vu.amax_bits());
    }
    const float weight = live ? s_rows.w[at] : 0.f;
    float f[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) f[c] = 0.f;
    if (live)
#pragma unroll
      for (int c = 0; c < 16; ++c) f[c] = gate[c] * sigmoid<T>(gate[c]) * up[c] * weight;
    if (q.codes) {
      float z[16];                               // past the row: zeros, also where the weight is not finite
#pragma unroll
      for (int c = 0; c < 16; ++c) z[c] = g * 16 + c < I ? f[c] : 0.f;
      store_mx(q, row, g, in, z, amax_bits16(z));
    }
    if (a) {
      uint32_t o[Group<T>::kWords];
      round16<T>(f, o);
      store_groups<T, kVec>(a + row * I + g * 16, in ? min(16, I - g * 16) : 0, o, run);
    }
  }
}

// P threads a row. The dots of a row's warps meet in shared memory.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4)
    swiglu_backward_kernel(const SwigluRows r, int rows, const T* __restrict__ d_a, int64_t stride, const Out8 kept,
                           const float* __restrict__ w, T* __restrict__ d_h, float* __restrict__ d_w, int P) {
  __shared__ Rows s_rows;
  __shared__ float s_dot[kMostRows][kThreads / 32];
  __shared__ alignas(16) T s_run[kVec ? 1 : kThreads / 32 * 512];
  T* run = kVec ? s_run : s_run + (threadIdx.x >> 5) * 512;
  // pairs that no row holds: masked slots
  if (d_w)
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; p < r.pairs;
         p += static_cast<int64_t>(gridDim.x) * kThreads)
      if (__ldg(r.slot + p) < 0) d_w[p] = 0.f;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows;
  look_up(s_rows, r, w, row0, rows);
  const int l = threadIdx.x % P, sub = threadIdx.x / P, subs = kThreads / P, I = r.I;
  const int groups = (I + 15) / 16;
  for (int i = sub; i < rows; i += subs) {
    const int64_t row = row0 + i;
    const bool live = s_rows.pair[i] >= 0;
    const float weight = s_rows.w[i];
    float dot = 0.f;
    for (int g = l; g - (l & 31) < groups; g += P) {
      float og[16], ou[16];
      if (live && g < groups) {
        const uint4* codes = reinterpret_cast<const uint4*>(kept.codes) + row * 2 * kept.groups + g;
        const uint8_t* sf = static_cast<const uint8_t*>(kept.sf) + row * 2 * kept.blocks + (g >> 1);
        Group<T> vd;
        vd.template load<kVec>(d_a + row * stride, g * 16, I);
        const uint4 cg = __ldg(codes), cu = __ldg(codes + kept.groups);
        const uint32_t sg = __ldg(sf), su = __ldg(sf + kept.blocks);
        float gate[16], up[16], d[16];
        decode16(cg, ue8m0_value(sg), gate);
        decode16(cu, ue8m0_value(su), up);
        vd.floats(d);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float s = sigmoid<T>(gate[c]);
          const float silu = gate[c] * s;
          if (kVec || g * 16 + c < I) dot = fmaf(d[c] * silu, up[c], dot);
          const float dw = d[c] * weight;
          og[c] = dw * up[c] * (s * (1.0f + gate[c] * (1.0f - s)));
          ou[c] = dw * silu;
        }
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) og[c] = ou[c] = 0.f;
      }
      uint32_t o[Group<T>::kWords];
      T* at = d_h + row * 2 * I + g * 16;
      const int n = row < r.rows ? min(16, I - g * 16) : 0;
      round16<T>(og, o);
      store_groups<T, kVec>(at, n, o, run);
      round16<T>(ou, o);
      store_groups<T, kVec>(at + I, n, o, run);
    }
    if (d_w) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if ((threadIdx.x & 31) == 0) s_dot[i][l >> 5] = dot;
    }
  }
  if (!d_w) return;
  __syncthreads();
  for (int i = threadIdx.x; i < rows; i += kThreads)
    if (s_rows.pair[i] >= 0) {
      float v = 0.f;
      for (int k = 0; k < P / 32; ++k) v += s_dot[i][k];
      d_w[s_rows.pair[i]] = v;
    }
}

// Rows of a CTA: about four groups of 16 columns a thread, as many as share the rows out evenly over whole rounds of four
// CTAs an SM. (Forward / back with cold caches, us: 13248 rows of 2048 columns 45 / 46, by two or eight groups 46 / 47 and
// 44 / 44; 4093 of 2731 in fp16 32 / 33, with four groups whatever the rounds 35 / 38; 3000 of 4096 24 / 24, 27 / 27.)
int cta_rows(int64_t rows, int groups) {
  const int64_t slots = 4 * dev_info().sms, most = slots * 4 * kThreads / groups;          // rows of a round
  const int64_t rounds = most > 0 ? (2 * rows + most) / (2 * most) : 1;
  const int64_t ctas = slots * (rounds > 0 ? rounds : 1), n = (rows + ctas - 1) / ctas;
  return static_cast<int>(n < 1 ? 1 : n > kMostRows ? kMostRows : n);
}

Out8 kept_rows(void* codes, void* sf, int I) {
  return Out8{kMx, static_cast<uint8_t*>(codes), sf, groups8(I, kMx), blocks8(I, kMx)};
}

}  // namespace

cudaError_t launch_swiglu(const SwigluRows& r, int dtype, const void* h, int64_t stride, const float* w, void* a,
                          void* codes, void* sf, void* kept, void* kept_sf, cudaStream_t s) {
  const int elem = dtype_size(dtype);
  const bool vec = whole_groups(h, stride * elem, r.I) && whole_groups(a, static_cast<int64_t>(r.I) * elem, r.I);
  const int rows = cta_rows(r.rows, groups8(r.I, kMx));
  const unsigned grid = static_cast<unsigned>((r.rows + rows - 1) / rows);
  const Out8 q = kept_rows(codes, sf, r.I), k = kept_rows(kept, kept_sf, r.I);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* p = static_cast<const T*>(h);
    T* o = static_cast<T*>(a);
    if (vec) swiglu_kernel<T, true><<<grid, kThreads, 0, s>>>(r, rows, p, stride, w, o, q, k);
    else swiglu_kernel<T, false><<<grid, kThreads, 0, s>>>(r, rows, p, stride, w, o, q, k);
    return cudaGetLastError();
  });
}

cudaError_t launch_swiglu_backward(const SwigluRows& r, int dtype, const void* d_a, int64_t stride, const void* kept,
                                   const void* kept_sf, const float* w, void* d_h, float* d_w, cudaStream_t s) {
  const int elem = dtype_size(dtype);
  const bool vec = whole_groups(d_a, stride * elem, r.I) && whole_groups(d_h, static_cast<int64_t>(r.I) * elem, r.I);
  const int P = row_threads((r.I + 15) / 16, 1, kThreads);
  int rows = cta_rows(r.rows, (r.I + 15) / 16);
  const int subs = kThreads / P;
  rows = rows < subs ? subs : rows / subs * subs;
  const unsigned grid = static_cast<unsigned>((r.rows + rows - 1) / rows);
  const Out8 k = kept_rows(const_cast<void*>(kept), const_cast<void*>(kept_sf), r.I);
  return with_dtype(dtype, [&](auto tag) {
    using T = decltype(tag);
    const T* p = static_cast<const T*>(d_a);
    T* o = static_cast<T*>(d_h);
    if (vec) swiglu_backward_kernel<T, true><<<grid, kThreads, 0, s>>>(r, rows, p, stride, k, w, o, d_w, P);
    else swiglu_backward_kernel<T, false><<<grid, kThreads, 0, s>>>(r, rows, p, stride, k, w, o, d_w, P);
    return cudaGetLastError();
  });
}

}  // namespace mm

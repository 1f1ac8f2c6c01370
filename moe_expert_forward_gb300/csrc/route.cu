// The router: top-k of each token's logits with their weights, and the gradient
// of those weights with respect to the logits.
//
//   key_e = l_e, or sigmoid(l_e) + bias_e; the K largest keys of a row in
//   descending order, equal keys by ascending expert.  -inf and NaN logits are
//   never chosen; a row with fewer than K others ends in index -1, weight 0.
//   softmax: p_e = exp(l_e - m) / sum_j exp(l_j - m); sigmoid: p_e = 1 / (1 + exp(-l_e)).
//   w_k = scale * p_k / z, z = 1, or with renorm the sum of the chosen p (softmax)
//   or that sum + 1e-20 (sigmoid, whose scores may all underflow).
//
// Gradient, g_k = scale * dw_k on the chosen k, d_k = dL/dp_k:
//   d_k = g_k, or with renorm (g_k - sum_j g_j p_j / z) / z;
//   sigmoid: dl_k = d_k p_k (1 - p_k);  softmax: dl_e = p_e (d_e - sum_j d_j p_j), d_e = 0 where
//   e is not chosen.  Under softmax with renorm the p cancel to q_k = exp(l_k - m) / sum of the
//   chosen: dl_k = q_k (g_k - sum_j g_j q_j), and every other expert's gradient is zero.
//
// A group of G lanes takes a row and keeps its logits in registers, P consecutive
// ones per access, so a row is read once.  A round of the choice is the largest key
// of the lane, a reduction over the group for the key and one for the lowest
// expert that holds it; where the logits have 16 bits and there is no bias, key and
// expert fit one word, all words differ, one reduction does both, and a round takes
// the largest word below the last choice, one add-and-max per logit: of differences
// k - last mod 2^32, those of words below `last` are the larger ones.  Two forms:
//   G = 32, P = 1  a warp a row: few rows, where the latency of one row counts
//   G = 8, P = 2   four rows a warp: many rows; the reductions and the work at a
//                  row's end are shared by four
// What bounds many rows (65536 of 160 read 21 MB, 3 us): the choice, the integer pipe and the
// issue slots while an SM is busy (67 % of them used; most warps that do not issue wait for
// that pipe or for their turn), with a bias the chains of dependent instructions (96 registers
// a thread leave 28 % of the warps); the gradient, the latency of its loads.
//
// The softmax's exponentials of differences x <= 0 are 2^t by the fast unit, t = x log2 e
// rounded, times 1 + c for what the rounding left out: e^x = 2^t e^c, c = x - t ln 2, |c| < 2^-16
// where the result is not 0, so that 1 + c is e^c to fp32.  That stays within 4 units in the
// last place however far a logit lies below the largest (without c: 15 at a distance of 40, 30 at
// 80) and is shorter than expf.  The sigmoid, whose sums with the bias decide the choice, takes
// expf and the IEEE division.
#include <type_traits>

#include "rowtypes.cuh"

namespace mm {
namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

// Reductions over each group of G consecutive lanes; the whole warp takes part.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
    return v;
  }
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) { return ~group_max<G>(~v); }

// Unsigned integers in the order of the floats (-0 counts as +0); -inf and NaN, never chosen, are 0.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (!(f > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o >> 31) ? (o ^ 0x80000000u) : ~o);
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  const uint32_t o = group_max<G>(ordered(v));
  return o ? unordered(o) : -INFINITY;
}

// Key and expert of a 16-bit logit in one word: the float's bits in order on top, 0xFFFF - e below, so that the
// larger of two equal logits' words is the lower expert's. v is no NaN and no -0 (clean).
template <typename T>
__device__ __forceinline__ uint32_t packed_key(T v, uint32_t rest) {
  uint32_t u;
  if constexpr (std::is_same<T, __half>::value) u = static_cast<uint32_t>(__half_as_ushort(v)) << 16;
  else u = static_cast<uint32_t>(__bfloat16_as_ushort(v)) << 16;
  const uint32_t o = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return (o & 0xFFFF0000u) | rest;
}
// words of -inf, which is never chosen, are below this
template <typename T>
__device__ __forceinline__ uint32_t first_packed() {
  return std::is_same<T, __half>::value ? 0x04000000u : 0x00800000u;
}
template <typename T>
__device__ __forceinline__ float packed_value(uint32_t key) {
  uint32_t b = key >> 16;
  b = (b & 0x8000u) ? (b ^ 0x8000u) : (~b & 0xFFFFu);
  if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
  else return __uint_as_float(b << 16);
}
// NaN -> -inf, -0 -> +0
template <typename T>
__device__ __forceinline__ T clean(T v) {
  if constexpr (sizeof(T) == 4) return fmaxf(v + 0.0f, -INFINITY);
  else return __hmax(__hadd(v, from_float<T>(0.f)), from_float<T>(-INFINITY));
}
template <typename T>
__device__ __forceinline__ void clean2(T* v) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 r = __hmax2(__hadd2(__halves2half2(v[0], v[1]), __float2half2_rn(0.f)), __float2half2_rn(-INFINITY));
    v[0] = __low2half(r);
    v[1] = __high2half(r);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    const __nv_bfloat162 r = __hmax2(__hadd2(__halves2bfloat162(v[0], v[1]), __float2bfloat162_rn(0.f)),
                                     __float2bfloat162_rn(-INFINITY));
    v[0] = __low2bfloat16(r);
    v[1] = __high2bfloat16(r);
  } else {
    v[0] = clean(v[0]);
    v[1] = clean(v[1]);
  }
}

// e^x of x <= 0; results below fp32's normal range are 0, NaN stays
__device__ __forceinline__ float exp_below(float x) {
  float t, r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(-128.0f));   // -inf and what overflows t: 0 all the same
  t = x * 1.44269504f;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return fmaf(r, fmaf(t, -0.693147181f, x), r);
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

template <typename T>
__device__ __forceinline__ float load_logit(const T* row, int e, int E) {
  const float x = e < E ? to_float(row[e]) : -INFINITY;
  return x == x ? x : -INFINITY;
}

// A lane's V accesses of P logits: value i of access j is expert (j G + lane) P + i. E is a multiple of P.
template <typename T, int V, int G, int P>
__device__ __forceinline__ void load_row(const T* row, int lane, int E, T (&v)[V * P]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * G + lane) * P;
    Vec<T, P> a;
#pragma unroll
    for (int i = 0; i < P; ++i) a.v[i] = from_float<T>(-INFINITY);
    if (c < E) a = *reinterpret_cast<const Vec<T, P>*>(row + c);
    if constexpr (P == 2) clean2(a.v);
    else a.v[0] = clean(a.v[0]);
#pragma unroll
    for (int i = 0; i < P; ++i) v[j * P + i] = a.v[i];
  }
}

template <typename T, int V, int G, int P, bool kBias>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_kernel(const T* __restrict__ logits, int64_t stride, int T_, int E, int K, const float* __restrict__ bias,
                 int score, int renorm, float scale, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr bool kPacked = sizeof(T) == 2 && !kBias;
  constexpr int N = V * P;
  const int lane = threadIdx.x % G;
  const int t0 = blockIdx.x * (32 * kRouteWarps / G) + threadIdx.x / G;
  if (G == 32 && t0 >= T_) return;
  const int t = min(t0, T_ - 1);                  // a group past the last row repeats it and stores nothing
  const T* row = logits + t * stride;
  const bool all = score == MM_MOE_SCORE_SOFTMAX && !renorm;   // the sum runs over every expert
  T v[N];
  load_row<T, V, G, P>(row, lane, E, v);
  uint32_t key[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int e = (n / P * G + lane) * P + n % P;
    if constexpr (kPacked) key[n] = packed_key(v[n], static_cast<uint32_t>(0xFFFF - e));
    else if constexpr (kBias)
      key[n] = to_float(v[n]) > -INFINITY ? ordered(sigmoid(to_float(v[n])) + __ldg(bias + (e < E ? e : 0))) : 0u;
    else key[n] = ordered(to_float(v[n]));
  }
  // lane k ends up with the k-th choice
  int my_e = -1;
  uint32_t my_key = 0, first = 0, last = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t top = 0;
    unsigned at;
    if constexpr (kPacked) {
      uint32_t best = 0;
#pragma unroll
      for (int n = 0; n < N; ++n) best = __viaddmax_u32(key[n], 0u - last, best);
      top = group_max<G>(best) + last;
      last = top;
      if (top < first_packed<T>()) top = 0;         // and from here on every round ends here: all words below are -inf's
      at = 0xFFFFu - (top & 0xFFFFu);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) top = max(top, key[n]);
      top = group_max<G>(top);
      at = 0xffffffffu;
#pragma unroll
      for (int n = N - 1; n >= 0; --n)
        at = key[n] == top ? static_cast<unsigned>((n / P * G + lane) * P + n % P) : at;
      at = group_min<G>(at);
#pragma unroll
      for (int n = 0; n < N; ++n)
        key[n] = at == static_cast<unsigned>((n / P * G + lane) * P + n % P) ? 0u : key[n];
    }
    if (k == 0) first = top;
    if (G == 32 && top == 0) break;
    if (lane == k && top != 0) {
      my_e = static_cast<int>(at);
      my_key = top;
    }
  }
  // the chosen logits: from their keys, or read again where the key holds the bias
  auto value = [&](uint32_t k) { return kPacked ? packed_value<T>(k) : unordered(k); };
  float p = 0.f;
  if (score == MM_MOE_SCORE_SOFTMAX) {
    const float m = first ? value(first) : 0.f;   // the first choice is the row's largest logit
    if (my_e >= 0) p = exp_below(value(my_key) - m);
    if (all) {
      float z = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) z += exp_below(to_float(v[n]) - m);
      z = group_sum<G>(z);
      if (my_e >= 0) p = __fdiv_rn(p, z);
    }
  } else if (my_e >= 0) {
    p = sigmoid(kBias ? to_float(row[my_e]) : value(my_key));
  }
  if (renorm) p = __fdiv_rn(p, group_sum<G>(p) + 1e-20f);
  if (lane < K && t0 < T_) {
    topk_idx[static_cast<int64_t>(t) * K + lane] = my_e;
    // 0 where there is no choice, also where an infinite logit made the sum, and so p, NaN
    topk_w[static_cast<int64_t>(t) * K + lane] = my_e >= 0 ? p * scale : 0.f;
  }
}

template <typename T, int V, int G, int P>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_kernel(const T* __restrict__ logits, int64_t stride, const int32_t* __restrict__ topk_idx,
                          const float* __restrict__ d_w, int T_, int E, int K, int score, int renorm, float scale,
                          T* __restrict__ d_logits, int64_t d_stride) {
  constexpr int N = V * P;
  const int lane = threadIdx.x % G;
  const int t0 = blockIdx.x * (32 * kRouteWarps / G) + threadIdx.x / G;
  if (G == 32 && t0 >= T_) return;
  const int t = min(t0, T_ - 1);
  const T* row = logits + t * stride;
  T* d_row = d_logits + t * d_stride;
  const bool all = score == MM_MOE_SCORE_SOFTMAX && !renorm;
  T raw[N];
  if (all) load_row<T, V, G, P>(row, lane, E, raw);
  int e = -1;
  float g = 0.f, x = -INFINITY;
  if (lane < K) {
    e = topk_idx[static_cast<int64_t>(t) * K + lane];
    if (e < 0 || e >= E) e = -1;
    if (e >= 0) {
      x = load_logit(row, e, E);
      g = scale * d_w[static_cast<int64_t>(t) * K + lane];
    }
  }
  float d;                                          // lane k: the gradient of choice k's logit
  float v[N], r = 0.f;                              // the others': v r
  if (all) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = to_float(raw[n]);
      m = fmaxf(m, v[n]);
    }
    m = group_max<G>(m);
    if (m == -INFINITY) m = 0.f;                    // a row without logits: every exp is 0
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = exp_below(v[n] - m);
      z += v[n];
    }
    z = group_sum<G>(z);
    const float rz = z == 0.f ? 0.f : __fdiv_rn(1.0f, z);
    const float p = e >= 0 ? exp_below(x - m) * rz : 0.f;
    const float s = group_sum<G>(g * p);
    d = p * (g - s);
    r = -rz * s;
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = 0.f;
    if (score == MM_MOE_SCORE_SOFTMAX) {
      const float m = group_max<G>(x);
      const float q0 = e >= 0 ? exp_below(x - m) : 0.f;
      const float z = group_sum<G>(q0);
      const float q = e >= 0 ? __fdiv_rn(q0, z) : 0.f;
      d = q * (g - group_sum<G>(g * q));
    } else {
      const float p = e >= 0 ? sigmoid(x) : 0.f;
      float dp = g;
      if (renorm) {
        const float z = group_sum<G>(p) + 1e-20f;
        dp = __fdiv_rn(g - group_sum<G>(g * __fdiv_rn(p, z)), z);
      }
      d = dp * p * (1.0f - p);
    }
  }
  if (t0 < T_) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * G + lane) * P;
      Vec<T, P> o;
#pragma unroll
      for (int i = 0; i < P; ++i) o.v[i] = from_float<T>(v[j * P + i] * r);
      if (c < E) *reinterpret_cast<Vec<T, P>*>(d_row + c) = o;
    }
  }
  __syncwarp();                                     // the row's other entries first, then the chosen ones over them
  if (e >= 0 && t0 < T_) d_row[e] = from_float<T>(d);
}

template <int V, int G, int P>
struct Form {
  static constexpr int v = V, g = G, p = P;
  static unsigned grid(int T) { return static_cast<unsigned>((T + 32 * kRouteWarps / G - 1) / (32 * kRouteWarps / G)); }
};

// Four rows a warp from so many rows on; below, the rows do not fill the SMs' warps. Measured, us forward with cold
// caches, four rows a warp / a warp a row, softmax with renorm, bf16: 65536x160 top-4 12.8 / 21.1, 16384x256 top-8
// 8.5 / 9.2, 8192x256 top-8 5.6 / 5.7, 4096x256 top-8 4.0 / 3.5; fp32: 65536x160 21.6 / 30.8, 16384x256 top-8 15.8 /
// 16.1, 8192x256 top-8 10.3 / 9.3.
template <typename T>
constexpr int kManyRows = sizeof(T) == 2 ? 8192 : 16384;

// With a bias every logit is a sigmoid's argument and a lane has four times as many of them one after another: more
// rows, and fewer experts, have to make up for it. The same figures, fp32 (bf16 the same within 5 %): 65536x64 top-6
// 18.1 / 27.1, 16384x64 6.9 / 8.6, 8192x64 5.1 / 4.9; 65536x128 top-4 29.0 / 32.1, 32768x128 17.2 / 17.3, 16384x128
// 11.3 / 10.0; 65536x160 39.1 / 39.6, 16384x160 13.9 / 12.0; 65536x256 top-8 79.7 / 70.3, 8192x256 16.1 / 12.4.
template <typename T>
bool many_rows(int rows, int E, bool bias) {
  if (bias) return rows >= 16384 && E <= 160 && rows >= 256 * E;
  return rows >= kManyRows<T>;
}

// f with the form that takes E logits a row; `bits` are the row pitches' and addresses' in bytes, or-ed.
template <typename T, typename F>
cudaError_t with_form(int rows, int E, int K, bool bias, uint64_t bits, F f) {
  if (many_rows<T>(rows, E, bias) && K <= 8 && E <= 256 && E % 2 == 0 && bits % (2 * sizeof(T)) == 0) {
  const int n = (E + 15) / 16;
    if (n <= 2) return f(Form<2, 8, 2>{});
    if (n <= 4) return f(Form<4, 8, 2>{});
    if (n <= 6) return f(Form<6, 8, 2>{});
    if (n <= 8) return f(Form<8, 8, 2>{});
    if (n <= 10) return f(Form<10, 8, 2>{});
    if (n <= 12) return f(Form<12, 8, 2>{});
    return f(Form<16, 8, 2>{});
  }
  const int n = (E + 31) / 32;
  if (n <= 1) return f(Form<1, 32, 1>{});
  if (n <= 2) return f(Form<2, 32, 1>{});
  if (n <= 4) return f(Form<4, 32, 1>{});
  if (n <= 6) return f(Form<6, 32, 1>{});
  if (n <= 8) return f(Form<8, 32, 1>{});
  if (n <= 12) return f(Form<12, 32, 1>{});
  if (n <= 16) return f(Form<16, 32, 1>{});
  if (n <= 24) return f(Form<24, 32, 1>{});
  return f(Form<32, 32, 1>{});
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.logits) | static_cast<uint64_t>(a.stride) * sizeof(T);
    return with_form<T>(a.T, a.E, a.K, a.bias != nullptr, bits, [&](auto form) {
      using W = decltype(form);
      auto kernel = a.bias ? route_kernel<T, W::v, W::g, W::p, true> : route_kernel<T, W::v, W::g, W::p, false>;
      kernel<<<W::grid(a.T), 32 * kRouteWarps, 0, s>>>(static_cast<const T*>(a.logits), a.stride, a.T, a.E, a.K,
                                                       a.bias, a.score, a.renorm, a.scale, a.topk_idx, a.topk_w);
      return cudaGetLastError();
    });
  });
}

cudaError_t launch_route_backward(const RouteArgs& a, const int32_t* topk_idx, const float* d_w, void* d_logits,
                                  int64_t d_stride, cudaStream_t s) {
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(d_logits) |
                          static_cast<uint64_t>(a.stride | d_stride) * sizeof(T);
    return with_form<T>(a.T, a.E, a.K, a.bias != nullptr, bits, [&](auto form) {
      using W = decltype(form);
      route_backward_kernel<T, W::v, W::g, W::p><<<W::grid(a.T), 32 * kRouteWarps, 0, s>>>(
          static_cast<const T*>(a.logits), a.stride, topk_idx, d_w, a.T, a.E, a.K, a.score, a.renorm, a.scale,
          static_cast<T*>(d_logits), d_stride);
      return cudaGetLastError();
    });
  });
}

}  // namespace mm

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
// One warp takes one row and keeps its logits in registers, expert e in lane
// e % 32, so a row is read once.  A round of the choice is the largest key of the
// lane, one reduction over the warp for the key and one for the lowest expert
// that holds it; where the logits have 16 bits and there is no bias, key and
// expert fit one word and one reduction does both.  What bounds it is the issue of
// these instructions (65536 rows of 160 read 21 MB, 3 us), so nothing is kept or
// computed for more than the ceil(E / 32) logits a lane has.
//
// The softmax takes exp as 2^(x log2 e) by the fast unit, a few units in the last
// place of fp32 off for the arguments (<= 0) that matter; the sigmoid, whose sums
// with the bias decide the choice, takes expf and the IEEE division.
#include <type_traits>

#include "rowtypes.cuh"

namespace mm {
namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Unsigned integers in the order of the floats (-0 counts as +0); -inf and NaN, never chosen, are 0.
__device__ __forceinline__ uint32_t ordered(float f) {
  if (!(f > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o >> 31) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ float warp_max(float v) {
  const uint32_t o = __reduce_max_sync(kAll, ordered(v));
  return o ? unordered(o) : -INFINITY;
}

// Key and expert of a 16-bit logit in one word: the float's bits in order on top, 0xFFFF - e below, so that the
// larger of two equal logits' words is the lower expert's; 0 where it is never chosen.
template <typename T>
__device__ __forceinline__ uint32_t packed_key(T v, int e) {
  const float f = to_float(v);
  if (!(f > -INFINITY)) return 0u;
  uint32_t b;
  if constexpr (std::is_same<T, __half>::value) b = __half_as_ushort(v);
  else b = __bfloat16_as_ushort(v);
  b = b == 0x8000u ? 0u : b;
  b = (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
  return b << 16 | static_cast<uint32_t>(0xFFFF - e);
}
template <typename T>
__device__ __forceinline__ float packed_value(uint32_t key) {
  uint32_t b = key >> 16;
  b = (b & 0x8000u) ? (b ^ 0x8000u) : (~b & 0xFFFFu);
  if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
  else return __uint_as_float(b << 16);
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

template <typename T>
__device__ __forceinline__ float load_logit(const T* row, int e, int E) {
  const float x = e < E ? to_float(row[e]) : -INFINITY;
  return x == x ? x : -INFINITY;
}

template <typename T, int VPL, bool kBias>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_kernel(const T* __restrict__ logits, int64_t stride, int T_, int E, int K, const float* __restrict__ bias,
                 int score, int renorm, float scale, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  constexpr bool kPacked = sizeof(T) == 2 && !kBias;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= T_) return;
  const T* row = logits + t * stride;
  const bool all = score == MM_MOE_SCORE_SOFTMAX && !renorm;   // the sum runs over every expert
  float x[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    x[j] = load_logit(row, e, E);
    if constexpr (kPacked) key[j] = e < E ? packed_key(row[e], e) : 0u;
    else if constexpr (kBias) key[j] = x[j] == -INFINITY ? 0u : ordered(sigmoid(x[j]) + __ldg(bias + (e < E ? e : 0)));
    else key[j] = ordered(x[j]);
  }
  // lane k ends up with the k-th choice
  int my_e = -1;
  uint32_t my_key = 0, first = 0;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    if (top == 0) break;
    if (k == 0) first = top;
    unsigned at;
    if constexpr (kPacked) {
      at = 0xFFFFu - (top & 0xFFFFu);
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = key[j] == top ? 0u : key[j];
    } else {
      at = 0xffffffffu;
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j) at = key[j] == top ? static_cast<unsigned>(j * 32 + lane) : at;
      at = __reduce_min_sync(kAll, at);
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = at == static_cast<unsigned>(j * 32 + lane) ? 0u : key[j];
    }
    if (lane == k) {
      my_e = static_cast<int>(at);
      my_key = top;
    }
  }
  // the chosen logits: from their keys, or read again where the key holds the bias
  auto value = [&](uint32_t k) { return kPacked ? packed_value<T>(k) : unordered(k); };
  float p = 0.f;
  if (score == MM_MOE_SCORE_SOFTMAX) {
    const float m = value(first);                 // the first choice is the row's largest logit
    if (my_e >= 0) p = __expf(value(my_key) - m);
    if (all) {
      float z = 0.f;
      if (first) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) z += __expf(x[j] - m);
      }
      z = warp_sum(z);
      if (my_e >= 0) p = __fdiv_rn(p, z);
    }
  } else if (my_e >= 0) {
    p = sigmoid(kBias ? to_float(row[my_e]) : value(my_key));
  }
  if (renorm) p = __fdiv_rn(p, warp_sum(p) + 1e-20f);
  if (lane < K) {
    topk_idx[static_cast<int64_t>(t) * K + lane] = my_e;
    topk_w[static_cast<int64_t>(t) * K + lane] = p * scale;
  }
}

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_kernel(const T* __restrict__ logits, int64_t stride, const int32_t* __restrict__ topk_idx,
                          const float* __restrict__ d_w, int T_, int E, int K, int score, int renorm, float scale,
                          T* __restrict__ d_logits, int64_t d_stride) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= T_) return;
  const T* row = logits + t * stride;
  T* d_row = d_logits + t * d_stride;
  const bool all = score == MM_MOE_SCORE_SOFTMAX && !renorm;
  float v[VPL];
  if (all) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) v[j] = load_logit(row, j * 32 + lane, E);
  }
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
  if (all) {
    float m = v[0], z = 0.f;
#pragma unroll
    for (int j = 1; j < VPL; ++j) m = fmaxf(m, v[j]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;                    // a row without logits: every exp is 0
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      v[j] = __expf(v[j] - m);
      z += v[j];
    }
    z = warp_sum(z);
    const float rz = z == 0.f ? 0.f : __fdiv_rn(1.0f, z);
    const float p = e >= 0 ? __expf(x - m) * rz : 0.f;
    const float s = warp_sum(g * p);
    d = p * (g - s);
    const float r = -rz * s;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = j * 32 + lane;
      if (c < E) d_row[c] = from_float<T>(v[j] * r);
    }
  } else {
    if (score == MM_MOE_SCORE_SOFTMAX) {
      const float m = warp_max(x);
      const float q0 = e >= 0 ? __expf(x - m) : 0.f;
      const float z = warp_sum(q0);
      const float q = e >= 0 ? __fdiv_rn(q0, z) : 0.f;
      d = q * (g - warp_sum(g * q));
    } else {
      const float p = e >= 0 ? sigmoid(x) : 0.f;
      float dp = g;
      if (renorm) {
        const float z = warp_sum(p) + 1e-20f;
        dp = __fdiv_rn(g - warp_sum(g * __fdiv_rn(p, z)), z);
      }
      d = dp * p * (1.0f - p);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = j * 32 + lane;
      if (c < E) d_row[c] = from_float<T>(0.f);
    }
  }
  __syncwarp();                                     // the row's other entries first, then the chosen ones over them
  if (e >= 0) d_row[e] = from_float<T>(d);
}

// f with the logits a lane holds, ceil(E / 32) rounded up to a width that is built
template <typename F>
cudaError_t with_width(int E, F f) {
  const int n = (E + 31) / 32;
  if (n <= 1) return f(std::integral_constant<int, 1>{});
  if (n <= 2) return f(std::integral_constant<int, 2>{});
  if (n <= 3) return f(std::integral_constant<int, 3>{});
  if (n <= 4) return f(std::integral_constant<int, 4>{});
  if (n <= 5) return f(std::integral_constant<int, 5>{});
  if (n <= 6) return f(std::integral_constant<int, 6>{});
  if (n <= 8) return f(std::integral_constant<int, 8>{});
  if (n <= 12) return f(std::integral_constant<int, 12>{});
  if (n <= 16) return f(std::integral_constant<int, 16>{});
  if (n <= 24) return f(std::integral_constant<int, 24>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.T + kRouteWarps - 1) / kRouteWarps);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return with_width(a.E, [&](auto w) {
      constexpr int W = decltype(w)::value;
      auto kernel = a.bias ? route_kernel<T, W, true> : route_kernel<T, W, false>;
      kernel<<<grid, 32 * kRouteWarps, 0, s>>>(static_cast<const T*>(a.logits), a.stride, a.T, a.E, a.K, a.bias,
                                               a.score, a.renorm, a.scale, a.topk_idx, a.topk_w);
      return cudaGetLastError();
    });
  });
}

cudaError_t launch_route_backward(const RouteArgs& a, const int32_t* topk_idx, const float* d_w, void* d_logits,
                                  int64_t d_stride, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.T + kRouteWarps - 1) / kRouteWarps);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return with_width(a.E, [&](auto w) {
      route_backward_kernel<T, decltype(w)::value><<<grid, 32 * kRouteWarps, 0, s>>>(
          static_cast<const T*>(a.logits), a.stride, topk_idx, d_w, a.T, a.E, a.K, a.score, a.renorm, a.scale,
          static_cast<T*>(d_logits), d_stride);
      return cudaGetLastError();
    });
  });
}

}  // namespace mm

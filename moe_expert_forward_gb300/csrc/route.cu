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
// e % 32, so a row is read once.  Each of the K rounds is two warp reductions:
// the largest key, then the lowest expert that holds it.
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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Unsigned integers in the order of the floats (-0 counts as +0); 0 for a key that is never chosen.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, 1.0f + expf(-x)); }

template <typename T>
__device__ __forceinline__ float load_logit(const T* row, int e, int E) {
  const float x = e < E ? to_float(row[e]) : -INFINITY;
  return x == x ? x : -INFINITY;
}

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_kernel(const T* __restrict__ logits, int64_t stride, int T_, int E, int K, const float* __restrict__ bias,
                 int score, int renorm, float scale, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= T_) return;
  const T* row = logits + t * stride;
  float x[VPL];
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) x[j] = load_logit(row, j * 32 + lane, E);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = j * 32 + lane;
    float k = x[j];
    if (bias && e < E) k = sigmoid(k) + __ldg(bias + e);
    key[j] = (x[j] == -INFINITY || !(k == k)) ? 0u : ordered(k);
  }
  // lane k ends up with the k-th choice
  int my_e = -1;
  float my_x = -INFINITY;
  for (int k = 0; k < K; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < VPL; ++j) best = max(best, key[j]);
    const uint32_t top = __reduce_max_sync(kAll, best);
    if (top == 0) break;
    unsigned at = 0xffffffffu;
#pragma unroll
    for (int j = VPL - 1; j >= 0; --j)
      if (key[j] == top) at = j * 32 + lane;
    at = __reduce_min_sync(kAll, at);
    float xv = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (at == static_cast<unsigned>(j * 32 + lane)) {
        xv = x[j];
        key[j] = 0;
      }
    xv = __shfl_sync(kAll, xv, at & 31);
    if (lane == k) {
      my_e = static_cast<int>(at);
      my_x = xv;
    }
  }
  float p;
  if (score == MM_MOE_SCORE_SOFTMAX) {
    const float m = __shfl_sync(kAll, my_x, 0);   // the first choice is the row's largest logit
    p = my_e >= 0 ? expf(my_x - m) : 0.f;
    if (!renorm) {
      float z = 0.f;
      if (m != -INFINITY) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) z += expf(x[j] - m);
      }
      z = warp_sum(z);
      if (my_e >= 0) p = __fdiv_rn(p, z);
    }
  } else {
    p = my_e >= 0 ? sigmoid(my_x) : 0.f;
  }
  if (renorm) {
    const float z = warp_sum(p) + 1e-20f;
    p = __fdiv_rn(p, z);
  }
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
  if (score == MM_MOE_SCORE_SOFTMAX && !renorm) {
    float v[VPL];
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      v[j] = load_logit(row, j * 32 + lane, E);
      m = fmaxf(m, v[j]);
    }
    m = warp_max(m);
    if (m != -INFINITY) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        v[j] = expf(v[j] - m);
        z += v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) v[j] = 0.f;
    }
    z = warp_sum(z);
    const float rz = z > 0.f ? __fdiv_rn(1.0f, z) : (z == z ? 0.f : z);
    const float p = e >= 0 ? expf(x - m) * rz : 0.f;
    const float s = warp_sum(g * p);
    d = p * (g - s);
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = j * 32 + lane;
      if (c < E) d_row[c] = from_float<T>(-(v[j] * rz) * s);
    }
  } else {
    if (score == MM_MOE_SCORE_SOFTMAX) {
      const float m = warp_max(x);
      const float q0 = e >= 0 ? expf(x - m) : 0.f;
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

// registers a lane holds: the smallest bucket of logits that covers E
template <typename F>
cudaError_t with_width(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.T + kRouteWarps - 1) / kRouteWarps);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return with_width(a.E, [&](auto w) {
      route_kernel<T, decltype(w)::value><<<grid, 32 * kRouteWarps, 0, s>>>(
          static_cast<const T*>(a.logits), a.stride, a.T, a.E, a.K, a.bias, a.score, a.renorm, a.scale, a.topk_idx,
          a.topk_w);
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

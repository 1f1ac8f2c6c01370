// Tokens sorted by expert and back.  The routing kernels give every (token, k)
// pair a row (slot, -1 where masked) of a pool whose segments are padded to
// whole blocks, and every pool row its pair (src, -1 on padding).
//   permute            rows[slot[t,k]] = x[t]; padding rows = 0
//   unpermute          y[t] = sum_k w[t,k] rows[slot[t,k]]
//   unpermute backward d_rows[slot[t,k]] = w[t,k] dy[t], padding rows = 0;
//                      dw[t,k] = <dy[t], rows[slot[t,k]]>
// (permute's gradient is unpermute without weights: dx[t] = sum_k d_rows[slot[t,k]].)
// Sums are fp32 in ascending k (a dot: fp32 in a fixed tree), rounded once.
//
// All three move bytes and little else: a token's row is read once and its K
// pool rows are written (permute), or K rows are read and one written; memory
// bounds them.  Each token belongs to a group of threads as wide as its row has
// accesses of 32 or 16 bytes (8 to the CTA's threads), so short rows share a CTA and
// long rows get all of it; the pool rows of a token are independent loads in flight
// together.  Measured: permute 8192x7168 bf16 top-6 138 us (903 MB with the padding,
// 6.5 TB/s), its gradient 128 us (821 MB, 6.4), unpermute 8192x4096 top-8 94 us (604
// MB, 6.4), its gradients 183 us (1157 MB, 6.3).
#include "rowtypes.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;                // permute, unpermute
constexpr int kBackThreads = 128;            // the gradients (8192x4096 top-8: 190 us, with 256 threads 205)
constexpr int kPadRows = 8;                  // pool rows a padding CTA looks at
constexpr int kMaxGroups = kThreads / 8;     // tokens of one CTA at most

// Zeroes the padding among the 8 pool rows from 8 g on: rows whose src is -1, and rows past the last block, whose
// src the routing never wrote. The CTAs that do this come first in the grid and are many and small: the rows past the
// last block lie together, and in CTAs of 32 rows at the grid's end they were its tail (permute 8192x7168: 152 us then,
// 132 without zeroing any).
// zero_row(r, lane) zeroes one row with a warp.
template <typename F>
__device__ __forceinline__ void each_padding_row(const int32_t* __restrict__ src, const int32_t* __restrict__ blk_off,
                                                 int E, int block_m, int64_t num_rows, int64_t g, F zero_row) {
  const int64_t end = static_cast<int64_t>(__ldg(blk_off + E)) * block_m;
  for (int64_t r = g * kPadRows + (threadIdx.x >> 5); r < (g + 1) * kPadRows && r < num_rows; r += blockDim.x / 32)
    if (r >= end || __ldg(src + r) < 0) zero_row(r, static_cast<int>(threadIdx.x & 31));
}
template <int B>
__device__ __forceinline__ void zero_padding(const int32_t* __restrict__ src, const int32_t* __restrict__ blk_off, int E,
                                             int block_m, char* __restrict__ rows, int64_t num_rows, int64_t pitch,
                                             int64_t g) {
  using V = Vec<char, B>;
  V zero;
  memset(&zero, 0, B);
  each_padding_row(src, blk_off, E, block_m, num_rows, g, [&](int64_t r, int lane) {
    V* d = reinterpret_cast<V*>(rows + r * pitch);
    for (int i = lane; i < static_cast<int>(pitch / B); i += 32) store_once(d + i, zero);
  });
}
template <typename T>
__device__ __forceinline__ void zero_padding_any(const int32_t* __restrict__ src, const int32_t* __restrict__ blk_off,
                                                 int E, int block_m, T* __restrict__ rows, int64_t num_rows, int H,
                                                 int64_t g) {
  Vec<T, Granule<T>::kWhole> zero;
  memset(&zero, 0, 16);
  each_padding_row(src, blk_off, E, block_m, num_rows, g, [&](int64_t r, int lane) {
    for (int i = lane; i < Granule<T>::most(H); i += 32) {
      const Granule<T> q(rows + r * H, H, i);
      if (q.n > 0) q.store(rows + r * H, zero);
    }
  });
}

// The pool rows and weights of a CTA's tokens in shared memory.
struct TokenRows {
  int32_t row[kMaxGroups * kMaxK];
  float w[kMaxGroups * kMaxK];
};
__device__ __forceinline__ void load_token_rows(TokenRows& s, const int32_t* __restrict__ slot,
                                                const float* __restrict__ w, int64_t t0, int tokens, int64_t T, int K,
                                                int64_t num_rows) {
  for (int i = threadIdx.x; i < tokens * K; i += blockDim.x) {
    const int64_t p = t0 * K + i;
    int r = -1;
    float wv = 1.f;
    if (p < T * K) {
      r = __ldg(slot + p);
      if (r >= num_rows) r = -1;
      if (w) wv = __ldg(w + p);
    }
    s.row[i] = r;
    s.w[i] = wv;
  }
  __syncthreads();
}

template <int B>
__global__ void __launch_bounds__(kThreads)
    permute_kernel(const char* __restrict__ x, int64_t x_pitch, int64_t T, int64_t pitch, int lanes, unsigned pad_ctas,
                   const int32_t* __restrict__ slot, int K, const int32_t* __restrict__ src,
                   const int32_t* __restrict__ blk_off, int E, int block_m, char* __restrict__ rows,
                   int64_t num_rows) {
  using V = Vec<char, B>;
  if (blockIdx.x < pad_ctas) {
    zero_padding<B>(src, blk_off, E, block_m, rows, num_rows, pitch, blockIdx.x);
    return;
  }
  __shared__ TokenRows s;
  const int tokens = kThreads / lanes;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x - pad_ctas) * tokens;
  load_token_rows(s, slot, nullptr, t0, tokens, T, K, num_rows);
  const int sub = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t t = t0 + sub;
  if (t >= T) return;
  const V* xr = reinterpret_cast<const V*>(x + t * x_pitch);
  const int32_t* my = s.row + sub * K;
  const int n = static_cast<int>(pitch / B);
  for (int i = l; i < n; i += lanes) {
    const V v = load_once(xr + i);
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int64_t r = my[k];
      if (r >= 0) store_once(reinterpret_cast<V*>(rows + r * pitch) + i, v);
    }
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(kThreads)
    unpermute_kernel(const T* __restrict__ rows, int64_t num_rows, int H, int64_t tokens_total, int lanes,
                     const int32_t* __restrict__ slot, const float* __restrict__ w, int K, T* __restrict__ out,
                     int64_t out_stride) {
  using V = Vec<T, N>;
  __shared__ TokenRows s;
  const int tokens = kThreads / lanes;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  load_token_rows(s, slot, w, t0, tokens, tokens_total, K, num_rows);
  const int sub = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t t = t0 + sub;
  if (t >= tokens_total) return;
  const int32_t* my = s.row + sub * K;
  const float* mw = s.w + sub * K;
  const int n = H / N;
  for (int i = l; i < n; i += lanes) {
    float acc[N];
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int64_t r = my[k];
      if (r >= 0) {
        const V v = load_once(reinterpret_cast<const V*>(rows + r * H) + i);
        const float wk = mw[k];
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = fmaf(wk, to_float(v.v[c]), acc[c]);
      }
    }
    V o;
#pragma unroll
    for (int c = 0; c < N; ++c) o.v[c] = from_float<T>(acc[c]);
    store_once(reinterpret_cast<V*>(out + t * out_stride) + i, o);
  }
}

// The dots of a token summed over its threads: lanes of a warp, then (rows wider than a warp) its warps in order.
template <int KT>
__device__ __forceinline__ void sum_dots(float (&dot)[KT], float (&s_dot)[kBackThreads / 32][KT], float* __restrict__ d_w,
                                         int64_t t, int64_t tokens_total, int K, int lanes, int sub, int l) {
  const int width = lanes < 32 ? lanes : 32;
#pragma unroll
  for (int k = 0; k < KT; ++k)
    for (int o = width / 2; o > 0; o >>= 1) dot[k] += __shfl_xor_sync(0xffffffffu, dot[k], o);
  if (lanes <= 32) {
    if (l == 0 && t < tokens_total)
#pragma unroll
      for (int k = 0; k < KT; ++k)
        if (k < K) d_w[t * K + k] = dot[k];
    return;
  }
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < KT; ++k) s_dot[threadIdx.x >> 5][k] = dot[k];
  __syncthreads();
  if (l < K && t < tokens_total) {
    float v = 0.f;
    for (int i = 0; i < lanes / 32; ++i) v += s_dot[sub * (lanes / 32) + i][l];
    d_w[t * K + l] = v;
  }
}

// KT >= K: the dots of a token live in registers.
template <typename T, int N, int KT>
__global__ void __launch_bounds__(kBackThreads)
    unpermute_backward_kernel(const T* __restrict__ d_out, int64_t d_stride, const T* __restrict__ rows, int H,
                              int64_t tokens_total, int lanes, unsigned pad_ctas, const int32_t* __restrict__ slot,
                              const float* __restrict__ w, int K, const int32_t* __restrict__ src,
                              const int32_t* __restrict__ blk_off, int E, int block_m, T* __restrict__ d_rows,
                              int64_t num_rows, float* __restrict__ d_w) {
  using V = Vec<T, N>;
  if (blockIdx.x < pad_ctas) {
    zero_padding<N * sizeof(T)>(src, blk_off, E, block_m, reinterpret_cast<char*>(d_rows), num_rows,
                                static_cast<int64_t>(H) * sizeof(T), blockIdx.x);
    return;
  }
  __shared__ TokenRows s;
  __shared__ float s_dot[kBackThreads / 32][KT];
  const int tokens = kBackThreads / lanes;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x - pad_ctas) * tokens;
  load_token_rows(s, slot, w, t0, tokens, tokens_total, K, num_rows);
  const int sub = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t t = t0 + sub;
  float dot[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) dot[k] = 0.f;
  if (t < tokens_total) {
    const V* dr = reinterpret_cast<const V*>(d_out + t * d_stride);
    const int32_t* my = s.row + sub * K;
    const float* mw = s.w + sub * K;
    const int n = H / N;
    for (int i = l; i < n; i += lanes) {
      const V dv = load_once(dr + i);
      float d[N];
#pragma unroll
      for (int c = 0; c < N; ++c) d[c] = to_float(dv.v[c]);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const int64_t r = k < K ? my[k] : -1;
        if (r >= 0) {
          if (d_w) {
            const V v = load_once(reinterpret_cast<const V*>(rows + r * H) + i);
#pragma unroll
            for (int c = 0; c < N; ++c) dot[k] = fmaf(to_float(v.v[c]), d[c], dot[k]);
          }
          const float wk = mw[k];
          V o;
#pragma unroll
          for (int c = 0; c < N; ++c) o.v[c] = from_float<T>(wk * d[c]);
          store_once(reinterpret_cast<V*>(d_rows + r * H) + i, o);
        }
      }
    }
  }
  if (d_w) sum_dots<KT>(dot, s_dot, d_w, t, tokens_total, K, lanes, sub, l);
}

// ---------------------------------------------------------------- rows on no 16-byte boundary
// The same three by 16-byte granules of the rows they write (Granule): every row has its own offset from a
// boundary, and what is read is shifted to it. (With accesses as narrow as the rows' alignment, 4097x4095 bf16 top-6
// took 76, 116 and 230 us, one column more 41, 40 and 74.)
template <typename T>
__global__ void __launch_bounds__(kThreads)
    permute_any_kernel(const T* __restrict__ x, int64_t x_stride, int64_t tokens_total, int H, int lanes, unsigned pad_ctas,
                       const int32_t* __restrict__ slot, int K, const int32_t* __restrict__ src,
                       const int32_t* __restrict__ blk_off, int E, int block_m, T* __restrict__ rows,
                       int64_t num_rows) {
  if (blockIdx.x < pad_ctas) {
    zero_padding_any<T>(src, blk_off, E, block_m, rows, num_rows, H, blockIdx.x);
    return;
  }
  __shared__ TokenRows s;
  const int tokens = kThreads / lanes;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x - pad_ctas) * tokens;
  load_token_rows(s, slot, nullptr, t0, tokens, tokens_total, K, num_rows);
  const int sub = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t t = t0 + sub;
  if (t >= tokens_total) return;
  const T* xr = x + t * x_stride;
  const int32_t* my = s.row + sub * K;
  const int most = Granule<T>::most(H);
  for (int i = l; i < most; i += lanes)
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int64_t r = my[k];
      if (r < 0) continue;
      T* d = rows + r * H;
      const Granule<T> g(d, H, i);
      if (g.n > 0) g.store(d, g.load(xr));
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    unpermute_any_kernel(const T* __restrict__ rows, int64_t num_rows, int H, int64_t tokens_total, int lanes,
                         const int32_t* __restrict__ slot, const float* __restrict__ w, int K, T* __restrict__ out,
                         int64_t out_stride) {
  constexpr int N = Granule<T>::kWhole;
  __shared__ TokenRows s;
  const int tokens = kThreads / lanes;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens;
  load_token_rows(s, slot, w, t0, tokens, tokens_total, K, num_rows);
  const int sub = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t t = t0 + sub;
  if (t >= tokens_total) return;
  const int32_t* my = s.row + sub * K;
  const float* mw = s.w + sub * K;
  T* o = out + t * out_stride;
  const int most = Granule<T>::most(H);
  for (int i = l; i < most; i += lanes) {
    const Granule<T> g(o, H, i);
    if (g.n <= 0) continue;
    float acc[N];
#pragma unroll
    for (int c = 0; c < N; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int64_t r = my[k];
      if (r >= 0) {
        const Vec<T, N> v = g.load(rows + r * H);
        const float wk = mw[k];
#pragma unroll
        for (int c = 0; c < N; ++c) acc[c] = fmaf(wk, to_float(v.v[c]), acc[c]);
      }
    }
    Vec<T, N> v;
#pragma unroll
    for (int c = 0; c < N; ++c) v.v[c] = from_float<T>(acc[c]);
    g.store(o, v);
  }
}

template <typename T, int KT>
__global__ void __launch_bounds__(kBackThreads)
    unpermute_backward_any_kernel(const T* __restrict__ d_out, int64_t d_stride, const T* __restrict__ rows, int H,
                                  int64_t tokens_total, int lanes, unsigned pad_ctas,
                                  const int32_t* __restrict__ slot, const float* __restrict__ w, int K,
                                  const int32_t* __restrict__ src, const int32_t* __restrict__ blk_off, int E,
                                  int block_m, T* __restrict__ d_rows, int64_t num_rows, float* __restrict__ d_w) {
  constexpr int N = Granule<T>::kWhole;
  if (blockIdx.x < pad_ctas) {
    zero_padding_any<T>(src, blk_off, E, block_m, d_rows, num_rows, H, blockIdx.x);
    return;
  }
  __shared__ TokenRows s;
  __shared__ float s_dot[kBackThreads / 32][KT];
  const int tokens = kBackThreads / lanes;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x - pad_ctas) * tokens;
  load_token_rows(s, slot, w, t0, tokens, tokens_total, K, num_rows);
  const int sub = threadIdx.x / lanes, l = threadIdx.x % lanes;
  const int64_t t = t0 + sub;
  float dot[KT];
#pragma unroll
  for (int k = 0; k < KT; ++k) dot[k] = 0.f;
  if (t < tokens_total) {
    const T* dr = d_out + t * d_stride;
    const int32_t* my = s.row + sub * K;
    const float* mw = s.w + sub * K;
    const int most = Granule<T>::most(H);
    for (int i = l; i < most; i += lanes) {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const int64_t r = k < K ? my[k] : -1;
        if (r < 0) continue;
        T* o = d_rows + r * H;
        const Granule<T> g(o, H, i);
        if (g.n <= 0) continue;
        const Vec<T, N> dv = g.load(dr);
        if (d_w) {
          const Vec<T, N> v = g.load(rows + r * H);
#pragma unroll
          for (int c = 0; c < N; ++c)
            if (c < g.n) dot[k] = fmaf(to_float(v.v[c]), to_float(dv.v[c]), dot[k]);
        }
        const float wk = mw[k];
        Vec<T, N> v;
#pragma unroll
        for (int c = 0; c < N; ++c) v.v[c] = from_float<T>(wk * to_float(dv.v[c]));
        g.store(o, v);
      }
    }
  }
  if (d_w) sum_dots<KT>(dot, s_dot, d_w, t, tokens_total, K, lanes, sub, l);
}

// Threads of a token's group: its accesses rounded up to a power of two, 8 to the CTA's threads.
int group_lanes(int64_t accesses, int threads) {
  int l = 8;
  while (l < threads && l < accesses) l *= 2;
  return l;
}

uint64_t bits_of(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// f with the number of elements a 32- or 16-byte access holds, or with 0 where rows are on no 16-byte boundary
template <typename T, typename F>
cudaError_t with_access(int B, F f) {
  if (B == 32) return f(std::integral_constant<int, 32 / sizeof(T)>{});
  if (B == 16) return f(std::integral_constant<int, 16 / sizeof(T)>{});
  return f(std::integral_constant<int, 0>{});
}

}  // namespace

cudaError_t launch_permute(const RowsArgs& a, const void* x, int64_t x_stride, void* rows, cudaStream_t s) {
  const int es = dtype_size(a.dtype);
  const int64_t pitch = static_cast<int64_t>(a.H) * es;
  const int B = access_bytes(bits_of(x) | bits_of(rows) | pitch | x_stride * es);
  const int64_t pad = (a.num_rows + kPadRows - 1) / kPadRows;
  auto ctas = [&](int lanes) { return (a.T + kThreads / lanes - 1) / (kThreads / lanes); };
  if (B >= 16) {
    const int lanes = group_lanes(pitch / B, kThreads);
    const int64_t grid = pad + ctas(lanes);
    if (grid == 0) return cudaSuccess;
    auto kernel = B == 32 ? permute_kernel<32> : permute_kernel<16>;
    kernel<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
        static_cast<const char*>(x), x_stride * es, a.T, pitch, lanes, static_cast<unsigned>(pad), a.slot, a.K, a.src,
        a.blk_off, a.E, a.block_m, static_cast<char*>(rows), a.num_rows);
    return cudaGetLastError();
  }
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    const int lanes = group_lanes(Granule<T>::most(a.H), kThreads);
    const int64_t grid = pad + ctas(lanes);
    if (grid == 0) return cudaSuccess;
    permute_any_kernel<T><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(
        static_cast<const T*>(x), x_stride, a.T, a.H, lanes, static_cast<unsigned>(pad), a.slot, a.K, a.src, a.blk_off,
        a.E, a.block_m, static_cast<T*>(rows), a.num_rows);
    return cudaGetLastError();
  });
}

cudaError_t launch_unpermute(const RowsArgs& a, const void* rows, const float* w, void* out, int64_t out_stride,
                             cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int es = dtype_size(a.dtype);
  const int B = access_bytes(bits_of(rows) | bits_of(out) | static_cast<uint64_t>(a.H) * es |
                             static_cast<uint64_t>(out_stride) * es);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return with_access<T>(B, [&](auto n) {
      constexpr int N = decltype(n)::value;
      const int lanes = group_lanes(N ? a.H / (N ? N : 1) : Granule<T>::most(a.H), kThreads);
      const unsigned grid = static_cast<unsigned>((a.T + kThreads / lanes - 1) / (kThreads / lanes));
      const T* r = static_cast<const T*>(rows);
      T* o = static_cast<T*>(out);
      if constexpr (N > 0)
        unpermute_kernel<T, N><<<grid, kThreads, 0, s>>>(r, a.num_rows, a.H, a.T, lanes, a.slot, w, a.K, o, out_stride);
      else
        unpermute_any_kernel<T><<<grid, kThreads, 0, s>>>(r, a.num_rows, a.H, a.T, lanes, a.slot, w, a.K, o, out_stride);
      return cudaGetLastError();
    });
  });
}

cudaError_t launch_unpermute_backward(const RowsArgs& a, const void* d_out, int64_t d_stride, const void* rows,
                                      const float* w, void* d_rows, float* d_w, cudaStream_t s) {
  const int es = dtype_size(a.dtype);
  const int B = access_bytes(bits_of(rows) | bits_of(d_out) | bits_of(d_rows) | static_cast<uint64_t>(a.H) * es |
                             static_cast<uint64_t>(d_stride) * es);
  return with_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return with_access<T>(B, [&](auto n) {
      constexpr int N = decltype(n)::value;
      const int lanes = group_lanes(N ? a.H / (N ? N : 1) : Granule<T>::most(a.H), kBackThreads);
      const int64_t ctas = (a.T + kBackThreads / lanes - 1) / (kBackThreads / lanes);
      const int64_t pad = (a.num_rows + kPadRows - 1) / kPadRows, grid = pad + ctas;
      if (grid == 0) return cudaSuccess;
      auto go = [&](auto kt) {
        constexpr int KT = decltype(kt)::value;
        auto launch = [&](auto kernel) {
          kernel<<<static_cast<unsigned>(grid), kBackThreads, 0, s>>>(
              static_cast<const T*>(d_out), d_stride, static_cast<const T*>(rows), a.H, a.T, lanes,
              static_cast<unsigned>(pad), a.slot, w, a.K, a.src, a.blk_off, a.E, a.block_m, static_cast<T*>(d_rows),
              a.num_rows, d_w);
          return cudaGetLastError();
        };
        if constexpr (N > 0) return launch(unpermute_backward_kernel<T, N, KT>);
        else return launch(unpermute_backward_any_kernel<T, KT>);
      };
      if (a.K <= 4) return go(std::integral_constant<int, 4>{});
      if (a.K <= 8) return go(std::integral_constant<int, 8>{});
      return go(std::integral_constant<int, 16>{});
    });
  });
}

}  // namespace mm

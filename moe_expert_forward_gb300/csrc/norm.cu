// Root-mean-square norm of rows with the residual's addition, in rows and in 8 bits,
// and its gradients.
//   h = round(x + residual);  r = 1 / sqrt(mean(h^2) + eps);  y = h r weight
//   g = d_y weight, n = h r:  d_x = d_h + r (g - n mean(g n));  d_weight = sum_t d_y n
// All sums are fp32 in a fixed order.  The norm is taken of the rounded h, because h
// is what the residual stream carries on and what the gradients read again.
//
// Memory bounds both (read x and the residual, write h, y and the codes; back: read
// d_y, h and d_h, write d_x).  A row stays in the registers of its threads, 16
// elements a lane and access, between the sum and its use, up to kHeld elements;
// longer rows are read twice.  For d_weight a thread keeps the same columns of every
// row that its CTA takes, so the sums over tokens stay in registers too; the CTAs'
// parts are added up, in order, by a second kernel.
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kMostThreads = 512;

struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;      // or null
  int64_t r_stride;
  const void* weight;
  bool w_f32;                // else of the rows' type
  int64_t T;
  int H;
  float eps;
  void* h;                   // null without a residual
  void* y;                   // or null
  Out8 out;                  // codes null: none
  float* rstd;
  int row_threads;
};

// The sum of v over the row_threads threads of a row, for each of them. All threads of the CTA take part.
__device__ __forceinline__ float row_sum(float v, int row_threads, float* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (row_threads == 32) return v;
  const int warps = row_threads / 32, first = (threadIdx.x / row_threads) * warps;
  __syncthreads();                               // the parts of the sum before this one have been read
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < warps; ++i) v += s_part[first + i];
  return v;
}

// Weights of columns c .. c+15, zeros past H.
template <typename T, bool kVec>
__device__ __forceinline__ void load_weight(const void* w, bool w_f32, int c, int H, float (&f)[16]) {
  if (w_f32) {
    Group<float> g;
    g.template load<kVec>(static_cast<const float*>(w), c, H);
    g.floats(f);
  } else {
    Group<T> g;
    g.template load<kVec>(static_cast<const T*>(w), c, H);
    g.floats(f);
  }
}

// G > 0: a row's G groups a thread are held in registers. G = 0: any length, read twice.
template <typename T, bool kVec, int G>
__global__ void __launch_bounds__(kMostThreads) rms_norm_kernel(const NormArgs a) {
  __shared__ float s_part[kMostThreads / 32];
  extern __shared__ __align__(16) unsigned char s_dyn[];
  T* run = reinterpret_cast<T*>(s_dyn) + (threadIdx.x >> 5) * 512;
  const int P = a.row_threads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / P) + threadIdx.x / P;
  const int l = threadIdx.x % P;
  const bool live = row < a.T;
  const T* x = static_cast<const T*>(a.x) + (live ? row : 0) * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + (live ? row : 0) * a.r_stride;
  T* h = static_cast<T*>(a.h) + (live ? row : 0) * a.H;
  T* y = static_cast<T*>(a.y) + (live ? row : 0) * a.H;
  // groups of the row, to a whole number of warps; its codes may fill more groups than its elements
  const int groups = ((a.out.codes ? a.out.groups : (a.H + 15) / 16) + 31) / 32 * 32;

  // h of group g; `keep`: also stored
  auto take = [&](int g, bool keep, Group<T>& v) {
    if (!live || g * 16 >= a.H) v.clear();
    else v.template load<kVec>(x, g * 16, a.H);
    if (a.residual) {
      Group<T> w;
      if (!live || g * 16 >= a.H) w.clear();
      else w.template load<kVec>(res, g * 16, a.H);
      float f[16], q[16];
      v.floats(f);
      w.floats(q);
#pragma unroll
      for (int i = 0; i < 16; ++i) f[i] += q[i];
      round16<T>(f, v.w);
      if (keep) store_groups<T, kVec>(h + g * 16, live ? min(16, a.H - g * 16) : 0, v.w, run);
    }
  };
  auto squares = [](const Group<T>& v) {
    float f[16], s = 0.f;
    v.floats(f);
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(f[i], f[i], s);
    return s;
  };
  auto finish = [&](int g, const Group<T>& v, float r) {
    float f[16], w[16];
    v.floats(f);
    load_weight<T, kVec>(a.weight, a.w_f32, g * 16, a.H, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = f[i] * r * w[i];
    if (a.y) {
      uint32_t o[Group<T>::kWords];
      round16<T>(f, o);
      store_groups<T, kVec>(y + g * 16, live ? min(16, a.H - g * 16) : 0, o, run);
    }
    if (a.out.codes) {
      if (g * 16 >= a.H)                         // past the row: zeros, also where r is not finite
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = 0.f;
      else if (g * 16 + 16 > a.H)
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = g * 16 + i < a.H ? f[i] : 0.f;
      store8(a.out, row, g, live && g < a.out.groups, f, amax_bits16(f));
    }
  };

  float s = 0.f;
  Group<T> held[G > 0 ? G : 1];
  if constexpr (G > 0) {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (i * P + (l & ~31) < groups) take(i * P + l, true, held[i]);
      else held[i].clear();
#pragma unroll
    for (int i = 0; i < G; ++i) s += squares(held[i]);
  } else {
    for (int g = l; g - (l & 31) < groups; g += P) {
      Group<T> v;
      take(g, true, v);
      s += squares(v);
    }
  }
  s = row_sum(s, P, s_part);
  const float r = 1.0f / sqrtf(s / static_cast<float>(a.H) + a.eps);
  if (live && l == 0) a.rstd[row] = r;
  if constexpr (G > 0) {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (i * P + (l & ~31) < groups) finish(i * P + l, held[i], r);
  } else {
    for (int g = l; g - (l & 31) < groups; g += P) {
      Group<T> v;
      take(g, false, v);
      finish(g, v, r);
    }
  }
}

struct NormBackArgs {
  const void* d_y;
  int64_t dy_stride;
  const void* h;
  int64_t h_stride;
  const void* weight;
  bool w_f32;
  const float* rstd;
  const void* d_h;           // or null
  int64_t dh_stride;
  int64_t T;
  int H;
  void* d_x;
  float* parts;              // [CTAs x rows of a CTA][pitch]
  int pitch;
  int row_threads;
};

// One CTA takes rows in a fixed stride; each group of row_threads threads sums d_weight's part of its own rows.
template <typename T, bool kVec, int G>
__global__ void __launch_bounds__(kMostThreads) rms_norm_backward_kernel(const NormBackArgs a) {
  __shared__ float s_part[kMostThreads / 32];
  extern __shared__ __align__(16) unsigned char s_dyn[];
  T* run = reinterpret_cast<T*>(s_dyn) + (threadIdx.x >> 5) * 512;
  const int P = a.row_threads, rows = blockDim.x / P;
  const int l = threadIdx.x % P;
  const int groups = ((a.H + 15) / 16 + 31) / 32 * 32;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / P;
  float* part = a.parts + mine * a.pitch;
  float acc[G > 0 ? G : 1][16];
  if constexpr (G > 0) {
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int c = 0; c < 16; ++c) acc[i][c] = 0.f;
  } else {
    for (int g = l; g * 16 < a.H; g += P)
#pragma unroll
      for (int c = 0; c < 16; ++c) part[g * 16 + c] = 0.f;
  }
  // every thread of the CTA runs as long as one has a row: the sums are the CTA's
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows; row0 < a.T; row0 += static_cast<int64_t>(gridDim.x) * rows) {
    const int64_t row = row0 + threadIdx.x / P;
    const bool live = row < a.T;
    const T* dy = static_cast<const T*>(a.d_y) + (live ? row : 0) * a.dy_stride;
    const T* h = static_cast<const T*>(a.h) + (live ? row : 0) * a.h_stride;
    const T* dh = static_cast<const T*>(a.d_h) + (live ? row : 0) * a.dh_stride;
    T* dx = static_cast<T*>(a.d_x) + (live ? row : 0) * a.H;
    const float r = live ? __ldg(a.rstd + row) : 0.f;
    auto load = [&](const T* p, int g, Group<T>& v) {
      if (live && g * 16 < a.H) v.template load<kVec>(p, g * 16, a.H);
      else v.clear();
    };
    // sum over a group of g n
    auto dot = [&](int g, const Group<T>& vy, const Group<T>& vh) {
      float y[16], n[16], w[16], s = 0.f;
      vy.floats(y);
      vh.floats(n);
      load_weight<T, kVec>(a.weight, a.w_f32, g * 16, a.H, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) s = fmaf(y[i] * w[i], n[i] * r, s);
      return s;
    };
    auto finish = [&](int g, const Group<T>& vy, const Group<T>& vh, const Group<T>& vd, float mean, float (&sum)[16]) {
      float y[16], n[16], w[16], d[16];
      vy.floats(y);
      vh.floats(n);
      vd.floats(d);
      load_weight<T, kVec>(a.weight, a.w_f32, g * 16, a.H, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float ni = n[i] * r;
        sum[i] = fmaf(y[i], ni, sum[i]);
        d[i] += r * (y[i] * w[i] - ni * mean);
      }
      uint32_t o[Group<T>::kWords];
      round16<T>(d, o);
      store_groups<T, kVec>(dx + g * 16, live ? min(16, a.H - g * 16) : 0, o, run);
    };
    if constexpr (G > 0) {
      Group<T> vy[G], vh[G], vd[G];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        load(dy, i * P + l, vy[i]);
        load(h, i * P + l, vh[i]);
        if (a.d_h) load(dh, i * P + l, vd[i]);
        else vd[i].clear();
      }
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) s += dot(i * P + l, vy[i], vh[i]);
      const float mean = row_sum(s, P, s_part) / static_cast<float>(a.H);
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (i * P + (l & ~31) < groups) finish(i * P + l, vy[i], vh[i], vd[i], mean, acc[i]);
    } else {
      float s = 0.f;
      for (int g = l; g - (l & 31) < groups; g += P) {
        Group<T> vy, vh;
        load(dy, g, vy);
        load(h, g, vh);
        s += dot(g, vy, vh);
      }
      const float mean = row_sum(s, P, s_part) / static_cast<float>(a.H);
      for (int g = l; g - (l & 31) < groups; g += P) {
        Group<T> vy, vh, vd;
        load(dy, g, vy);
        load(h, g, vh);
        if (a.d_h) load(dh, g, vd);
        else vd.clear();
        float sum[16];
        const bool in = g * 16 < a.H;
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[c] = in ? part[g * 16 + c] : 0.f;
        finish(g, vy, vh, vd, mean, sum);
        if (in)
#pragma unroll
          for (int c = 0; c < 16; ++c) part[g * 16 + c] = sum[c];
      }
    }
  }
  if constexpr (G > 0) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int c = (i * P + l) * 16;
      if (c < a.H)
#pragma unroll
        for (int q = 0; q < 16; q += 4)
          *reinterpret_cast<float4*>(part + c + q) = make_float4(acc[i][q], acc[i][q + 1], acc[i][q + 2], acc[i][q + 3]);
    }
  }
}

// d_weight: the parts of each column in order. A CTA takes 32 columns, its warps every eighth part.
__global__ void __launch_bounds__(kThreads)
    norm_weight_kernel(const float* __restrict__ parts, int pitch, int count, int H, float* __restrict__ d_weight) {
  __shared__ float s[kThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int p = warp; p < count; p += kThreads / 32) v += parts[static_cast<int64_t>(p) * pitch + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < H) {
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v += s[i][lane];
    d_weight[c] = v;
  }
}

// Threads of a row, its groups a thread (0: more than are held) and rows of a CTA.
struct Shape {
  int P, G, rows;
};
Shape shape_for(int groups, int held) {
  Shape s;
  s.P = row_threads(groups, held > 1 ? 2 : 1, kThreads);
  if (s.P * held < groups) s.P = row_threads(groups, held, kMostThreads);
  s.G = 0;
  for (int g = 1; g <= held && !s.G; g *= 2)
    if (s.P * g >= groups) s.G = g;
  s.rows = s.P < kThreads ? kThreads / s.P : 1;
  return s;
}

constexpr int kHeldForward = 4, kHeldBack = 2;   // groups a thread

Shape back_shape(int H) { return shape_for((H + 15) / 16, kHeldBack); }
int64_t back_ctas(int64_t T, const Shape& s) {
  const int64_t all = (T + s.rows - 1) / s.rows, most = 2 * int64_t(kNormBackSms);
  return all < most ? all : most;
}
int back_pitch(int H) { return (H + 15) / 16 * 16; }

}  // namespace

size_t norm_scratch_bytes(int64_t T, int H) {
  const Shape s = back_shape(H);
  return static_cast<size_t>(back_ctas(T, s)) * s.rows * back_pitch(H) * sizeof(float);
}

cudaError_t launch_rms_norm(const NormLaunch& n, cudaStream_t s) {
  const int elem = dtype_size(n.dtype);
  NormArgs a{n.x, n.x_stride, n.residual, n.residual_stride, n.weight, n.weight_dtype == MM_MOE_DTYPE_F32, n.T, n.H,
             n.eps, n.h, n.y, {}, n.rstd, 0};
  if (n.codes)
    a.out = Out8{n.variant, static_cast<uint8_t*>(n.codes), n.sf, groups8(n.H, n.variant), blocks8(n.H, n.variant)};
  const Shape sh = shape_for(n.codes ? a.out.groups : (n.H + 15) / 16, kHeldForward);
  a.row_threads = sh.P;
  const int64_t pitch = static_cast<int64_t>(n.H) * elem;
  const bool vec = whole_groups(n.x, n.x_stride * elem, n.H) && whole_groups(n.residual, n.residual_stride * elem, n.H) &&
                   whole_groups(n.h, pitch, n.H) && whole_groups(n.y, pitch, n.H) && whole_groups(n.weight, 0, n.H);
  const unsigned grid = static_cast<unsigned>((n.T + sh.rows - 1) / sh.rows);
  const int threads = sh.P * sh.rows;
  return with_dtype(n.dtype, [&](auto tag) {
    using T = decltype(tag);
    const size_t smem = vec ? 0 : threads / 32 * 512 * sizeof(T);
    auto go = [&](auto v) {
      constexpr bool V = decltype(v)::value;
      if (sh.G == 1) rms_norm_kernel<T, V, 1><<<grid, threads, smem, s>>>(a);
      else if (sh.G == 2) rms_norm_kernel<T, V, 2><<<grid, threads, smem, s>>>(a);
      else if (sh.G == 4) rms_norm_kernel<T, V, 4><<<grid, threads, smem, s>>>(a);
      else rms_norm_kernel<T, V, 0><<<grid, threads, smem, s>>>(a);
      return cudaGetLastError();
    };
    return vec ? go(std::true_type{}) : go(std::false_type{});
  });
}

cudaError_t launch_rms_norm_backward(const NormBackLaunch& n, cudaStream_t s) {
  if (n.T == 0) return cudaMemsetAsync(n.d_weight, 0, sizeof(float) * static_cast<size_t>(n.H), s);
  const int elem = dtype_size(n.dtype);
  const Shape sh = back_shape(n.H);
  const int64_t pitch = static_cast<int64_t>(n.H) * elem;
  const NormBackArgs a{n.d_y, n.d_y_stride, n.h, n.h_stride, n.weight, n.weight_dtype == MM_MOE_DTYPE_F32, n.rstd, n.d_h,
                       n.d_h_stride, n.T, n.H, n.d_x, static_cast<float*>(n.scratch), back_pitch(n.H), sh.P};
  const bool vec = whole_groups(n.d_y, n.d_y_stride * elem, n.H) && whole_groups(n.h, n.h_stride * elem, n.H) &&
                   whole_groups(n.d_h, n.d_h_stride * elem, n.H) && whole_groups(n.d_x, pitch, n.H) &&
                   whole_groups(n.weight, 0, n.H);
  const unsigned grid = static_cast<unsigned>(back_ctas(n.T, sh));
  const int threads = sh.P * sh.rows;
  const cudaError_t e = with_dtype(n.dtype, [&](auto tag) {
    using T = decltype(tag);
    const size_t smem = vec ? 0 : threads / 32 * 512 * sizeof(T);
    auto go = [&](auto v) {
      constexpr bool V = decltype(v)::value;
      if (sh.G == 1) rms_norm_backward_kernel<T, V, 1><<<grid, threads, smem, s>>>(a);
      else if (sh.G == 2) rms_norm_backward_kernel<T, V, 2><<<grid, threads, smem, s>>>(a);
      else rms_norm_backward_kernel<T, V, 0><<<grid, threads, smem, s>>>(a);
      return cudaGetLastError();
    };
    return vec ? go(std::true_type{}) : go(std::false_type{});
  });
  if (e != cudaSuccess) return e;
  norm_weight_kernel<<<static_cast<unsigned>((n.H + 31) / 32), kThreads, 0, s>>>(
      a.parts, a.pitch, static_cast<int>(grid) * sh.rows, n.H, n.d_weight);
  return cudaGetLastError();
}

}  // namespace mm

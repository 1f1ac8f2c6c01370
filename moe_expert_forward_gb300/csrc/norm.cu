// Root-mean-square norm of rows with the residual's addition, in rows and in 8 bits,
// and its gradients.
//   h = round(x + residual);  r = 1 / sqrt(mean(h^2) + eps);  y = h r weight
//   g = d_y weight, n = h r:  d_x = d_h + r (g - n mean(g n));  d_weight = sum_t d_y n
// All sums are fp32 in a fixed order.  The norm is taken of the rounded h, because h
// is what the residual stream carries on and what the gradients read again.
//
// Memory bounds both (read x and the residual, write h, y and the codes; back: read
// d_y, h and d_h, write d_x).  A row stays in the registers of its threads, 16
// elements a lane and access, between the sum and its use.
//   ring   many long rows: persistent CTAs take rows in a fixed stride, and bulk copies
//          bring the next ones into a ring in shared memory meanwhile, so that loads are in
//          flight through the sum and the stores. Weights stay in registers.
//   rows   few rows, short ones, or rows on no 32-byte boundary: loaded by their threads.
//          Rows longer than the threads hold are read twice.
// Measured (with a residual or d_h, one of the calls of a graph over 400 MB of inputs, of the copy rate): forward 8192x4096
// bf16 47 us (83 %), fp32 95 (83 %), 8192x7168 bf16 with f8 codes 88 (89 %); gradients 8192x4096 bf16 51 us with the sum of
// d_weight's parts (77 %), fp32 100 (79 %).  By their threads, bf16 forward / back: 8192x1024 16 / 19 (61 and 51 %), 8192x2049
// 44 / 73 (45 and 27 %).  One row of 4096 takes 3 us, latency.
// For d_weight a thread keeps the same columns of every row that its CTA takes, so the
// sums over tokens stay in registers too; the CTAs' parts are added up, in order, by a
// second kernel.
#include "mx_linear.cuh"
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kMostThreads = 512;
constexpr int kRingBytes = 160 * 1024, kBackRingBytes = 200 * 1024;       // of the rings of an SM's CTAs
constexpr int kMostStages = 6;
constexpr uint64_t kTimeoutNs = 2000000000ull;
enum : int { kSiteForward = 201, kSiteBackward = 202 };

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

// The sum of a row's groups of 16 columns, in every thread of the row: v[i] that of the thread's i-th group. Groups are
// added up by 32 that follow each other, and those sums in order, so that a row's sum depends on its length alone, not on
// the kernel and the threads that take it, nor on how many rows there are.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], float* s_part, int warps, int warp) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if ((threadIdx.x & 31) == 0) s_part[i * warps + warp] = v[i];
  }
}
__device__ __forceinline__ float sum_in_order(const float* s_part, int n) {
  float v = s_part[0];
  for (int i = 1; i < n; ++i) v += s_part[i];
  return v;
}
// All threads of the CTA take part; its rows have row_threads threads each.
template <int N>
__device__ __forceinline__ float row_sum(float (&v)[N], int row_threads, float* s_part) {
  const int warps = row_threads / 32, row = threadIdx.x / row_threads;
  __syncthreads();                               // the parts of the sum before this one have been read
  warp_sums(v, s_part + row * warps * N, warps, (threadIdx.x >> 5) - row * warps);
  if (row_threads == 32 && N == 1) return v[0];
  __syncthreads();
  return sum_in_order(s_part + row * warps * N, warps * N);
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
  __shared__ float s_part[2 * kMostThreads / 32];
  extern __shared__ __align__(128) unsigned char s_dyn[];
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

  float s[G > 0 ? G : 1] = {};
  Group<T> held[G > 0 ? G : 1];
  if constexpr (G > 0) {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (i * P + (l & ~31) < groups) take(i * P + l, true, held[i]);
      else held[i].clear();
#pragma unroll
    for (int i = 0; i < G; ++i) s[i] = squares(held[i]);
  } else {
    for (int g = l; g - (l & 31) < groups; g += P) {
      Group<T> v;
      take(g, true, v);
      s[0] += squares(v);
    }
  }
  const float r = 1.0f / sqrtf(row_sum(s, P, s_part) / static_cast<float>(a.H) + a.eps);
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
  float* parts;              // [CTAs][pitch]
  int pitch;
  int row_threads;
};

// d: d_h on entry, d_x on return; sum: d_weight's part of these columns.
__device__ __forceinline__ void back16(const float (&y)[16], const float (&h)[16], const float (&w)[16], float r, float mean,
                                       float (&d)[16], float (&sum)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float n = h[i] * r;
    sum[i] = fmaf(y[i], n, sum[i]);
    d[i] = fmaf(r, fmaf(y[i], w[i], -n * mean), d[i]);
  }
}

// Brings up to 16 of the n elements from p on into L2, by addresses of theirs 32 bytes apart.
template <typename T>
__device__ __forceinline__ void prefetch_group(const T* p, int n) {
  constexpr int kStep = 32 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16; i += kStep)
    if (i < n) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i));
}

// One CTA takes rows in a fixed stride; each group of row_threads threads sums d_weight's part of its own rows. The next
// row is on its way into L2 meanwhile, and the weights stay in registers where a thread has one group of columns (cold
// caches, without the two / with them, us: 8192 rows of 512 in fp32 50 / 27, 1024 in bf16 31 / 25, 1025 in fp16 61 / 48, 2049
// in bf16 106 / 78; 4096 of 4097 112 / 85; 2954 of 6047 in fp32 138 / 120).
template <typename T, bool kVec, int G>
__global__ void __launch_bounds__(kMostThreads) rms_norm_backward_kernel(const NormBackArgs a) {
  __shared__ float s_part[2 * kMostThreads / 32];
  extern __shared__ __align__(128) unsigned char s_dyn[];
  T* run = reinterpret_cast<T*>(s_dyn) + (threadIdx.x >> 5) * 512;
  const int P = a.row_threads, rows = blockDim.x / P;
  const int l = threadIdx.x % P;
  const int groups = ((a.H + 15) / 16 + 31) / 32 * 32;
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * a.pitch;
  float acc[G > 0 ? G : 1][16], w[16];           // G = 1: the weights of the thread's columns
  if constexpr (G == 1) load_weight<T, kVec>(a.weight, a.w_f32, l * 16, a.H, w);
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
      float y[16], n[16], s = 0.f;
      vy.floats(y);
      vh.floats(n);
      if (G != 1) load_weight<T, kVec>(a.weight, a.w_f32, g * 16, a.H, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) s = fmaf(y[i] * w[i], n[i] * r, s);
      return s;
    };
    auto finish = [&](int g, const Group<T>& vy, const Group<T>& vh, const Group<T>& vd, float mean, float (&sum)[16]) {
      float y[16], n[16], d[16];
      vy.floats(y);
      vh.floats(n);
      vd.floats(d);
      if (G != 1) load_weight<T, kVec>(a.weight, a.w_f32, g * 16, a.H, w);
      back16(y, n, w, r, mean, d, sum);
      uint32_t o[Group<T>::kWords];
      round16<T>(d, o);
      store_groups<T, kVec>(dx + g * 16, live ? min(16, a.H - g * 16) : 0, o, run);
    };
    if constexpr (G > 0) {
      Group<T> vy[G], vh[G], vd[G];
      const int64_t after = row + static_cast<int64_t>(gridDim.x) * rows;      // the row after this one
      if (after < a.T)
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int c = (i * P + l) * 16;
          prefetch_group(static_cast<const T*>(a.d_y) + after * a.dy_stride + c, a.H - c);
          prefetch_group(static_cast<const T*>(a.h) + after * a.h_stride + c, a.H - c);
          if (a.d_h) prefetch_group(static_cast<const T*>(a.d_h) + after * a.dh_stride + c, a.H - c);
        }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        load(dy, i * P + l, vy[i]);
        load(h, i * P + l, vh[i]);
        if (a.d_h) load(dh, i * P + l, vd[i]);
        else vd[i].clear();
      }
      float s[G];
#pragma unroll
      for (int i = 0; i < G; ++i) s[i] = dot(i * P + l, vy[i], vh[i]);
      const float mean = row_sum(s, P, s_part) / static_cast<float>(a.H);
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (i * P + (l & ~31) < groups) finish(i * P + l, vy[i], vh[i], vd[i], mean, acc[i]);
    } else {
      float s[1] = {};
      for (int g = l; g - (l & 31) < groups; g += P) {
        Group<T> vy, vh;
        load(dy, g, vy);
        load(h, g, vh);
        s[0] += dot(g, vy, vh);
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
    if (rows > 1) {                              // G is 1: the CTA's groups of threads in order
      float* all = reinterpret_cast<float*>(s_dyn);
      __syncthreads();                           // the rows on their way out have left shared memory
#pragma unroll
      for (int c = 0; c < 16; ++c) all[c * blockDim.x + threadIdx.x] = acc[0][c];
      __syncthreads();
      if (threadIdx.x >= P) return;
      for (int k = 1; k < rows; ++k)
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[0][c] += all[c * blockDim.x + k * P + threadIdx.x];
    }
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

// Rows of whole 32-byte pieces that bulk copies bring into a ring in shared memory: `arrays` of them a stage.
struct RowRing {
  uint8_t* base;
  uint64_t* full;
  int* abort;
  int stages, arrays;
  uint32_t row_bytes;
  int s;                     // of the row at hand
  uint32_t phase;
  int loads;                 // by the loading thread

  __device__ __forceinline__ RowRing(uint8_t* smem, int stages, int arrays, uint32_t row_bytes)
      : base(smem), stages(stages), arrays(arrays), row_bytes(row_bytes), s(0), phase(0), loads(0) {
    full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(stages) * arrays * row_bytes);
    abort = reinterpret_cast<int*>(full + stages);
    if (threadIdx.x == 0) {
      for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
      *abort = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  static int bytes(int stages, int arrays, uint32_t row_bytes) { return stages * (arrays * static_cast<int>(row_bytes) + 8) + 16; }
  __device__ __forceinline__ const uint8_t* row(int stage, int array) const {
    return base + (static_cast<size_t>(stage) * arrays + array) * row_bytes;
  }
  // One thread: the arrays' rows at p[] into the stage after the last one's, which nobody reads any more.
  template <int N>
  __device__ __forceinline__ void load(const void* const (&p)[N]) {
    const int stage = loads++ % stages;
    mbar_arrive_expect_tx(&full[stage], arrays * row_bytes);
    int k = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (p[i]) bulk_load(const_cast<uint8_t*>(row(stage, k++)), p[i], row_bytes, &full[stage]);
  }
  // Every thread: the rows of stage s are there. `abort` gives the CTA one answer behind its next barrier.
  __device__ __forceinline__ bool wait(const Status& st, int where) {
    return mbar_wait(&full[s], phase, st, abort, where);
  }
  __device__ __forceinline__ void step() {
    if (++s == stages) {
      s = 0;
      phase ^= 1;
    }
  }
  // The loading thread, after a wait that ran out: what it has in flight.
  __device__ __forceinline__ void drain(const Status& st, int where) const {
    for (int i = 0; i < stages && i < loads; ++i) mbar_wait_drain(&full[i], ((loads - 1 - i) / stages) & 1, st, where);
  }
};
// 16 elements of a row in shared memory, zeros past H.
template <typename T>
__device__ __forceinline__ void take16(Group<T>& v, const uint8_t* row, int g, int H) {
  if (g * 16 >= H) {
    v.clear();
    return;
  }
  const uint4* p = reinterpret_cast<const uint4*>(row) + g * (Group<T>::kWords / 4);
#pragma unroll
  for (int q = 0; q < Group<T>::kWords / 4; ++q) {
    const uint4 w = p[q];
    v.w[4 * q] = w.x; v.w[4 * q + 1] = w.y; v.w[4 * q + 2] = w.z; v.w[4 * q + 3] = w.w;
  }
}
// The row_sum of a CTA's one row; s_part alternates between two arrays, so that one barrier does.
template <int N>
__device__ __forceinline__ float cta_sum(float (&v)[N], float* s_part) {
  const int warps = static_cast<int>(blockDim.x) / 32;
  warp_sums(v, s_part, warps, threadIdx.x >> 5);
  __syncthreads();
  return sum_in_order(s_part, warps * N);
}

template <typename T, typename W, int G>
__global__ void __launch_bounds__(kMostThreads)
    rms_norm_ring_kernel(const NormArgs a, int stages, int* report) {
  extern __shared__ __align__(128) unsigned char s_dyn[];
  __shared__ float s_part[2][G * kMostThreads / 32];
  const uint32_t row_bytes = a.H * static_cast<uint32_t>(sizeof(T));
  RowRing ring(s_dyn, stages, a.residual ? 2 : 1, row_bytes);
  const Status st{report, kTimeoutNs};
  const int l = threadIdx.x;
  auto load = [&](int64_t row) {
    const void* const p[2] = {static_cast<const T*>(a.x) + row * a.x_stride,
                              a.residual ? static_cast<const T*>(a.residual) + row * a.r_stride : nullptr};
    ring.load(p);
  };
  int64_t next = blockIdx.x;                     // the row to load
  if (l == 0)
    for (int i = 0; i < stages && next < a.T; ++i, next += gridDim.x) load(next);
  Group<W> w[G];
#pragma unroll
  for (int i = 0; i < G; ++i) w[i].template load<true>(static_cast<const W*>(a.weight), (i * static_cast<int>(blockDim.x) + l) * 16, a.H);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, ring.step(), turn ^= 1) {
    const bool ok = ring.wait(st, kSiteForward);
    Group<T> h[G];
    float s[G] = {};
    if (ok) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int g = i * static_cast<int>(blockDim.x) + l;
        take16(h[i], ring.row(ring.s, 0), g, a.H);
        float f[16];
        h[i].floats(f);
        if (a.residual) {
          Group<T> r;
          take16(r, ring.row(ring.s, 1), g, a.H);
          float q[16];
          r.floats(q);
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] += q[c];
          round16<T>(f, h[i].w);
          store_groups<T, true>(static_cast<T*>(a.h) + row * a.H + g * 16, g * 16 < a.H ? 16 : 0, h[i].w, nullptr);
          h[i].floats(f);
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) s[i] = fmaf(f[c], f[c], s[i]);
      }
    }
    const float sum = cta_sum(s, s_part[turn]);  // and everyone has read the stage
    if (*reinterpret_cast<volatile int*>(ring.abort)) break;
    if (l == 0 && next < a.T) {
      load(next);
      next += gridDim.x;
    }
    const float r = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
    if (l == 0) a.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int g = i * static_cast<int>(blockDim.x) + l;
      float f[16], q[16];
      h[i].floats(f);
      w[i].floats(q);
#pragma unroll
      for (int c = 0; c < 16; ++c) f[c] = f[c] * r * q[c];
      if (a.y) {
        uint32_t o[Group<T>::kWords];
        round16<T>(f, o);
        store_groups<T, true>(static_cast<T*>(a.y) + row * a.H + g * 16, g * 16 < a.H ? 16 : 0, o, nullptr);
      }
      if (a.out.codes && i * static_cast<int>(blockDim.x) + (l & ~31) < a.out.groups) {
        if (g * 16 >= a.H)                       // past the row: zeros, also where r is not finite
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] = 0.f;
        store8(a.out, row, g, g < a.out.groups, f, amax_bits16(f));
      }
    }
  }
  if (*reinterpret_cast<volatile int*>(ring.abort) && l == 0) ring.drain(st, kSiteForward);
}

template <typename T, typename W, int G>
__global__ void __launch_bounds__(kMostThreads)
    rms_norm_backward_ring_kernel(const NormBackArgs a, int stages, int* report) {
  extern __shared__ __align__(128) unsigned char s_dyn[];
  __shared__ float s_part[2][G * kMostThreads / 32];
  const uint32_t row_bytes = a.H * static_cast<uint32_t>(sizeof(T));
  RowRing ring(s_dyn, stages, a.d_h ? 3 : 2, row_bytes);
  const Status st{report, kTimeoutNs};
  const int l = threadIdx.x;
  auto load = [&](int64_t row) {
    const void* const p[3] = {static_cast<const T*>(a.d_y) + row * a.dy_stride, static_cast<const T*>(a.h) + row * a.h_stride,
                              a.d_h ? static_cast<const T*>(a.d_h) + row * a.dh_stride : nullptr};
    ring.load(p);
  };
  int64_t next = blockIdx.x;
  if (l == 0)
    for (int i = 0; i < stages && next < a.T; ++i, next += gridDim.x) load(next);
  Group<W> w[G];
  float acc[G][16];
#pragma unroll
  for (int i = 0; i < G; ++i) {
    w[i].template load<true>(static_cast<const W*>(a.weight), (i * static_cast<int>(blockDim.x) + l) * 16, a.H);
#pragma unroll
    for (int c = 0; c < 16; ++c) acc[i][c] = 0.f;
  }
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, ring.step(), turn ^= 1) {
    const bool ok = ring.wait(st, kSiteBackward);
    const float r = __ldg(a.rstd + row);
    float s[G] = {};
    if (ok)
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int g = i * static_cast<int>(blockDim.x) + l;
        Group<T> v;
        float y[16], n[16], q[16];
        take16(v, ring.row(ring.s, 0), g, a.H);
        v.floats(y);
        take16(v, ring.row(ring.s, 1), g, a.H);
        v.floats(n);
        w[i].floats(q);
#pragma unroll
        for (int c = 0; c < 16; ++c) s[i] = fmaf(y[c] * q[c], n[c] * r, s[i]);
      }
    const float sum = cta_sum(s, s_part[turn]);  // and everyone is done with the row before
    if (*reinterpret_cast<volatile int*>(ring.abort)) break;
    if (l == 0 && row != blockIdx.x && next < a.T) {
      load(next);
      next += gridDim.x;
    }
    const float mean = sum / static_cast<float>(a.H);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int g = i * static_cast<int>(blockDim.x) + l;
      Group<T> v;
      float y[16], n[16], d[16], q[16];
      take16(v, ring.row(ring.s, 0), g, a.H);
      v.floats(y);
      take16(v, ring.row(ring.s, 1), g, a.H);
      v.floats(n);
      if (a.d_h) take16(v, ring.row(ring.s, 2), g, a.H);
      else v.clear();
      v.floats(d);
      w[i].floats(q);
      back16(y, n, q, r, mean, d, acc[i]);
      round16<T>(d, v.w);
      store_groups<T, true>(static_cast<T*>(a.d_x) + row * a.H + g * 16, g * 16 < a.H ? 16 : 0, v.w, nullptr);
    }
  }
  float* part = a.parts + static_cast<int64_t>(blockIdx.x) * a.pitch;
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const int c = (i * static_cast<int>(blockDim.x) + l) * 16;
    if (c < a.H)
#pragma unroll
      for (int q = 0; q < 16; q += 4)
        *reinterpret_cast<float4*>(part + c + q) = make_float4(acc[i][q], acc[i][q + 1], acc[i][q + 2], acc[i][q + 3]);
  }
  if (*reinterpret_cast<volatile int*>(ring.abort) && l == 0) ring.drain(st, kSiteBackward);
}

// d_weight: the parts of each column in order. A CTA takes 32 columns, each of its 32 warps every 32nd part.
__global__ void __launch_bounds__(1024)
    norm_weight_kernel(const float* __restrict__ parts, int pitch, int count, int H, float* __restrict__ d_weight) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.f;
  pdl_wait();
  if (c < H) {
#pragma unroll 8
    for (int p = warp; p < count; p += 32) v += parts[static_cast<int64_t>(p) * pitch + c];
  }
  s[warp][lane] = v;
  __syncthreads();
  v = s[lane][warp];                             // column `warp` of the CTA's
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && blockIdx.x * 32 + warp < H) d_weight[blockIdx.x * 32 + warp] = v;
}

// Threads of a row, its groups a thread (0: more than are held) and rows of a CTA.
struct Shape {
  int P, G, rows;
};
Shape shape_for(int groups) {
  Shape s;
  const int warps = (groups + 31) / 32;
  s.G = warps <= 16 ? 1 : warps <= 32 ? 2 : 0;
  s.P = s.G == 0 ? kMostThreads : (warps + s.G - 1) / s.G * 32;
  s.rows = s.P < kThreads ? kThreads / s.P : 1;
  return s;
}

// A ring's CTAs: threads, groups of each, stages, CTAs.
struct RingShape {
  int threads, G, stages, ctas;
};
// stages 0: not by a ring. 512 threads an SM in CTAs as small as hold a row (16384 elements at most) and two stages; a row
// is then a CTA's for less time, and more of them are under way. From 2048 columns on (the gradients: 3584), and more rows
// than two CTAs an SM take at once. bf16 with a residual, cold caches, us, by a ring / by their threads (f8: with those
// codes):
//   8192 rows of   1536       2048       2560       3584       4096       7168       8192     16384 (4096 rows)
//   forward      27 / 27    28 / 34    36 / 38    46 / 50    51 / 56   83 / 107   93 / 110   91 / 105
//   f8           36 / 32    38 / 40    46 / 44    53 / 59    61 / 68   92 / 133  112 / 137  106 / 126
//   back         43 / 33    48 / 36    50 / 47    54 / 55    57 / 57   93 / 109   99 / 115  111 / 145
//   320 rows of 4096 11.4 / 10.3, 1024 rows 14.2 / 14.6
// CTAs of 256 threads for 2560 columns: 42, f8 61; the gradients with 160 KB of ring: 5120 columns 81 us, with 200 KB 71.
RingShape ring_for(int64_t T, int H, int elem, int arrays, bool vec, int least_groups, int least_threads, int bytes) {
  const int64_t stage = static_cast<int64_t>(arrays) * H * elem;
  const int groups = (H + 15) / 16;
  if (vec && groups >= least_groups && T > 2 * kNormSms)
    for (int threads = least_threads; threads <= kMostThreads; threads *= 2) {
      const int per_sm = kMostThreads / threads, n = static_cast<int>(bytes / per_sm / stage);
      if (groups <= 2 * threads && n >= 2)
        return {threads, groups <= threads ? 1 : 2, n < kMostStages ? n : kMostStages, per_sm * kNormSms};
    }
  return {0, 0, 0, 0};
}

// Most CTAs, and parts of d_weight, of the gradients.
int64_t back_ctas(int64_t T) { return T < 2 * int64_t(kNormSms) ? T : 2 * int64_t(kNormSms); }
int back_pitch(int H) { return (H + 15) / 16 * 16; }

// f(W{}, G) of a ring's kernel: weights' type, and groups a thread
template <typename T, typename F>
cudaError_t with_ring(bool w_f32, int G, F f) {
  auto go = [&](auto w) {
    return G == 1 ? f(w, std::integral_constant<int, 1>{}) : f(w, std::integral_constant<int, 2>{});
  };
  return w_f32 ? go(float{}) : go(T{});
}

}  // namespace

size_t norm_scratch_bytes(int64_t T, int H) {
  return static_cast<size_t>(back_ctas(T)) * back_pitch(H) * sizeof(float);
}

cudaError_t launch_rms_norm(const NormLaunch& n, cudaStream_t s) {
  const int elem = dtype_size(n.dtype);
  NormArgs a{n.x, n.x_stride, n.residual, n.residual_stride, n.weight, n.weight_dtype == MM_MOE_DTYPE_F32, n.T, n.H,
             n.eps, n.h, n.y, {}, n.rstd, 0};
  if (n.codes)
    a.out = Out8{n.variant, static_cast<uint8_t*>(n.codes), n.sf, groups8(n.H, n.variant), blocks8(n.H, n.variant)};
  const int64_t pitch = static_cast<int64_t>(n.H) * elem;
  const bool vec = whole_groups(n.x, n.x_stride * elem, n.H) && whole_groups(n.residual, n.residual_stride * elem, n.H) &&
                   whole_groups(n.h, pitch, n.H) && whole_groups(n.y, pitch, n.H) && whole_groups(n.weight, 0, n.H);
  const int arrays = n.residual ? 2 : 1;
  const RingShape ring = ring_for(n.T, n.H, elem, arrays, vec, 128, 128, kRingBytes);
  if (ring.stages) {
    int* report = nullptr;
    if (cudaError_t e = mx_report(&report)) return e;
    const int smem = RowRing::bytes(ring.stages, arrays, static_cast<uint32_t>(pitch));
    return with_dtype(n.dtype, [&](auto tag) {
      using T = decltype(tag);
      return with_ring<T>(a.w_f32, ring.G, [&](auto w, auto g) {
        auto kernel = rms_norm_ring_kernel<T, decltype(w), decltype(g)::value>;
        if (cudaError_t e = configure_kernel(reinterpret_cast<const void*>(kernel), 0, kBackRingBytes + 1024)) return e;
        kernel<<<ring.ctas, ring.threads, smem, s>>>(a, ring.stages, report);
        return cudaGetLastError();
      });
    });
  }
  const Shape sh = shape_for(n.codes ? a.out.groups : (n.H + 15) / 16);
  a.row_threads = sh.P;
  const unsigned grid = static_cast<unsigned>((n.T + sh.rows - 1) / sh.rows);
  const int threads = sh.P * sh.rows;
  return with_dtype(n.dtype, [&](auto tag) {
    using T = decltype(tag);
    const size_t smem = vec ? 0 : threads / 32 * 512 * sizeof(T);
    auto go = [&](auto v) {
      constexpr bool V = decltype(v)::value;
      if (sh.G == 1) rms_norm_kernel<T, V, 1><<<grid, threads, smem, s>>>(a);
      else if (sh.G == 2) rms_norm_kernel<T, V, 2><<<grid, threads, smem, s>>>(a);
      else rms_norm_kernel<T, V, 0><<<grid, threads, smem, s>>>(a);
      return cudaGetLastError();
    };
    return vec ? go(std::true_type{}) : go(std::false_type{});
  });
}

cudaError_t launch_rms_norm_backward(const NormBackLaunch& n, cudaStream_t s) {
  if (n.T == 0) return cudaMemsetAsync(n.d_weight, 0, sizeof(float) * static_cast<size_t>(n.H), s);
  const int elem = dtype_size(n.dtype);
  const Shape sh = shape_for((n.H + 15) / 16);
  const int64_t pitch = static_cast<int64_t>(n.H) * elem;
  const NormBackArgs a{n.d_y, n.d_y_stride, n.h, n.h_stride, n.weight, n.weight_dtype == MM_MOE_DTYPE_F32, n.rstd, n.d_h,
                       n.d_h_stride, n.T, n.H, n.d_x, static_cast<float*>(n.scratch), back_pitch(n.H), sh.P};
  const bool vec = whole_groups(n.d_y, n.d_y_stride * elem, n.H) && whole_groups(n.h, n.h_stride * elem, n.H) &&
                   whole_groups(n.d_h, n.d_h_stride * elem, n.H) && whole_groups(n.d_x, pitch, n.H) &&
                   whole_groups(n.weight, 0, n.H);
  const int arrays = n.d_h ? 3 : 2;
  const RingShape ring = ring_for(n.T, n.H, elem, arrays, vec, 224, 256, kBackRingBytes);     // back_ctas at most
  int count = ring.ctas;
  cudaError_t e;
  if (ring.stages) {
    int* report = nullptr;
    e = mx_report(&report);
    if (e != cudaSuccess) return e;
    const int smem = RowRing::bytes(ring.stages, arrays, static_cast<uint32_t>(pitch));
    e = with_dtype(n.dtype, [&](auto tag) {
      using T = decltype(tag);
      return with_ring<T>(a.w_f32, ring.G, [&](auto w, auto g) {
        auto kernel = rms_norm_backward_ring_kernel<T, decltype(w), decltype(g)::value>;
        if (cudaError_t c = configure_kernel(reinterpret_cast<const void*>(kernel), 0, kBackRingBytes + 1024)) return c;
        kernel<<<ring.ctas, ring.threads, smem, s>>>(a, ring.stages, report);
        return cudaGetLastError();
      });
    });
  } else {
    const int64_t all = (n.T + sh.rows - 1) / sh.rows;
    count = static_cast<int>(all < back_ctas(n.T) ? all : back_ctas(n.T));
    const int threads = sh.P * sh.rows;
    e = with_dtype(n.dtype, [&](auto tag) {
      using T = decltype(tag);
      size_t smem = vec ? 0 : threads / 32 * 512 * sizeof(T);
      if (sh.rows > 1 && smem < static_cast<size_t>(threads) * 64) smem = static_cast<size_t>(threads) * 64;
      auto go = [&](auto v) {
        constexpr bool V = decltype(v)::value;
        if (sh.G == 1) rms_norm_backward_kernel<T, V, 1><<<count, threads, smem, s>>>(a);
        else if (sh.G == 2) rms_norm_backward_kernel<T, V, 2><<<count, threads, smem, s>>>(a);
        else rms_norm_backward_kernel<T, V, 0><<<count, threads, smem, s>>>(a);
        return cudaGetLastError();
      };
      return vec ? go(std::true_type{}) : go(std::false_type{});
    });
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((n.H + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_weight_kernel, static_cast<const float*>(a.parts), a.pitch, count, n.H, n.d_weight);
}

}  // namespace mm

// The 4-bit linear of a few rows in one launch: x is quantised (mx_quant.cuh) by
// every CTA for itself, and the weights are read once from global memory into
// registers, with no tensor cores: at one to four rows a weight row is two dot
// products of small integers per 16-byte load.
//
// Twice an e2m1 value is an integer of 4 bits and a sign (0, 1, 2, 3, 4, 6, 8, 12), so a
// block of 32 is eight 4-way integer dots, exact, times 2^(ea + eb - 2), exact where
// the result is in fp32's range (a weight scale below one is multiplied first: the dot,
// up to 4608, times x's scale alone may pass the largest fp32); the blocks are summed
// in fp32, each lane's in ascending order, then over the warp in a fixed tree.
//
// What bounds it is latency, then the weights' bytes. A warp takes two weight
// rows and a lane one block of 32 (16 bytes) of each per step; the first steps'
// loads are issued before x is quantised. A CTA takes sets of sixteen rows, chosen
// so that their scales (mx_sf_word) fill whole 32-byte sectors, and quantises x once
// for all of its sets.
#include "mx_quant.cuh"

namespace mm {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;            // steps of 1024 elements whose weights are loaded before x is there

struct FewArgs {
  const void* x;
  int64_t stride;
  int C, N, NB, KB;                  // NB: 128-row scale blocks of one expert's weights
  const uint8_t* w;
  const uint8_t* w_sf;
  const int32_t* slot;               // routed: pair p's row (grid y = pairs); null: rows 0 .. rows-1 (grid y = 1)
  const int32_t* blk_off;
  int E, K;
  int64_t num_rows;
  char* out;
  int64_t out_stride;                // elements
  int32_t* status;
};

// Four bytes of the eight in {b, a}, one per selector nibble; a nibble's top bit spreads its byte's sign bit instead.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Eight e2m1 codes -> twice their values as two words of four int8, in order.
__device__ __forceinline__ uint2 twice_values(uint32_t w) {
  const uint32_t mag = w & 0x77777777u, low = w << 4;
  // each byte's top bit is the sign of an odd code (in w) or of an even one (in w << 4), spread over the byte
  const uint32_t s0 = prmt(low, w, 0xD9C8), s1 = prmt(low, w, 0xFBEA);
  const uint32_t p0 = prmt(0x03020100u, 0x0C080604u, mag), p1 = prmt(0x03020100u, 0x0C080604u, mag >> 16);
  const uint32_t n0 = prmt(0xFDFEFF00u, 0xF4F8FAFCu, mag), n1 = prmt(0xFDFEFF00u, 0xF4F8FAFCu, mag >> 16);
  return make_uint2((p0 & ~s0) | (n0 & s0), (p1 & ~s1) | (n1 & s1));
}

// NT rows of x at most per CTA (one where routed).
template <typename T, int NT, bool kVec>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 3 : 2) few_kernel(const FewArgs a, int rows, int sets) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int n32 = a.C / 32;
  // per row of x: the first and second 16 int8 of every block, then every block's scale
  uint4* s_lo = reinterpret_cast<uint4*>(smem);
  uint4* s_hi = s_lo + NT * n32;
  float* s_sc = reinterpret_cast<float*>(s_hi + NT * n32);
  __shared__ int s_expert;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (a.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 4) a.status[threadIdx.x] = 0;

  int64_t row0 = 0, token0 = 0;
  int e = 0;
  if (a.slot) {
    row0 = __ldg(a.slot + blockIdx.y);
    token0 = blockIdx.y / a.K;
    if (row0 < 0 || row0 >= a.num_rows) return;      // the same for the whole CTA
    const int b = static_cast<int>(row0 >> 7);
    if (threadIdx.x == 0) s_expert = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kThreads)
      if (__ldg(a.blk_off + i) <= b && b < __ldg(a.blk_off + i + 1)) s_expert = i;
    __syncthreads();
    e = s_expert;
    if (e < 0) return;                               // a row of no expert's block
  }
  for (int set = blockIdx.x; set < sets; set += gridDim.x) {
    // the warp's two weight rows: n and n + 1
    const int n = (set >> 3) * 128 + (set & 7) * 4 + (warp & 1) * 2 + (warp >> 1) * 32;
    const uint4* wr[2];
    const uint8_t* sr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int m = min(n + r, a.N - 1);               // past the last row: its values again, not stored
      wr[r] = reinterpret_cast<const uint4*>(a.w + (static_cast<int64_t>(e) * a.N + m) * (a.C / 2));
      sr[r] = a.w_sf + static_cast<size_t>(e) * a.NB * a.KB * kSFChunk + mx_sf_word(m, 0, a.KB);
    }
    uint4 wv[kAhead][2];
    uint32_t sv[kAhead][2];
    auto load = [&](int u, int b) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        wv[u][r] = b < n32 ? __ldg(wr[r] + b) : make_uint4(0, 0, 0, 0);
        sv[u][r] = b < n32 ? __ldg(sr[r] + static_cast<size_t>(b >> 2) * kSFChunk + (b & 3)) : 0u;
      }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, u * 32 + lane);

    if (set == static_cast<int>(blockIdx.x)) {
      // x: two lanes a block
      const T* x = static_cast<const T*>(a.x) + token0 * a.stride;
      const int groups = NT * n32 * 2;
      for (int g0 = 0; g0 < groups; g0 += kThreads) {
        const int g = g0 + threadIdx.x;
        const int t = g / (n32 * 2), q = g - t * n32 * 2;
        Group<T> v;
        if (g < groups && t < rows) v.template load<kVec>(x + t * a.stride, q * 16, a.C);
        else v.clear();
        uint2 codes;
        const uint32_t byte = quantize_group(v, codes);
        if (g < groups) {
          const uint2 v0 = twice_values(codes.x), v1 = twice_values(codes.y);
          const int b = t * n32 + (q >> 1);
          ((q & 1) ? s_hi : s_lo)[b] = make_uint4(v0.x, v0.y, v1.x, v1.y);
          if ((q & 1) == 0) s_sc[b] = ue8m0_value(byte) * 0.25f;
        }
      }
      __syncthreads();
    }

    float acc[2][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[0][t] = acc[1][t] = 0.f;
    for (int b0 = 0; b0 < n32; b0 += 32 * kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int b = b0 + u * 32 + lane;
        if (b < n32) {
          uint2 d[2][4];
          float sc[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            d[r][0] = twice_values(wv[u][r].x);
            d[r][1] = twice_values(wv[u][r].y);
            d[r][2] = twice_values(wv[u][r].z);
            d[r][3] = twice_values(wv[u][r].w);
            sc[r] = ue8m0_value(sv[u][r]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 lo = s_lo[t * n32 + b], hi = s_hi[t * n32 + b];
            const float sx = s_sc[t * n32 + b];
            const uint32_t xs[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              int dot = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                dot = __dp4a(static_cast<int>(d[r][i].x), static_cast<int>(xs[2 * i]), dot);
                dot = __dp4a(static_cast<int>(d[r][i].y), static_cast<int>(xs[2 * i + 1]), dot);
              }
              // Neither order of the two scales loses a result that fits: with sc < 1 first, |dot| * sc is below 4608
              // and, an integer times a power of two of 2^-127 at least, exact; with sx first where sc >= 1, a product
              // that overflows does so with sc too.
              const bool below = sc[r] < 1.0f;
              acc[r][t] += static_cast<float>(dot) * (below ? sc[r] : sx) * (below ? sx : sc[r]);
            }
          }
        }
        load(u, b + 32 * kAhead);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float v = acc[r][t];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0 && n + r < a.N && t < rows)
          reinterpret_cast<T*>(a.out)[(row0 + t) * a.out_stride + n + r] = from_float<T>(v);
      }
  }
}

template <typename T, int NT>
cudaError_t launch_few(const FewArgs& a, int rows, int64_t groups, cudaStream_t s) {
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) | static_cast<uintptr_t>(a.stride * sizeof(T))) % 32 == 0;
  auto kernel = vec ? few_kernel<T, NT, true> : few_kernel<T, NT, false>;
  const int smem = NT * (a.C / 32) * 36;
  if (cudaError_t e = configure_kernel(reinterpret_cast<const void*>(kernel), 0, kMxFewSmem)) return e;
  // as many CTAs as the SMs hold, spread over the groups
  const int sets = (a.N + 127) / 128 * 8;
  const int64_t room = static_cast<int64_t>(dev_info().sms) * (NT <= 2 ? 3 : 2) / groups;
  const dim3 grid(static_cast<unsigned>(sets < room ? sets : (room < 1 ? 1 : room)), static_cast<unsigned>(groups));
  kernel<<<grid, kThreads, smem, s>>>(a, rows, sets);
  return cudaGetLastError();
}

}  // namespace

// Where one launch is the faster: its time grows with rows * N * C, the tensor-core kernels' (up to 128 rows) hardly
// with the rows. Measured (us, this kernel / the others): 1 row, 8192x4096 8.4 / 10.5, 16384x8192 21.6 / 18.8; 2 rows,
// 4096x4096 6.1 / 7.9, 8192x4096 10.1 / 10.4, 16384x8192 25.6 / 18.8; 4 rows, 4096x4096 7.7 / 7.9, 8192x4096
// 13.1 / 10.5; 4 pairs 4096x4096 16.2 / 20.3, 8 pairs 24.5 / 19.9.
bool mx_few_rows(int T, int C, int N, int K) {
  const int64_t rows = K ? static_cast<int64_t>(T) * K : (T <= 1 ? 1 : (T <= 2 ? 2 : 4));
  if (K ? rows > kMxFewPairs : T > kMxFewTokens) return false;
  const int64_t smem = (K ? 1 : rows) * (C / 32) * 36;     // codes and scales of x
  return rows * N <= kMxFewWork / C && smem <= kMxFewSmem;
}

cudaError_t launch_mx_few(const MxQuantArgs& q, const MxProductArgs& p, cudaStream_t s) {
  const FewArgs a{q.x, q.stride, p.C, p.N, (p.N + 127) / 128, mx_chunks(p.C), p.w, p.w_sf, q.slot, p.blk_off, p.E,
                  q.slot ? q.K : 1, p.rows, static_cast<char*>(p.out), p.out_stride, p.status};
  return with_dtype(p.dtype, [&](auto tag) {
    using T = decltype(tag);
    if (q.slot) return launch_few<T, 1>(a, 1, q.R * q.K, s);
    const int rows = static_cast<int>(q.R);
    if (rows <= 1) return launch_few<T, 1>(a, rows, 1, s);
    if (rows <= 2) return launch_few<T, 2>(a, rows, 1, s);
    return launch_few<T, 4>(a, rows, 1, s);
  });
}

}  // namespace mm

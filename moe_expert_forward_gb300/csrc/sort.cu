// The routing of one batch in one launch: counts, block offsets, the pool row of
// every (token, k) pair and the pair of every pool row, with the results of the
// two dispatch kernels (kernels_misc.cu) bit for bit.
//
// One cluster of up to 16 CTAs takes the pairs, every warp a contiguous run of
// them.  Each warp counts its experts in shared memory (equal experts of 32
// pairs found with votes), a CTA turns its warps' counts into offsets, the
// CTAs read one another's totals through distributed shared memory, and every
// warp then ranks its pairs.  The order inside an expert is ascending pair.
// What bounds it is latency, a chain of a few barriers, then each SM's scattered
// stores; the two dispatch kernels spread over all SMs and take over where a warp's
// run gets long. Measured (us, this kernel / the two): 1024 pairs over 256 experts
// 6.3 / 12.3, 49152 over 384 9.9 / 20.5, over 256 65536 10.5 / 16.5, 131072 15.5 / 18.5,
// 196608 21.0 / 20.6, 229376 23.7 / 20.6, 262144 25.5 / 20.7; 196608 over 64 18.8 / 18.5,
// over 384 21.8 / 28.0, over 1024 26.0 / 45.2.
#include "cluster.cuh"
#include "internal.h"

namespace mm {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;       // more than 8 is an opt-in of the kernel
constexpr int kBatch = 8;             // a lane's index loads in flight
constexpr unsigned kAll = 0xffffffffu;

struct SortArgs {
  const int32_t* idx;
  int64_t pairs;
  int64_t per;               // pairs of a warp, a multiple of 32
  int E, block_m;
  int32_t *cnt, *blk_off, *slot, *src, *status;
};

// The valid lanes whose expert is this lane's (any mask where this one is not valid): a vote per bit of the ids.
// (__match_any_sync took 2000 cycles for the 32 warps of a CTA, these votes a few hundred.)
__device__ __forceinline__ unsigned same_expert(int e, bool valid, int bits) {
  unsigned m = __ballot_sync(kAll, valid);
#pragma unroll 2
  for (int b = 0; b < bits; ++b) {
    const bool one = (e >> b) & 1;
    const unsigned v = __ballot_sync(kAll, one);
    m &= one ? v : ~v;
  }
  return m;
}

__global__ void __launch_bounds__(kThreads, 1) sort_kernel(const SortArgs a) {
  extern __shared__ int sm[];
  const int E = a.E;
  int* wc = sm;                       // [kWarps][E]: counts, then each warp's offset inside the CTA's share
  int* s_tot = wc + kWarps * E;       // [E + 1]: this CTA's pairs of each expert; [E]: ids out of range seen
  int* s_start = s_tot + E + 1;       // [E]: the pool row of this CTA's first pair of each expert
  int* s_cnt = s_start + E;           // [E]: all pairs of each expert
  int* s_blk = s_cnt + E;             // [E + 1]: first blocks
  __shared__ int s_warp[kWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank(), ctas = cluster_nctarank();
  const int gw = static_cast<int>(rank) * kWarps + w;

  const int bits = 32 - __clz(E - 1);  // of an id; 0 for one expert
  for (int i = tid; i < kWarps * E; i += kThreads) wc[i] = 0;
  __syncthreads();
  const int64_t beg = gw * a.per;
  const int64_t end = beg + a.per < a.pairs ? beg + a.per : a.pairs;
  int* my = wc + w * E;
  bool bad = false;
  for (int64_t p0 = beg; p0 < end; p0 += 32 * kBatch) {
    int ev[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t p = p0 + j * 32 + lane;
      ev[j] = p < end ? __ldg(a.idx + p) : -1;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (p0 + j * 32 >= end) break;  // the same for the warp
      const int e = ev[j];
      const bool valid = e >= 0 && e < E;
      bad |= e < -1 || e >= E;
      const unsigned m = same_expert(e, valid, bits);
      if (valid && lane == __ffs(m) - 1) my[e] += __popc(m);
      __syncwarp();
    }
  }
  const int any_bad = __syncthreads_or(bad);
  if (tid == 0) s_tot[E] = any_bad;
  for (int e = tid; e < E; e += kThreads) {
    int run = 0;
#pragma unroll 8
    for (int i = 0; i < kWarps; ++i) {
      const int c = wc[i * E + e];
      wc[i * E + e] = run;
      run += c;
    }
    s_tot[e] = run;
  }
  cluster_barrier();
  // totals over the cluster; E <= kThreads: one expert a thread, and a scan of its blocks
  int base = 0, tot = 0;
  if (tid < E)
    for (uint32_t c = 0; c < ctas; ++c) {
      const int v = peer_int(s_tot + tid, c);
      base += c < rank ? v : 0;
      tot += v;
    }
  const int blocks = (tot + a.block_m - 1) / a.block_m;
  int incl = blocks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) s_warp[w] = incl;
  __syncthreads();
  if (w == 0) {
    int v = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kAll, v, o);
      if (lane >= o) v += n;
    }
    s_warp[lane] = v;
  }
  __syncthreads();
  const int first = incl - blocks + (w ? s_warp[w - 1] : 0);
  if (tid < E) {
    s_start[tid] = first * a.block_m + base;
    s_cnt[tid] = tot;
    s_blk[tid] = first;
    if (rank == 0) {
      a.cnt[tid] = tot;
      a.blk_off[tid] = first;
    }
  }
  if (tid == kThreads - 1) {
    s_blk[E] = first + blocks;
    if (rank == 0) a.blk_off[E] = first + blocks;
  }
  if (rank == 0 && tid < 4) {
    int code = 0;
    if (tid == 0)
      for (uint32_t c = 0; c < ctas; ++c) code |= peer_int(s_tot + E, c);
    a.status[tid] = code ? MM_MOE_ERR_BAD_ROUTING : 0;
  }
  cluster_barrier();                     // the totals were read: a CTA may leave; and s_start is there

  for (int64_t p0 = beg; p0 < end; p0 += 32 * kBatch) {
    int ev[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t p = p0 + j * 32 + lane;
      ev[j] = p < end ? __ldg(a.idx + p) : -1;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (p0 + j * 32 >= end) break;
      const int64_t p = p0 + j * 32 + lane;
      const int e = ev[j];
      const bool valid = e >= 0 && e < E;
      const unsigned m = same_expert(e, valid, bits);
      int before = 0;
      if (valid) before = my[e];
      __syncwarp();
      if (valid) {
        const int row = s_start[e] + before + __popc(m & ((1u << lane) - 1u));
        a.slot[p] = row;
        a.src[row] = static_cast<int32_t>(p);
        if (lane == __ffs(m) - 1) my[e] = before + __popc(m);
      } else if (p < end) {
        a.slot[p] = -1;
      }
      __syncwarp();
    }
  }
  for (int e = gw; e < E; e += static_cast<int>(ctas) * kWarps) {
    const int64_t hi = static_cast<int64_t>(s_blk[e + 1]) * a.block_m;
    for (int64_t r = static_cast<int64_t>(s_blk[e]) * a.block_m + s_cnt[e] + lane; r < hi; r += 32) a.src[r] = -1;
  }
}

}  // namespace

bool sort_in_one_launch(int64_t pairs) { return pairs <= kSortOneLaunchPairs; }

cudaError_t launch_sort(const int32_t* topk_idx, int T, int K, int E, int block_m, int32_t* cnt, int32_t* blk_off,
                        int32_t* slot, int32_t* src, int32_t* status, int32_t* scratch, int64_t scratch_ints,
                        cudaStream_t s) {
  const int64_t pairs = static_cast<int64_t>(T) * K;
  if (!sort_in_one_launch(pairs)) {
    cudaError_t e = cudaMemsetAsync(status, 0, 16, s);
    if (e != cudaSuccess) return e;
    return launch_dispatch(topk_idx, T, K, E, block_m, cnt, blk_off, slot, src, status, scratch, scratch_ints, s);
  }
  // as many CTAs as keep a warp's run at 32 pairs, then longer runs; 4 at least, for the padding rows (1024 pairs
  // over 256 experts: 1 CTA 8.3 us, 4 CTAs 6.3)
  int ctas = 4;
  while (ctas < kMaxCluster && pairs > static_cast<int64_t>(ctas) * kWarps * 32) ctas *= 2;
  int64_t per = (pairs + ctas * kWarps - 1) / (ctas * kWarps);
  per = (per + 31) / 32 * 32;
  const SortArgs a{topk_idx, pairs, per, E, block_m, cnt, blk_off, slot, src, status};
  auto smem = [](int e) { return static_cast<int>(((kWarps + 4) * e + 2) * sizeof(int)); };
  const void* fn = reinterpret_cast<const void*>(sort_kernel);
  if (cudaError_t e = configure_kernel(fn, 0, smem(kMaxE))) return e;
  if (ctas > 8)
    if (cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem(E);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas; attr.val.clusterDim.y = 1; attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_kernel, a);
}

}  // namespace mm

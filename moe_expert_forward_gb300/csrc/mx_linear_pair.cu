// The dense 4-bit product (mx_linear.cu) on CTA pairs, for many rows: a task is two
// 128-row blocks times 256 weight rows, 4-bit codes streamed in stages of 256
// elements, M = 256, N = 256 tcgen05 cta_group::2 MMAs.  (Routed rows stay with the
// single-CTA kernel: an expert's last odd block would leave half a pair idle, and
// from 256 to 2048 rows an expert pairs measured between 9 % slower and 3 % faster.)
//
// Why pairs: what bounds the product is how fast the L2 feeds the SMs, not the
// tensor cores. CTA r holds row block r and weight rows [128 r, 128 r + 128) of
// the tile, so an SM fetches 35 KB a stage where a 128 x 256 tile of its own
// takes 51 KB, and six stages fit instead of four.
//
// Every copy of both CTAs completes on the leader's stage barrier. One leader
// thread waits for it and copies the scales of both CTAs into tensor memory (6
// instructions), another waits for that and issues 4 MMAs: with the copies, the
// commits and one wait in one thread a stage measured 724 cycles alone, apart 513,
// the MMAs' own time. The epilogue packs 16-bit results into registers and hands
// the accumulator back before it stores them.
//
// Measured: 8192 x 7168 x 4096 in 85 us, 5.7 PFLOP/s, 830 cycles a stage; with the
// copies but no MMAs 72 us, with MMAs at their own rate it would be 52. (A relay of
// per-CTA barriers through cluster-scope arrivals took 1650 cycles a stage, scales
// stored to tensor memory by warps 1725, one thread for copies and MMAs 1190. Tiles of
// 256 x 384, which fetch a sixth less: 91 us against 90, 385 against 379 at 65536 x
// 4096 x 4096, 43 against 33 at 2048 x 7168 x 4096.)
//
// Warps per CTA: 8 epilogue, 1 MMA and 1 scale-copy (the leader's issue; both
// CTAs' MMA warps allocate TMEM), 6 producers (one a stage). Every wait is bounded.
#include "cluster.cuh"
#include "mx_linear.cuh"

namespace mm {
namespace {

constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kMmaWarp = kEpiWarps;
constexpr int kScaleWarp = kMmaWarp + 1;
constexpr int kProducer0 = kScaleWarp + 1;
constexpr int kThreads = 32 * (kProducer0 + kStages);
constexpr int kTileN = 256;
constexpr int kSfCols = 24;                      // per stage: 8 of A, 16 of B
constexpr int kSfCol0 = kTileN;
constexpr int kTmemCols = 512;
constexpr int kCtaBytes = 2 * kMxTileBytes + 3 * kMxSfBytes;   // one CTA's copies of a stage
static_assert(kSfCol0 + kStages * kSfCols <= kTmemCols, "tensor memory");

struct Smem {
  static constexpr int tok = 0;
  static constexpr int wgt = tok + kStages * kMxTileBytes;
  static constexpr int sfa = wgt + kStages * kMxTileBytes;
  static constexpr int sfb = sfa + kStages * kMxSfBytes;
  static constexpr int bars = sfb + kStages * 2 * kMxSfBytes;
  static constexpr int nbars = 3 * kStages + 4;  // full, ready, empty, tfull, tempty, 2 drains
  static constexpr int exit = bars + nbars * 8 + 16;   // per stage: phases the leader armed, phases the peer loaded
  static constexpr int total = exit + 2 * kStages * 4 + 1024;
};
static_assert(Smem::total <= 232448, "shared memory");

enum : int {
  kSiteEmpty = 171, kSiteFull = 172, kSiteReady = 173, kSiteTmemEmpty = 174, kSiteTmemFull = 175,
  kSiteDrainCopies = 176, kSiteDrainMma = 177, kSiteDrainEmpty = 178
};

// each CTA's 512-byte chunk at the descriptor's offset goes to the same TMEM columns of that CTA
__device__ __forceinline__ void tc_cp_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Copies into this CTA's shared memory that complete on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void st_cluster_int(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

struct Maps {
  CUtensorMap w, a;
  CUtensorMap w_sf, sf;      // scale chunks as [128-row blocks][chunks x 2][256 bytes]
};

__device__ __forceinline__ void tc_mma_mxf4_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// This CTA's share of pair task i: its row block and the rows of it that exist (0: a ghost, which
// computes the pair's first block again and stores nothing).
struct Task {
  int b, n, valid;
};
__device__ __forceinline__ Task task_at(int i, uint32_t rank, const MxArgs& a) {
  Task t;
  const int pb = i / a.NT;
  t.n = i - pb * a.NT;
  t.b = 2 * pb;
  t.valid = min(kMxRows, a.rows - (t.b + static_cast<int>(rank)) * kMxRows);
  if (t.valid > 0) t.b += static_cast<int>(rank);
  else t.valid = 0;
  return t;
}

template <typename T, bool kLines>
__global__ void __launch_bounds__(kThreads, 1)
    mx_product_pair_kernel(const __grid_constant__ Maps maps, const MxArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem::bars);   // leader: both CTAs' copies of a stage landed
  uint64_t* ready = full + kStages;              // leader: the stage's scales are in tensor memory
  uint64_t* empty = ready + kStages;             // the stage's MMAs have completed
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 1;                  // leader: both CTAs have read the accumulator
  uint64_t* drain = tempty + 1;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full + Smem::nbars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_armed = reinterpret_cast<int*>(smem + Smem::exit);
  int* s_peer = s_armed + kStages;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const Status st{args.status, args.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&ready[i], 1);
      mbar_init(&empty[i], 1);
      s_armed[i] = 0;
      s_peer[i] = 0;
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kEpiWarps);
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_barrier();                             // both CTAs' barriers exist before anything targets them
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int ntasks = (args.nblk + 1) / 2 * args.NT;
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;

  if (warp >= kProducer0) {
    // ------------------------------------------------------------------ TMA producers, one per stage
    if (lane == 0) {
      const int p = warp - kProducer0;
      const uint64_t pol = policy_evict_normal();
      uint8_t* tk = smem + Smem::tok + p * kMxTileBytes;
      uint8_t* wt = smem + Smem::wgt + p * kMxTileBytes;
      uint8_t* sa = smem + Smem::sfa + p * kMxSfBytes;
      uint8_t* sb = smem + Smem::sfb + p * 2 * kMxSfBytes;
      const uint32_t bar = map_shared(&full[p], 0);
      int step = 0;                              // stages of this CTA's tasks so far
      int loaded = 0;                            // phases of this stage loaded
      bool waited = args.wait_prior == 0;
      for (int i = first; i < ntasks && !*s_abort; i += stride) {
        const Task t = task_at(i, rank, args);
        int ks = ((p - step) % kStages + kStages) % kStages;
        for (; ks < args.KS; ks += kStages) {
          const uint32_t phase = ((step + ks) / kStages) & 1;
          if (args.unreachable && i + stride >= ntasks && ks == args.KS - 1) break;
          if (!mbar_wait(&empty[p], phase ^ 1, st, s_abort, kSiteEmpty)) break;
          if (rank == 0) mbar_arrive_expect_tx(&full[p], 2 * kCtaBytes);
          ++loaded;
          tma_load_2d_pair(wt, &maps.w, bar, ks * kMxStageBytes,
                           t.n * kTileN + static_cast<int>(rank) * 128, pol);
          tma_load_3d_pair(sb, &maps.w_sf, bar, 0, 4 * ks, 2 * t.n, pol);
          if (!waited) {                         // the weights do not depend on the kernel before; the rows do
            pdl_wait();
            waited = true;
          }
          tma_load_2d_pair(tk, &maps.a, bar, ks * kMxStageBytes, t.b * kMxRows, pol);
          tma_load_3d_pair(sa, &maps.sf, bar, 0, 4 * ks, t.b, pol);
        }
        step += args.KS;
      }
      if (rank == 0) {
        s_armed[p] = loaded;
        if (loaded) mbar_drain(&full[p], (loaded - 1) & 1, st, s_abort, kSiteDrainCopies);
      } else {
        st_cluster_int(map_shared(&s_peer[p], 0), loaded);
      }
      // the leader's last commit to this CTA's barrier has arrived before the CTA leaves
      if (loaded && !*s_abort) mbar_drain(&empty[p], (loaded - 1) & 1, st, s_abort, kSiteDrainEmpty);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMAs (leader)
    if (rank == 0 && lane == 0) {
      const uint64_t dtok = make_smem_desc(smem_u32(smem + Smem::tok), 16, 1024, 2);
      const uint64_t dwgt = make_smem_desc(smem_u32(smem + Smem::wgt), 16, 1024, 2);
      uint32_t phase = 0;
      int it = 0, ks = 0, task = first - stride;
      auto start_task = [&]() -> bool {
        task += stride;
        if (task >= ntasks || *s_abort) return false;
        if (!mbar_wait_cluster(tempty, (it & 1) ^ 1, st, s_abort, kSiteTmemEmpty)) return false;
        tc_fence_after();
        return true;
      };
      bool live = start_task();
      while (live) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {      // the stage index is a constant in each copy of the body
          if (live) {
            if (!mbar_wait(&ready[s], phase, st, s_abort, kSiteReady)) {
              live = false;
            } else {
              tc_fence_after();
              const uint32_t sfa = tmem + kSfCol0 + s * kSfCols;
              const uint64_t da = dtok + ((s * kMxTileBytes) >> 4);
              const uint64_t db = dwgt + ((s * kMxTileBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)     // 64 elements: 32 bytes, two descriptor units
                tc_mma_mxf4_pair(tmem, da + 2 * kk, db + 2 * kk, idesc_mxf4(kTileN, 256, kk & 1), sfa + 4 * (kk >> 1),
                                 sfa + 8 + 8 * (kk >> 1), (ks | kk) != 0);
              tc_commit_pair(map_shared(&empty[s], 0));
              tc_commit_pair(map_shared(&empty[s], 1));
              if (++ks == args.KS) {
                tc_commit_pair(map_shared(tfull, 0));
                tc_commit_pair(map_shared(tfull, 1));
                ks = 0;
                ++it;
                live = start_task();
              }
            }
          }
        }
        phase ^= 1;
      }
      tc_commit_pair(map_shared(drain, 0));
      mbar_drain(drain, 0, st, s_abort, kSiteDrainMma);
    }
    __syncwarp();
  } else if (warp == kScaleWarp) {
    // ------------------------------------------------------------------ scale copies (leader)
    if (rank == 0 && lane == 0) {
      const uint64_t dsfa = make_smem_desc(smem_u32(smem + Smem::sfa), 0, 128, 0);
      const uint64_t dsfb = make_smem_desc(smem_u32(smem + Smem::sfb), 0, 128, 0);
      uint32_t phase = 0;
      int64_t left = first < ntasks ? static_cast<int64_t>((ntasks - 1 - first) / stride + 1) * args.KS : 0;
      while (left > 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
          if (left > 0) {
            if (!mbar_wait(&full[s], phase, st, s_abort, kSiteFull)) {
              left = 0;
            } else {
              --left;
              tc_fence_after();
              const uint32_t sfa = tmem + kSfCol0 + s * kSfCols;
#pragma unroll
              for (int h = 0; h < 2; ++h) {      // 128-wide halves of the stage
                tc_cp_pair(sfa + 4 * h, dsfa + ((s * kMxSfBytes + h * kSFChunk) >> 4));
                tc_cp_pair(sfa + 8 + 8 * h, dsfb + ((2 * s * kMxSfBytes + h * kSFChunk) >> 4));
                tc_cp_pair(sfa + 12 + 8 * h, dsfb + (((2 * s + 1) * kMxSfBytes + h * kSFChunk) >> 4));
              }
              tc_commit_pair(map_shared(&ready[s], 0));
            }
          }
        }
        phase ^= 1;
      }
      tc_commit_pair(map_shared(drain + 1, 0));
      mbar_drain(drain + 1, 0, st, s_abort, kSiteDrainMma);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    constexpr int kCols = kTileN / 2;            // columns of one warp
    const int c0 = (warp >> 2) * kCols;
    const uint32_t src = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c0;
    int it = 0;
    for (int i = first; i < ntasks; i += stride, ++it) {
      const Task t = task_at(i, rank, args);
      if (!mbar_wait_warp(tfull, it & 1, st, s_abort, kSiteTmemFull)) break;
      tc_fence_after();
      const int n = t.n * kTileN + c0;
      const int row0 = (warp & 3) * 32;
      char* dst = args.out + (static_cast<int64_t>(t.b) * kMxRows + row0) * args.out_pitch + n * sizeof(T);
      store_accumulator<T, kCols, kLines>(src, dst, args.out_pitch, t.valid - row0, args.N - n, lane, [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_shared(tempty, 0));
      });
    }
  }
  // Each role waited for what it issued; the peer's copies complete on the leader's barriers. After the first
  // barrier the peer has issued its last copy: a phase it loaded that the leader never armed (the leader stopped
  // first, on a timeout) is armed with the peer's share and waited for. After the second nothing targets either CTA.
  __syncthreads();
  cluster_barrier();
  if (rank == 0 && threadIdx.x < kStages) {
    const int p = threadIdx.x;
    if (s_peer[p] > s_armed[p]) {
      mbar_arrive_expect_tx(&full[p], kCtaBytes);
      mbar_drain(&full[p], (s_peer[p] - 1) & 1, st, s_abort, kSiteDrainCopies);
    }
  }
  __syncthreads();
  cluster_barrier();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  if (threadIdx.x == 0) note_given_up(args, s_abort);
}

}  // namespace

cudaError_t launch_mx_product_pair(const MxProductArgs& p, cudaStream_t s) {
  return with_dtype(p.dtype, [&](auto tag) {
    using T = decltype(tag);
    const MxArgs a = mx_args(p, sizeof(T), kTileN);
    Maps maps;
    if (mx_codes_map(&maps.w, p.w, p.N, p.C, 128) != CUDA_SUCCESS ||
        mx_codes_map(&maps.a, p.codes, p.rows, p.C, kMxRows) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    // a stage's two chunks of two weight row blocks (past the last one: zeros, in columns that are not stored), and
    // of one activation block
    auto scales_map = [&](CUtensorMap* m, const uint8_t* sf, int64_t row_blocks, uint32_t box) {
      const uint64_t dims[3] = {256, static_cast<uint64_t>(a.KB) * 2, static_cast<uint64_t>(row_blocks)};
      const uint64_t strides[2] = {256, static_cast<uint64_t>(a.KB) * kSFChunk};
      const uint32_t boxes[3] = {256, 4, box};
      return encode_tmap(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, sf, dims, strides, boxes, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    if (scales_map(&maps.w_sf, p.w_sf, a.NB, 2) != CUDA_SUCCESS ||
        scales_map(&maps.sf, p.sf, a.nblk, 1) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
    auto kernel = a.lines ? mx_product_pair_kernel<T, true> : mx_product_pair_kernel<T, false>;
    const void* fn = reinterpret_cast<const void*>(kernel);
    if (cudaError_t e = configure_kernel(fn, 0, Smem::total)) return e;
    int clusters = 0;
    if (cudaError_t e = max_pair_clusters(fn, kThreads, Smem::total, &clusters)) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    const int64_t tasks = static_cast<int64_t>((a.nblk + 1) / 2) * a.NT;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * static_cast<unsigned>(tasks < clusters ? tasks : clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem::total;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2; attr[0].val.clusterDim.y = 1; attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.after_quantize ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a);
  });
}

}  // namespace mm

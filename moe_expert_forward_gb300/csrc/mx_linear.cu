// Products of microscaled 4-bit operands: out[r, n] = sum over c of
// a[r, c] w[e, n, c], a and w e2m1 values times one power of two per 32
// elements of the contraction, e the expert that owns row r's 128-row block (or
// the one matrix of a dense product).  The products are exact, the sums fp32.
//
// tcgen05 kind::mxf4 takes both operands as packed nibbles, 64 elements of the
// contraction per MMA, and their scales from tensor memory.  A task is one
// 128-row block times BN weight rows; the contraction runs in stages of 256
// elements (128 bytes of codes a row, one 128-byte swizzle atom), four MMAs a
// stage.  Persistent CTAs take tasks in a fixed stride, block-major, so the
// weight tiles of an expert with several blocks are read again from L2.
//
// Warps: 4 or 8 epilogue warps (one or two per TMEM lane quadrant), one that
// issues scale copies and MMAs, and one TMA producer per stage.
// Every wait is bounded; on a timeout each role winds down what it issued.
#include <mutex>

#include "cluster.cuh"
#include "mx_linear.cuh"

namespace mm {
namespace {

enum : int {
  kSiteEmpty = 161, kSiteFull = 162, kSiteTmemEmpty = 163, kSiteTmemFull = 164, kSiteDrainCopies = 165,
  kSiteDrainMma = 166
};

template <int BN>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 4 : (BN == 128 ? 6 : 8);
  static constexpr int kEpiWarps = BN == 64 ? 4 : 8;
  static constexpr int kThreads = 32 * (kEpiWarps + 1 + kStages);
  static constexpr int kAccBufs = BN == 256 ? 1 : 2;
  static constexpr int kWgtBytes = BN * kMxStageBytes;
  static constexpr int kWgtBlocks = (BN + 127) / 128;            // 128-row scale blocks of a weight tile
  static constexpr int kSfCols = 8 + 8 * kWgtBlocks;             // TMEM columns of a stage's scales
  static constexpr int kSfCol0 = kAccBufs * BN;
  static constexpr int kTmemCols = kSfCol0 + kStages * kSfCols <= 256 ? 256 : 512;
  static constexpr int tok = 0;
  static constexpr int wgt = tok + kStages * kMxTileBytes;
  static constexpr int sft = wgt + kStages * kWgtBytes;
  static constexpr int sfw = sft + kStages * kMxSfBytes;
  static constexpr int bars = sfw + kStages * kWgtBlocks * kMxSfBytes;
  static constexpr int nbars = 2 * kStages + 2 * kAccBufs + 1;   // full, empty, tfull, tempty, drain
  static constexpr int meta = bars + nbars * 8 + 16;             // blk_off[E + 1], cnt[E]
  static int total(int E) { return meta + (2 * E + 1) * 4 + 1024; }
  static constexpr int kPartPitch = BN + 4;                      // floats of a row of partial sums
  static_assert(kMxRows * kPartPitch * 4 <= sft, "partial sums fit the stages");
  static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory");
  static_assert(meta + (2 * kMaxE + 1) * 4 + 1024 <= 232448, "shared memory");
};

struct Maps {
  CUtensorMap w;
  CUtensorMap a[3];          // activation rows in boxes of 32, 64 and 128
};

__device__ __forceinline__ void tc_mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

struct Task {
  int b, n, e, valid;        // row block, weight tile, expert, rows of the block that exist
};

// Task i of the CTA-strided list: block-major, then weight tile.
__device__ __forceinline__ Task task_at(int i, const MxArgs& a, const int* s_blk, const int* s_cnt) {
  Task t;
  t.b = i / a.NT;
  t.n = i - t.b * a.NT;
  if (a.blk_off) {
    t.e = last_not_above(s_blk, a.E, t.b);       // the last expert that starts at or before block b
    t.valid = min(kMxRows, s_cnt[t.e] - (t.b - s_blk[t.e]) * kMxRows);
  } else {
    t.e = 0;
    t.valid = min(kMxRows, a.rows - t.b * kMxRows);
  }
  return t;
}

// kSplit: a cluster takes one task, each CTA a range of its stages; the partial accumulators meet in shared memory.
// kLines: see store_accumulator.
template <int BN, typename T, bool kSplit, bool kLines>
__global__ void __launch_bounds__(Cfg<BN>::kThreads, 1)
    mx_product_kernel(const __grid_constant__ Maps maps, const MxArgs args) {
  using C = Cfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::bars);
  uint64_t* full = bars;
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + C::kAccBufs;
  uint64_t* drain = tempty + C::kAccBufs;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + C::nbars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_blk = reinterpret_cast<int*>(smem + C::meta);
  int* s_cnt = s_blk + args.E + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const Status st{args.status, args.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kAccBufs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kEpiWarps) {
    tmem_alloc(s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (args.blk_off) {
    for (int i = threadIdx.x; i <= args.E; i += C::kThreads) s_blk[i] = args.blk_off[i];
    for (int i = threadIdx.x; i < args.E; i += C::kThreads) s_cnt[i] = args.cnt[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int ntasks = (args.blk_off ? min(s_blk[args.E], args.rows / kMxRows) : args.nblk) * args.NT;

  // this CTA's tasks, and its stages [k0, k0 + nks) of each
  const int part = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int parts = kSplit ? static_cast<int>(cluster_nctarank()) : 1;
  const int first = static_cast<int>(blockIdx.x) / parts, stride = static_cast<int>(gridDim.x) / parts;
  const int k0 = kSplit ? args.KS * part / parts : 0;
  const int nks = kSplit ? args.KS * (part + 1) / parts - k0 : args.KS;

  if (warp > C::kEpiWarps) {
    // ------------------------------------------------------------------ TMA producers, one per stage
    if (lane == 0) {
      const int p = warp - C::kEpiWarps - 1;
      const uint64_t pol = policy_evict_normal();
      uint8_t* tk = smem + C::tok + p * kMxTileBytes;
      uint8_t* wt = smem + C::wgt + p * C::kWgtBytes;
      uint8_t* sa = smem + C::sft + p * kMxSfBytes;
      uint8_t* sw = smem + C::sfw + p * C::kWgtBlocks * kMxSfBytes;
      int step = 0;                              // stages of this CTA's tasks so far
      bool armed = false, waited = args.wait_prior == 0;
      uint32_t armed_parity = 0;
      for (int i = first; i < ntasks && !*s_abort; i += stride) {
        const Task t = task_at(i, args, s_blk, s_cnt);
        const int box = t.valid > 64 ? 2 : (t.valid > 32 ? 1 : 0);
        const int n0 = t.n * BN;
        const int nb0 = n0 / 128;
        const int nbs = min(C::kWgtBlocks, args.NB - nb0);
        const uint32_t bytes = (32u << box) * kMxStageBytes + C::kWgtBytes + (1 + nbs) * kMxSfBytes;
        int ks = ((p - step) % S + S) % S;
        for (; ks < nks; ks += S) {
          const uint32_t phase = ((step + ks) / S) & 1;
          if (args.unreachable && i + stride >= ntasks && ks == nks - 1) break;
          if (!mbar_wait(&empty[p], phase ^ 1, st, s_abort, kSiteEmpty)) break;
          mbar_arrive_expect_tx(&full[p], bytes);
          armed = true;
          armed_parity = phase;
          tma_load_2d(wt, &maps.w, &full[p], (k0 + ks) * kMxStageBytes, t.e * args.N + n0, pol);
          for (int j = 0; j < nbs; ++j)
            bulk_load(sw + j * kMxSfBytes,
                      args.w_sf + ((static_cast<size_t>(t.e) * args.NB + nb0 + j) * args.KB + 2 * (k0 + ks)) * kSFChunk,
                      kMxSfBytes, &full[p]);
          if (!waited) {                         // the weights do not depend on the kernel before; the rows do
            pdl_wait();
            waited = true;
          }
          tma_load_2d(tk, &maps.a[box], &full[p], (k0 + ks) * kMxStageBytes, t.b * kMxRows, pol);
          bulk_load(sa, args.sf + (static_cast<size_t>(t.b) * args.KB + 2 * (k0 + ks)) * kSFChunk, kMxSfBytes, &full[p]);
        }
        step += nks;
      }
      if (armed) mbar_drain(&full[p], armed_parity, st, s_abort, kSiteDrainCopies);
    }
  } else if (warp == C::kEpiWarps) {
    // ------------------------------------------------------------------ scale copies and MMAs
    if (lane == 0) {
      const uint64_t dtok = make_smem_desc(smem_u32(smem + C::tok), 16, 1024, 2);
      const uint64_t dwgt = make_smem_desc(smem_u32(smem + C::wgt), 16, 1024, 2);
      const uint64_t dsft = make_smem_desc(smem_u32(smem + C::sft), 0, 128, 0);
      const uint64_t dsfw = make_smem_desc(smem_u32(smem + C::sfw), 0, 128, 0);
      uint32_t phase = 0;
      int it = 0, ks = 0, task = first - stride;
      uint32_t acc = 0, sfw_shift = 0;
      auto start_task = [&]() -> bool {
        task += stride;
        if (task >= ntasks || *s_abort) return false;
        const int buf = it % C::kAccBufs;
        acc = tmem + buf * BN;
        // a 64-row tile's scales are the lower or upper two of a chunk's four columns
        sfw_shift = BN == 64 ? ((task % args.NT) & 1) * 2 : 0;
        if (!mbar_wait(&tempty[buf], ((it / C::kAccBufs) & 1) ^ 1, st, s_abort, kSiteTmemEmpty)) return false;
        tc_fence_after();
        return true;
      };
      bool live = start_task();
      while (live) {
#pragma unroll
        for (int s = 0; s < S; ++s) {            // the stage index is a constant in each copy of the body
          if (live) {
            if (!mbar_wait(&full[s], phase, st, s_abort, kSiteFull)) {
              live = false;
            } else {
              tc_fence_after();
              const uint32_t sfa = tmem + C::kSfCol0 + s * C::kSfCols;
              const uint32_t sfb = sfa + 8;
#pragma unroll
              for (int h = 0; h < 2; ++h) {      // 128-wide halves of the stage
                tc_cp_32x128b_warpx4(sfa + 4 * h, dsft + ((s * kMxSfBytes + h * kSFChunk) >> 4));
#pragma unroll
                for (int j = 0; j < C::kWgtBlocks; ++j)
                  tc_cp_32x128b_warpx4(sfb + h * 4 * C::kWgtBlocks + 4 * j,
                                       dsfw + (((s * C::kWgtBlocks + j) * kMxSfBytes + h * kSFChunk) >> 4));
              }
              const uint64_t da = dtok + ((s * kMxTileBytes) >> 4);
              const uint64_t db = dwgt + ((s * C::kWgtBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)     // 64 elements: 32 bytes, two descriptor units
                tc_mma_mxf4(acc, da + 2 * kk, db + 2 * kk, idesc_mxf4(BN, kMxRows, kk & 1), sfa + 4 * (kk >> 1),
                            sfb + (kk >> 1) * 4 * C::kWgtBlocks + sfw_shift, (ks | kk) != 0);
              tc_commit(&empty[s]);
              if (++ks == nks) {
                tc_commit(&tfull[it % C::kAccBufs]);
                ks = 0;
                ++it;
                live = start_task();
              }
            }
          }
        }
        phase ^= 1;
      }
      tc_commit(drain);
      mbar_drain(drain, 0, st, s_abort, kSiteDrainMma);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    constexpr int kCols = C::kEpiWarps == 8 ? BN / 2 : BN;       // columns of one warp
    const int quad = warp & 3;
    const int c0 = C::kEpiWarps == 8 ? (warp >> 2) * kCols : 0;
    int it = 0;
    for (int i = first; i < ntasks; i += stride, ++it) {
      const Task t = task_at(i, args, s_blk, s_cnt);
      const int buf = it % C::kAccBufs;
      if (!mbar_wait_warp(&tfull[buf], (it / C::kAccBufs) & 1, st, s_abort, kSiteTmemFull)) break;
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * BN + c0;
      const int row = quad * 32 + lane;
      if constexpr (kSplit) {                    // every MMA of the task has completed: the stages' memory is free
        float* d = reinterpret_cast<float*>(smem) + row * C::kPartPitch + c0;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(src + c, v);
          tmem_ld_wait();
          if (row < t.valid)
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(d + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
        continue;
      }
      const int n = t.n * BN + c0;
      char* dst = args.out + (static_cast<int64_t>(t.b) * kMxRows + quad * 32) * args.out_pitch + n * sizeof(T);
      store_accumulator<T, kCols, kLines>(src, dst, args.out_pitch, t.valid - quad * 32, args.N - n, lane, [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
      });
    }
  }
  if constexpr (kSplit) {
    // every CTA adds up its share of the columns, the parts in order
    cluster_barrier();
    if (first < ntasks) {
      const Task t = task_at(first, args, s_blk, s_cnt);
      const int quads = BN / 4 / parts;          // groups of four columns
      for (int i = threadIdx.x; i < t.valid * quads; i += C::kThreads) {
        const int row = i / quads;
        const int c = part * (BN / parts) + (i - row * quads) * 4;
        const float* src = reinterpret_cast<const float*>(smem) + row * C::kPartPitch + c;
        float4 sum = peer_float4(src, 0);
        for (int s = 1; s < parts; ++s) {
          const float4 v = peer_float4(src, s);
          sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
        }
        Vec<T, 4> o;
        o.v[0] = from_float<T>(sum.x); o.v[1] = from_float<T>(sum.y);
        o.v[2] = from_float<T>(sum.z); o.v[3] = from_float<T>(sum.w);
        const int n = t.n * BN + c;
        T* dst = reinterpret_cast<T*>(args.out + (static_cast<int64_t>(t.b) * kMxRows + row) * args.out_pitch) + n;
        if (kLines && n + 4 <= args.N) {
          *reinterpret_cast<Vec<T, 4>*>(dst) = o;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < args.N) dst[j] = o.v[j];
        }
      }
    }
    cluster_barrier();                           // the others have read this CTA's part
  }
  __syncthreads();
  if (warp == C::kEpiWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (threadIdx.x == 0) note_given_up(args, s_abort);
}

static __device__ int32_t g_report[4];

constexpr int kMaxDevices = 64;
int32_t* g_report_addr[kMaxDevices] = {nullptr};
std::mutex g_report_mu;

template <int BN, typename T, bool kSplit>
cudaError_t launch_impl(const MxProductArgs& p, int parts, cudaStream_t s) {
  using C = Cfg<BN>;
  Maps maps;
  const MxArgs a = mx_args(p, sizeof(T), BN);
  if (mx_codes_map(&maps.w, p.w, static_cast<int64_t>(p.E) * p.N, p.C, BN) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  for (int i = 0; i < 3; ++i)
    if (mx_codes_map(&maps.a[i], p.codes, p.rows, p.C, 32 << i) != CUDA_SUCCESS) return cudaErrorInvalidValue;
  auto kernel = a.lines ? mx_product_kernel<BN, T, kSplit, true> : mx_product_kernel<BN, T, kSplit, false>;
  if (cudaError_t e = configure_kernel(reinterpret_cast<const void*>(kernel), 0, C::total(kMaxE))) return e;
  const int64_t tasks = static_cast<int64_t>(a.nblk) * a.NT;
  const int sms = dev_info().sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(kSplit ? tasks * parts : (tasks < sms ? tasks : sms)));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::total(p.blk_off ? p.E : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (p.after_quantize) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (kSplit) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = parts; attr[na].val.clusterDim.y = 1; attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

// Weight rows of a tile and CTAs that share a task's contraction.
struct Tile {
  int bn, parts;
};

// The cheapest of the tile widths and splits by a model in SM cycles: a stage costs 560 and 1.75 per weight row;
// splitting costs 1500, a quarter cycle per partial sum of a CTA, and 36 per CTA for launching clusters. Measured
// (rows x N x C, us with the quantiser): 512x4096x4096 at 128/1 12.8, 256/1 14.1, 256/2 15.1, 64/1 19.1;
// 128x4096x7168 at 128/4 13.0, 128/1 15.8, 256/4 14.1, 64/1 16.6; 64x1000x4096 at 64/4 7.8, 256/1 27.2, 64/1 14.3.
// Clusters of 8 gain nothing over 4: too few of them fit a GPC.
Tile choose_tile(int64_t blocks, int rows, int N, int KS, int sms) {
  Tile best{256, 1};
  int64_t least = INT64_MAX;
  for (int bn = 256; bn >= 64; bn /= 2) {
    const int64_t tasks = blocks * ((N + bn - 1) / bn);
    for (int parts = 1; parts <= 4 && parts <= KS; parts *= 2) {
      if (parts > 1 && tasks * parts > sms) break;
      const int64_t waves = (tasks * parts + sms - 1) / sms;
      const int64_t split = parts > 1 ? 1500 + static_cast<int64_t>(rows) * bn / 4 + 36 * tasks * parts : 0;
      const int64_t cost = waves * ((KS + parts - 1) / parts) * (560 + 7 * bn / 4) + split;
      if (cost < least) {
        least = cost;
        best = {bn, parts};
      }
    }
  }
  return best;
}

template <typename T, bool kSplit>
cudaError_t launch_tile(const MxProductArgs& p, const Tile& t, cudaStream_t s) {
  if (t.bn == 256) return launch_impl<256, T, kSplit>(p, t.parts, s);
  if (t.bn == 128) return launch_impl<128, T, kSplit>(p, t.parts, s);
  return launch_impl<64, T, kSplit>(p, t.parts, s);
}

}  // namespace

cudaError_t mx_report(int32_t** record) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_report_mu);
  if (!g_report_addr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_report);
    if (e != cudaSuccess) return e;
    g_report_addr[dev] = static_cast<int32_t*>(p);
  }
  *record = g_report_addr[dev];
  return cudaSuccess;
}

cudaError_t launch_mx_product(const MxProductArgs& args, cudaStream_t s) {
  if (args.rows == 0) return cudaSuccess;
  MxProductArgs p = args;
  if (cudaError_t e = mx_report(&p.report)) return e;
  const int64_t blocks = (p.rows + kMxRows - 1) / kMxRows;
  const int sms = dev_info().sms;
  const int KS = mx_chunks(p.C) / 2;
  // pairs where every pair of SMs has a whole task of full blocks and a task has 16 stages or more: a shorter one is
  // mostly hand-over (us with the quantiser, pairs / one CTA a tile, 8192 x C x 4096: C 7168 109 / 119, 4096 72 / 74,
  // 512 24 / 19; 2048 x 7168 x 4096 34.8 / 36.4)
  const int64_t full_pairs = p.blk_off ? 0 : p.rows / (2 * kMxRows);
  if (KS >= 16 && full_pairs * ((p.N + 255) / 256) >= sms / 2) return launch_mx_product_pair(p, s);
  const Tile t = choose_tile(blocks, p.rows < kMxRows ? static_cast<int>(p.rows) : kMxRows, p.N, KS, sms);
  return with_dtype(p.dtype, [&](auto tag) {
    using T = decltype(tag);
    return t.parts > 1 ? launch_tile<T, true>(p, t, s) : launch_tile<T, false>(p, t, s);
  });
}

}  // namespace mm

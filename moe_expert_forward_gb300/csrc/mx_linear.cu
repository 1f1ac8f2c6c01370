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
#include "mx_linear.h"
#include "ptx.cuh"
#include "rowtypes.cuh"

namespace mm {
namespace {

constexpr int kBM = 128;
constexpr int kStageK = 256;                     // contraction elements per stage
constexpr int kStageBytes = kStageK / 2;         // of one row's codes
constexpr int kTokBytes = kBM * kStageBytes;
constexpr int kSfBytes = 2 * kSFChunk;           // the two chunks of 128 rows

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
  static constexpr int kWgtBytes = BN * kStageBytes;
  static constexpr int kWgtBlocks = (BN + 127) / 128;            // 128-row scale blocks of a weight tile
  static constexpr int kSfCols = 8 + 8 * kWgtBlocks;             // TMEM columns of a stage's scales
  static constexpr int kSfCol0 = kAccBufs * BN;
  static constexpr int kTmemCols = kSfCol0 + kStages * kSfCols <= 256 ? 256 : 512;
  static constexpr int tok = 0;
  static constexpr int wgt = tok + kStages * kTokBytes;
  static constexpr int sft = wgt + kStages * kWgtBytes;
  static constexpr int sfw = sft + kStages * kSfBytes;
  static constexpr int bars = sfw + kStages * kWgtBlocks * kSfBytes;
  static constexpr int nbars = 2 * kStages + 2 * kAccBufs + 1;   // full, empty, tfull, tempty, drain
  static constexpr int meta = bars + nbars * 8 + 16;             // blk_off[E + 1], cnt[E]
  static int total(int E) { return meta + (2 * E + 1) * 4 + 1024; }
  static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory");
  static_assert(meta + (2 * kMaxE + 1) * 4 + 1024 <= 232448, "shared memory");
};

struct Args {
  int rows, C, E, N;
  int KS, KB;                // 256-wide stages, scale chunks along the contraction
  int NB, NT;                // 128-row scale blocks and BN-row tiles of one expert's weights
  int nblk;                  // row blocks of a dense product
  const uint8_t* sf;
  const uint8_t* w_sf;
  const int* cnt;
  const int* blk_off;
  char* out;
  int64_t out_pitch;         // bytes
  int wide;                  // out rows and base are 32-byte aligned
  int wait_prior;            // launched programmatically: activations come from the kernel before
  int* status;
  uint64_t timeout_ns;
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

// Instruction descriptor of kind::mxf4: A and B e2m1 (1) in [9:7] and [11:10],
// both K-major, N >> 3 in [22:17], UE8M0 scales (bit 23), M >> 7 in [28:27];
// the scale bytes a 64-wide MMA takes from each 32-bit word: 0 (bytes 0, 1) or 2
// (bytes 2, 3) in [30:29] for A and [5:4] for B.
__host__ __device__ constexpr uint32_t idesc_mxf4(int n, int m, int half) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 7) << 27) | (static_cast<uint32_t>(2 * half) << 29) |
         (static_cast<uint32_t>(2 * half) << 4);
}

struct Task {
  int b, n, e, valid;        // row block, weight tile, expert, rows of the block that exist
};

// Task i of the CTA-strided list: block-major, then weight tile.
__device__ __forceinline__ Task task_at(int i, const Args& a, const int* s_blk, const int* s_cnt) {
  Task t;
  t.b = i / a.NT;
  t.n = i - t.b * a.NT;
  if (a.blk_off) {
    int lo = 0, hi = a.E - 1;                    // the last expert that starts at or before block b
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_blk[mid] <= t.b) lo = mid; else hi = mid - 1;
    }
    t.e = lo;
    t.valid = min(kBM, s_cnt[lo] - (t.b - s_blk[lo]) * kBM);
  } else {
    t.e = 0;
    t.valid = min(kBM, a.rows - t.b * kBM);
  }
  return t;
}

// 32 accumulator columns of one row, to N - c columns at most.
template <typename T>
__device__ __forceinline__ void store_columns(T* p, const uint32_t (&v)[32], int cols, bool wide) {
  if (wide && cols >= 32) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) st_global_v8(reinterpret_cast<float*>(p) + 8 * i, v + 8 * i);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        Vec<T, 2> h;
        h.v[0] = from_float<T>(__uint_as_float(v[2 * i]));
        h.v[1] = from_float<T>(__uint_as_float(v[2 * i + 1]));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      st_global_v8(reinterpret_cast<float*>(p), w);
      st_global_v8(reinterpret_cast<float*>(p) + 8, w + 8);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < cols) p[i] = from_float<T>(__uint_as_float(v[i]));
  }
}

template <int BN, typename T>
__global__ void __launch_bounds__(Cfg<BN>::kThreads, 1)
    mx_product_kernel(const __grid_constant__ Maps maps, const Args args) {
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
  const int ntasks = (args.blk_off ? min(s_blk[args.E], args.rows / kBM) : args.nblk) * args.NT;

  if (warp > C::kEpiWarps) {
    // ------------------------------------------------------------------ TMA producers, one per stage
    if (lane == 0) {
      const int p = warp - C::kEpiWarps - 1;
      const uint64_t pol = policy_evict_normal();
      uint8_t* tk = smem + C::tok + p * kTokBytes;
      uint8_t* wt = smem + C::wgt + p * C::kWgtBytes;
      uint8_t* sa = smem + C::sft + p * kSfBytes;
      uint8_t* sw = smem + C::sfw + p * C::kWgtBlocks * kSfBytes;
      int step = 0;                              // stages of this CTA's tasks so far
      bool armed = false, waited = args.wait_prior == 0;
      uint32_t armed_parity = 0;
      for (int i = blockIdx.x; i < ntasks && !*s_abort; i += gridDim.x) {
        const Task t = task_at(i, args, s_blk, s_cnt);
        const int box = t.valid > 64 ? 2 : (t.valid > 32 ? 1 : 0);
        const int n0 = t.n * BN;
        const int nb0 = n0 / 128;
        const int nbs = min(C::kWgtBlocks, args.NB - nb0);
        const uint32_t bytes = (32u << box) * kStageBytes + C::kWgtBytes + (1 + nbs) * kSfBytes;
        int ks = ((p - step) % S + S) % S;
        for (; ks < args.KS; ks += S) {
          const uint32_t phase = ((step + ks) / S) & 1;
          if (!mbar_wait(&empty[p], phase ^ 1, st, s_abort, kSiteEmpty)) break;
          mbar_arrive_expect_tx(&full[p], bytes);
          armed = true;
          armed_parity = phase;
          tma_load_2d(wt, &maps.w, &full[p], ks * kStageBytes, t.e * args.N + n0, pol);
          for (int j = 0; j < nbs; ++j)
            bulk_load(sw + j * kSfBytes,
                      args.w_sf + ((static_cast<size_t>(t.e) * args.NB + nb0 + j) * args.KB + 2 * ks) * kSFChunk,
                      kSfBytes, &full[p]);
          if (!waited) {                         // the weights do not depend on the kernel before; the rows do
            pdl_wait();
            waited = true;
          }
          tma_load_2d(tk, &maps.a[box], &full[p], ks * kStageBytes, t.b * kBM, pol);
          bulk_load(sa, args.sf + (static_cast<size_t>(t.b) * args.KB + 2 * ks) * kSFChunk, kSfBytes, &full[p]);
        }
        step += args.KS;
      }
      if (armed) mbar_wait_drain(&full[p], armed_parity, st, kSiteDrainCopies);
    }
  } else if (warp == C::kEpiWarps) {
    // ------------------------------------------------------------------ scale copies and MMAs
    if (lane == 0) {
      const uint64_t dtok = make_smem_desc(smem_u32(smem + C::tok), 16, 1024, 2);
      const uint64_t dwgt = make_smem_desc(smem_u32(smem + C::wgt), 16, 1024, 2);
      const uint64_t dsft = make_smem_desc(smem_u32(smem + C::sft), 0, 128, 0);
      const uint64_t dsfw = make_smem_desc(smem_u32(smem + C::sfw), 0, 128, 0);
      uint32_t phase = 0;
      int it = 0, ks = 0, task = static_cast<int>(blockIdx.x) - static_cast<int>(gridDim.x);
      uint32_t acc = 0, sfw_shift = 0;
      auto start_task = [&]() -> bool {
        task += gridDim.x;
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
                tc_cp_32x128b_warpx4(sfa + 4 * h, dsft + ((s * kSfBytes + h * kSFChunk) >> 4));
#pragma unroll
                for (int j = 0; j < C::kWgtBlocks; ++j)
                  tc_cp_32x128b_warpx4(sfb + h * 4 * C::kWgtBlocks + 4 * j,
                                       dsfw + (((s * C::kWgtBlocks + j) * kSfBytes + h * kSFChunk) >> 4));
              }
              const uint64_t da = dtok + ((s * kTokBytes) >> 4);
              const uint64_t db = dwgt + ((s * C::kWgtBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)     // 64 elements: 32 bytes, two descriptor units
                tc_mma_mxf4(acc, da + 2 * kk, db + 2 * kk, idesc_mxf4(BN, kBM, kk & 1), sfa + 4 * (kk >> 1),
                            sfb + (kk >> 1) * 4 * C::kWgtBlocks + sfw_shift, (ks | kk) != 0);
              tc_commit(&empty[s]);
              if (++ks == args.KS) {
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
      mbar_wait_drain(drain, 0, st, kSiteDrainMma);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    constexpr int kCols = C::kEpiWarps == 8 ? BN / 2 : BN;       // columns of one warp
    const int quad = warp & 3;
    const int c0 = C::kEpiWarps == 8 ? (warp >> 2) * kCols : 0;
    int it = 0;
    for (int i = blockIdx.x; i < ntasks; i += gridDim.x, ++it) {
      const Task t = task_at(i, args, s_blk, s_cnt);
      const int buf = it % C::kAccBufs;
      if (!mbar_wait(&tfull[buf], (it / C::kAccBufs) & 1, st, s_abort, kSiteTmemFull)) break;
      tc_fence_after();
      const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * BN + c0;
      const int row = quad * 32 + lane;
      const int n = t.n * BN + c0;
      T* dst = reinterpret_cast<T*>(args.out + (static_cast<int64_t>(t.b) * kBM + row) * args.out_pitch) + n;
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(src + c, v);
        tmem_ld_wait();
        if (c + 32 == kCols) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        }
        if (row < t.valid) store_columns(dst + c, v, args.N - n - c, args.wide != 0);
      }
    }
  }
  __syncthreads();
  if (warp == C::kEpiWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BN, typename T>
cudaError_t launch_impl(const MxProductArgs& p, cudaStream_t s) {
  using C = Cfg<BN>;
  Maps maps;
  Args a{};
  a.rows = static_cast<int>(p.rows);
  a.C = p.C; a.E = p.E; a.N = p.N;
  a.KB = mx_chunks(p.C); a.KS = a.KB / 2;
  a.NB = (p.N + 127) / 128; a.NT = (p.N + BN - 1) / BN;
  a.nblk = static_cast<int>((p.rows + kBM - 1) / kBM);
  a.sf = p.sf; a.w_sf = p.w_sf; a.cnt = p.cnt; a.blk_off = p.blk_off;
  a.out = static_cast<char*>(p.out);
  a.out_pitch = p.out_stride * static_cast<int64_t>(sizeof(T));
  a.wide = (reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(a.out_pitch)) % 32 == 0;
  a.wait_prior = p.after_quantize;
  a.status = p.status; a.timeout_ns = p.timeout_ns;
  const uint64_t pitch = static_cast<uint64_t>(p.C) / 2;
  if (encode_tmap_2d(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, pitch, static_cast<uint64_t>(p.E) * p.N, pitch,
                     kStageBytes, BN, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  for (int i = 0; i < 3; ++i)
    if (encode_tmap_2d(&maps.a[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, p.codes, pitch, static_cast<uint64_t>(p.rows), pitch,
                       kStageBytes, 32u << i, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  auto kernel = mx_product_kernel<BN, T>;
  if (cudaError_t e = configure_kernel(reinterpret_cast<const void*>(kernel), 0, C::total(kMaxE))) return e;
  const int64_t tasks = static_cast<int64_t>(a.nblk) * a.NT;
  const int sms = dev_info().sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tasks < sms ? tasks : sms));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::total(p.blk_off ? p.E : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.after_quantize ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

}  // namespace

cudaError_t launch_mx_product(const MxProductArgs& p, cudaStream_t s) {
  if (p.rows == 0) return cudaSuccess;
  // the widest weight tile that still gives every SM a task
  const int64_t blocks = (p.rows + kBM - 1) / kBM;
  const int sms = dev_info().sms;
  return with_dtype(p.dtype, [&](auto tag) {
    using T = decltype(tag);
    if (blocks * ((p.N + 255) / 256) >= sms) return launch_impl<256, T>(p, s);
    if (blocks * ((p.N + 127) / 128) >= sms) return launch_impl<128, T>(p, s);
    return launch_impl<64, T>(p, s);
  });
}

}  // namespace mm

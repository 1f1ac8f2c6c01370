// Weight gradients from rows kept in 8 bits: out[e][n][c] = sum over expert e's rows r
// of d_y[r][n] x[r][c], d_y in bf16 and x as e4m3 codes with UE8M0 scales per 32
// columns (or one dense sum over all rows).  x is exact in bf16, so the products are
// those of kind::f16 tcgen05 MMAs with fp32 sums, rounded once.
//
// The contraction runs over rows, the slow dimension of both operands in memory, so
// both are MN-major: 64 columns (128 bytes) of 8 rows are one swizzle atom.  The scale
// of x belongs to a (row, 32 columns) block and cannot be one of the MMA's own scales,
// which run along the contraction: converter warps decode codes into bf16 on their way
// into shared memory instead, where TMA brings d_y next to them.
//
// A task is 128 columns of d_y (M) times 256 of x (N) of one expert; the contraction
// runs in stages of 64 rows, four MMAs a stage.  Persistent CTAs take tasks in a fixed
// stride; the accumulator is double buffered, so that a task's stores overlap the next
// one's products.
//
// Warps: 8 epilogue, 1 MMA, 1 TMA producer, 8 converters.  Every wait is bounded.
#include "cluster.cuh"
#include "mx_linear.cuh"
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kStages = 4;
constexpr int kRowsPerStage = 64;
constexpr int kTileN = 128;                      // columns of d_y: M
constexpr int kTileC = 256;                      // columns of x: N
constexpr int kEpiWarps = 8, kMmaWarp = 8, kTmaWarp = 9, kConvert0 = 10, kConvertWarps = 8;
constexpr int kThreads = 32 * (kConvert0 + kConvertWarps);
constexpr int kAtom = 1024;                      // 8 rows of 64 columns
constexpr int kChunkBytes = kRowsPerStage * 128; // 64 columns of a stage
constexpr int kABytes = kTileN / 64 * kChunkBytes, kBBytes = kTileC / 64 * kChunkBytes;

struct Smem {
  static constexpr int a = 0;
  static constexpr int b = a + kStages * kABytes;
  static constexpr int bars = b + kStages * kBBytes;
  static constexpr int nbars = 3 * kStages + 5;  // full of A and of B, empty, tfull, tempty, drain
  static constexpr int meta = bars + nbars * 8 + 16;             // blk_off[E + 1], cnt[E]
  static int total(int E) { return meta + (2 * E + 1) * 4 + 1024; }
};
static_assert(Smem::meta + (2 * kMaxE + 1) * 4 + 1024 <= 232448, "shared memory");

enum : int {
  kSiteEmpty = 181, kSiteFullA = 182, kSiteFullB = 183, kSiteTmemEmpty = 184, kSiteTmemFull = 185,
  kSiteDrainCopies = 186, kSiteDrainMma = 187
};

struct Args {
  const __nv_bfloat16* d_y;
  int64_t dy_stride;
  int N, C, E, block_m;
  int NT, CT;                // tiles of N and of C
  int rows;                  // of d_y
  const uint8_t* codes;
  const uint8_t* sf;
  int pitch, blocks;         // bytes of a row of codes, scales of a row
  const int* cnt;            // null: dense
  const int* blk_off;
  const int* src;            // x's rows are tokens: pool row -> pair; null: x's rows are d_y's
  int K;
  char* out;
  int64_t out_pitch;         // bytes of a row of out
  int unreachable;           // leave x of the CTA's last stage out
  int* report;
  uint64_t timeout_ns;
};

// kind::f16: fp32 accumulator (1 in [5:4]), A and B bf16 (1 in [9:7] and [12:10]), both MN-major (bits 15 and 16),
// N >> 3 in [22:17], M >> 4 in [28:24].
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            (static_cast<uint32_t>(kTileC >> 3) << 17) | (static_cast<uint32_t>(kTileN >> 4) << 24);

__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// this thread's shared-memory stores before later reads by the tensor cores
__device__ __forceinline__ void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

struct Task {
  int e, n0, c0;
  int64_t row0;              // first row of the expert
  int rows;                  // its rows
};
__device__ __forceinline__ Task task_at(int i, const Args& a, const int* s_blk, const int* s_cnt) {
  Task t;
  const int nt = i % a.NT;
  i /= a.NT;
  const int ct = i % a.CT;
  t.e = i / a.CT;
  t.n0 = nt * kTileN;
  t.c0 = ct * kTileC;
  t.row0 = a.cnt ? static_cast<int64_t>(s_blk[t.e]) * a.block_m : 0;
  t.rows = a.cnt ? max(0, static_cast<int>(min(static_cast<int64_t>(s_cnt[t.e]), a.rows - t.row0))) : a.rows;
  return t;
}

// Two e4m3 codes, in bytes 1 and 3 of w, as bf16 times 2^-120: sign to bit 15, exponent and fraction to bits 10 to 4, where
// they stand for the same value with bf16's larger bias (subnormals too).
__device__ __forceinline__ uint32_t widen(uint32_t w) { return ((w >> 4) & 0x07F007F0u) | (w & 0x80008000u); }
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 codes times 2^(byte - 127) as 16 bf16, exact where bf16 has the value. Byte 255: NaN.
__device__ __forceinline__ void to_bf16(const uint4& c, uint32_t byte, uint32_t (&w)[8]) {
  const uint32_t in[4] = {c.x, c.y, c.z, c.w};
  // 2^(byte - 127) 2^120 has the exponent field byte + 120; past 254 in two factors
  const uint32_t f1 = min(byte + 120u, 254u) << 7, p1 = byte == 255u ? 0x7FC07FC0u : f1 | (f1 << 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[2 * i] = mul_bf16x2(widen(__byte_perm(in[i], 0, 0x1404)), p1);
    w[2 * i + 1] = mul_bf16x2(widen(__byte_perm(in[i], 0, 0x3424)), p1);
  }
  if (byte > 134u) {
    const uint32_t f2 = (min(byte, 254u) - 134u + 127u) << 7, p2 = f2 | (f2 << 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = mul_bf16x2(w[i], p2);
  }
}

// One stage of x as a converter lane holds it: 16 columns of each of its four rows.
struct Fetched {
  uint4 c[4];
  uint32_t byte[4];
};

// kTma: d_y comes by TMA (16-byte aligned rows); else the converters load it.
template <typename T, bool kTma, bool kLines>
__global__ void __launch_bounds__(kThreads, 1)
    weight_grad_kernel(const __grid_constant__ CUtensorMap map, const Args args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + Smem::bars);
  uint64_t* full_b = full_a + kStages;
  uint64_t* empty = full_b + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full_a + Smem::nbars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_blk = reinterpret_cast<int*>(smem + Smem::meta);
  int* s_cnt = s_blk + args.E + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const Status st{args.report, args.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_a[i], 1);
      mbar_init(&full_b[i], kConvertWarps);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (args.cnt) {
    for (int i = threadIdx.x; i <= args.E; i += kThreads) s_blk[i] = args.blk_off[i];
    for (int i = threadIdx.x; i < args.E; i += kThreads) s_cnt[i] = args.cnt[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int ntasks = args.E * args.NT * args.CT;
  const int first = blockIdx.x, stride = gridDim.x;

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------------ d_y by TMA
    if (kTma && lane == 0) {
      const uint64_t pol = policy_evict_normal();
      int step = 0;                              // stages so far
      int armed[kStages];                        // phases armed of each stage
#pragma unroll
      for (int s = 0; s < kStages; ++s) armed[s] = 0;
      bool live = true;
      for (int i = first; i < ntasks && live; i += stride) {
        const Task t = task_at(i, args, s_blk, s_cnt);
        const int nks = (t.rows + kRowsPerStage - 1) / kRowsPerStage;
        for (int ks = 0; ks < nks && live; ++ks, ++step) {
          const int s = step % kStages;
          live = !*s_abort && mbar_wait(&empty[s], ((step / kStages) & 1) ^ 1, st, s_abort, kSiteEmpty);
          if (!live) break;
          mbar_arrive_expect_tx(&full_a[s], kABytes);
#pragma unroll
          for (int q = 0; q < kStages; ++q) armed[q] += q == s;
          uint8_t* d = smem + Smem::a + s * kABytes;
          const int row = static_cast<int>(t.row0) + ks * kRowsPerStage;
          tma_load_2d(d, &map, &full_a[s], t.n0, row, pol);
          tma_load_2d(d + kChunkBytes, &map, &full_a[s], t.n0 + 64, row, pol);
        }
      }
#pragma unroll
      for (int s = 0; s < kStages; ++s)
        if (armed[s]) mbar_drain(&full_a[s], (armed[s] - 1) & 1, st, s_abort, kSiteDrainCopies);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      // 64-column chunks kChunkBytes apart, 8-row groups one atom apart
      const uint64_t da0 = make_smem_desc(smem_u32(smem + Smem::a), kChunkBytes, kAtom, 2);
      const uint64_t db0 = make_smem_desc(smem_u32(smem + Smem::b), kChunkBytes, kAtom, 2);
      int step = 0, it = 0;
      bool live = true;
      for (int i = first; i < ntasks && live; i += stride) {
        const Task t = task_at(i, args, s_blk, s_cnt);
        if (t.rows == 0) continue;
        const int buf = it & 1;
        live = !*s_abort && mbar_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, st, s_abort, kSiteTmemEmpty);
        tc_fence_after();
        const uint32_t acc = tmem + buf * kTileC;
        for (int row = 0; row < t.rows && live; row += kRowsPerStage, ++step) {
          const int s = step % kStages;
          const uint32_t phase = (step / kStages) & 1;
          if (kTma) live = mbar_wait(&full_a[s], phase, st, s_abort, kSiteFullA);
          live = live && mbar_wait(&full_b[s], phase, st, s_abort, kSiteFullB);
          if (!live) break;
          tc_fence_after();
          const uint64_t da = da0 + ((s * kABytes) >> 4), db = db0 + ((s * kBBytes) >> 4);
          const int n = min(4, (t.rows - row + 15) / 16);
          for (int k = 0; k < n; ++k)            // 16 rows: two atoms
            tc_mma_f16(acc, da + k * (2 * kAtom >> 4), db + k * (2 * kAtom >> 4), kIdesc, (row | k) != 0);
          tc_commit(&empty[s]);
        }
        if (!live) break;
        tc_commit(&tfull[buf]);
        ++it;
      }
      tc_commit(drain);
      mbar_drain(drain, 0, st, s_abort, kSiteDrainMma);
    }
    __syncwarp();
  } else if (warp >= kConvert0) {
    // ------------------------------------------------------------------ x into bf16
    // a warp takes 64 columns of every second group of 8 rows; 4 lanes a row, so that 8 lanes' 16-byte stores (two rows
    // of one chunk) fall into 8 different bank groups
    const int cw = warp - kConvert0, chunk = cw & 3, r8 = lane >> 2, q = lane & 3;
    int task = first - stride, ks = 0, nks = 0;
    Task t{};
    auto next = [&]() -> bool {                  // the stage after this one
      if (++ks < nks) return true;
      do {
        task += stride;
        if (task >= ntasks) return false;
        t = task_at(task, args, s_blk, s_cnt);
      } while (t.rows == 0);
      ks = 0;
      nks = (t.rows + kRowsPerStage - 1) / kRowsPerStage;
      return true;
    };
    auto fetch = [&](Fetched& f) {
      const int col = t.c0 + chunk * 64 + q * 16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ks * kRowsPerStage + ((cw >> 2) + 2 * i) * 8 + r8;
        int64_t row = -1;
        if (r < t.rows && col < args.pitch) {
          row = t.row0 + r;
          if (args.src) {
            const int pair = __ldg(args.src + row);
            row = pair < 0 ? -1 : pair / args.K;
          }
        }
        f.c[i] = make_uint4(0, 0, 0, 0);
        f.byte[i] = 127;
        if (row >= 0) {
          f.c[i] = __ldg(reinterpret_cast<const uint4*>(args.codes + row * args.pitch + col));
          f.byte[i] = __ldg(args.sf + row * args.blocks + (col >> 5));
        }
      }
    };
    int step = 0;
    bool live = next();
    Fetched f;
    if (live) fetch(f);
    while (live) {
      const Fetched g = f;
      const int rows = t.rows - ks * kRowsPerStage;      // left from this stage on
      const int n0 = t.n0;
      const int64_t row0 = t.row0 + ks * kRowsPerStage;
      live = next();
      if (live) fetch(f);
      else if (args.unreachable) break;
      const int s = step % kStages;
      const uint32_t phase = (step / kStages) & 1;
      if (!mbar_wait_warp(&empty[s], phase ^ 1, st, s_abort, kSiteEmpty)) break;
      uint8_t* b = smem + Smem::b + s * kBBytes + chunk * kChunkBytes;
      uint8_t* am = smem + Smem::a + s * kABytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[8];
        to_bf16(g.c[i], g.byte[i], w);
        uint8_t* p = b + ((cw >> 2) + 2 * i) * kAtom + r8 * 128;
        *reinterpret_cast<uint4*>(p + (((2 * q) ^ r8) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + (((2 * q + 1) ^ r8) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
      }
      if constexpr (!kTma) {                     // d_y by hand: 16 lanes a row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 16 + cw * 2 + (lane >> 4), p = lane & 15;
          const int n = args.N - (n0 + p * 8);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < rows && n > 0) {
            v = load16_any(args.d_y + (row0 + r) * args.dy_stride + n0 + p * 8, (n < 8 ? n : 8) * 2);
            if (n < 8) {
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = 2 * j + 1 < n ? w[j] : (2 * j < n ? w[j] & 0xFFFFu : 0u);
              v = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          *reinterpret_cast<uint4*>(am + (p >> 3) * kChunkBytes + (r >> 3) * kAtom + (r & 7) * 128 +
                                    (((p & 7) ^ (r & 7)) << 4)) = v;
        }
      } else if (rows < kRowsPerStage && (rows & 15)) {
        // the sum ends inside an MMA: whatever d_y's rows behind it hold becomes zero
        if (!mbar_wait_warp(&full_a[s], phase, st, s_abort, kSiteFullA)) break;
        const int end = (rows + 15) & ~15;
        for (int i = (rows * 16) + cw * 32 + lane; i < end * 16; i += 32 * kConvertWarps) {
          const int r = i >> 4, p = i & 15;
          *reinterpret_cast<uint4*>(am + (p >> 3) * kChunkBytes + (r >> 3) * kAtom + (r & 7) * 128 + ((p & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full_b[s]);
      ++step;
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    constexpr int kCols = 64;                    // columns of a warp at a time
    const int quad = warp & 3, half = (warp >> 2) * (kTileC / 2);
    int it = 0;
    for (int i = first; i < ntasks; i += stride) {
      const Task t = task_at(i, args, s_blk, s_cnt);
      const int64_t row = static_cast<int64_t>(t.e) * args.N + t.n0 + quad * 32;
      const int rows = args.N - t.n0 - quad * 32;
      if (t.rows == 0) {                         // an expert without rows
        for (int r = 0; r < 32 && r < rows; ++r) {
          T* p = reinterpret_cast<T*>(args.out + (row + r) * args.out_pitch);
          for (int c = t.c0 + half + lane; c < min(args.C, t.c0 + half + kTileC / 2); c += 32) p[c] = from_float<T>(0.f);
        }
        continue;
      }
      const int buf = it & 1;
      if (!mbar_wait_warp(&tfull[buf], (it >> 1) & 1, st, s_abort, kSiteTmemFull)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kTileC / 2; c += kCols) {
        const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kTileC + half + c;
        const int col = t.c0 + half + c;
        store_accumulator<T, kCols, kLines>(src, args.out + row * args.out_pitch + col * static_cast<int64_t>(sizeof(T)),
                                            args.out_pitch, rows, args.C - col, lane, [&] {
                                              if (c + kCols < kTileC / 2) return;
                                              tc_fence_before();
                                              __syncwarp();
                                              if (lane == 0) mbar_arrive(&tempty[buf]);
                                            });
      }
      ++it;
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T>
cudaError_t launch(const WeightGradLaunch& p, const Args& a, cudaStream_t s) {
  const bool tma = reinterpret_cast<uintptr_t>(p.d_y) % 16 == 0 && p.d_stride % 8 == 0;
  const bool lines = (reinterpret_cast<uintptr_t>(p.out) | static_cast<uintptr_t>(a.out_pitch)) % 32 == 0;
  CUtensorMap map{};
  if (tma && encode_tmap_2d(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.d_y, static_cast<uint64_t>(p.N),
                            static_cast<uint64_t>(p.rows), static_cast<uint64_t>(p.d_stride) * 2, 64, kRowsPerStage,
                            CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  auto kernel = tma ? (lines ? weight_grad_kernel<T, true, true> : weight_grad_kernel<T, true, false>)
                    : (lines ? weight_grad_kernel<T, false, true> : weight_grad_kernel<T, false, false>);
  if (cudaError_t e = configure_kernel(reinterpret_cast<const void*>(kernel), 0, Smem::total(kMaxE))) return e;
  const int64_t tasks = static_cast<int64_t>(a.E) * a.NT * a.CT;
  const int sms = dev_info().sms;
  kernel<<<static_cast<unsigned>(tasks < sms ? tasks : sms), kThreads, Smem::total(p.cnt ? a.E : 0), s>>>(map, a);
  return cudaGetLastError();
}

}  // namespace

int64_t weight_grad_tasks(int E, int N, int C) {
  return static_cast<int64_t>(E) * ((N + kTileN - 1) / kTileN) * ((C + kTileC - 1) / kTileC);
}

cudaError_t launch_weight_grad(const WeightGradLaunch& p, cudaStream_t s) {
  Args a{};
  if (cudaError_t e = mx_report(&a.report)) return e;
  a.d_y = static_cast<const __nv_bfloat16*>(p.d_y);
  a.dy_stride = p.d_stride;
  a.N = p.N; a.C = p.C; a.E = p.E; a.block_m = p.block_m;
  a.NT = (p.N + kTileN - 1) / kTileN;
  a.CT = (p.C + kTileC - 1) / kTileC;
  a.rows = static_cast<int>(p.rows);
  a.codes = p.codes; a.sf = p.sf;
  a.blocks = blocks8(p.C, MM_MOE_VARIANT_MX);
  a.pitch = a.blocks * kMxBlock;
  a.cnt = p.cnt; a.blk_off = p.blk_off; a.src = p.src; a.K = p.K;
  a.out = static_cast<char*>(p.out);
  a.out_pitch = static_cast<int64_t>(p.C) * dtype_size(p.dtype);
  a.unreachable = p.unreachable;
  a.timeout_ns = p.timeout_ns;
  return p.dtype == MM_MOE_DTYPE_F32 ? launch<float>(p, a, s) : launch<__nv_bfloat16>(p, a, s);
}

}  // namespace mm

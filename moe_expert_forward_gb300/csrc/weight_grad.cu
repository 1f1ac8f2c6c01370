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
// A task is 256 columns of d_y (M) times 256 of x (N) of one expert, by a CTA pair
// (cta_group::2); the contraction runs in stages of 64 rows, four MMAs a stage.  Why
// pairs: each CTA holds 128 columns of either operand, so a code is decoded once for 256
// columns of d_y, and a stage moves 64 KB through each SM's shared memory in the 512 cycles of
// its MMAs where a 128 x 256 tile of one CTA would move 96.  Persistent pairs take tasks
// in a fixed stride; the accumulator is double buffered, so that a task's stores overlap
// the next one's products.  Few tasks are split along the contraction into parts of their own, whose fp32 sums go to
// scratch and are added up in order by a second kernel. (Clusters of 8 CTAs that add up in shared memory do not all fit
// at once: 8192x256x4096 50 us.)
//
// The MMA's accumulation drops bits below its accumulator's last: of random sign 8192 rows in
// one accumulator are 3.7e-6 off (rounding to nearest: 3.6e-7), of one sign up to 6e-9 a row
// too small: 2^18 rows lost 1.2e-3, a third of bf16's half step and more, and 2^21 1.2e-2.  fp32
// results are sums of sums over 1024 rows (kSegment stages), added by the epilogue in memory;
// bf16 results of more than 16384 rows (kLongSegment; what one accumulator of these drops is
// 5 % of a half step at most) of sums over 16384, which the epilogue keeps in a tile of fp32
// scratch of the pair's own. How many rows an expert has is known on the device alone, and one
// may have all pairs, so the kernel that can do so (kLong) runs wherever there are more pairs,
// or dense rows (bf16, cold caches, us, one accumulator / several: 65536x4096x4096 1298 / 1325,
// 65536x1024x4096 404 / 440, 8 experts of 24576 rows and 2048x2048 993 / 1010).
//
// Codes come by TMA too, their scales by 4-byte asynchronous copies, into a ring of their own: converters that load
// for themselves keep the SM's loads in flight at their limit, and wait for it (1000 cycles a stage and more).  With
// many tiles of N, and where x's rows are tokens (TMA's own gather, four rows an instruction, took 1900 cycles a stage), a
// kernel before this one decodes x into bf16 rows, and the product takes both operands by TMA.  Rows of d_y, or of scales,
// that start on no 16-byte, or 4-byte, boundary are copied first.
//
// The loops of all roles have to fit the instruction cache together: none is unrolled over its ring (unrolled, a third
// of the fetches missed and a stage took 1500 cycles).
//
// Warps per CTA: 4 epilogue, 1 MMA (the leader's issues for both), 1 TMA producer of
// d_y, 1 of codes and scales, 1 that waits for a stage's operands, fences them towards
// the tensor cores and tells the leader, 12 converters.  Every wait is bounded.
#include "cluster.cuh"
#include "mx_linear.cuh"
#include "rows8.cuh"

namespace mm {
namespace {

constexpr int kRaw = 6;                          // stages of codes
constexpr int kRowsPerStage = 64;
constexpr int kTile = 256;                       // columns of d_y (M) and of x (N) of a pair; 128 of each in a CTA
constexpr int kEpiWarps = 4, kConvertWarps = 12;
constexpr int kMmaWarp = kEpiWarps, kTmaWarp = kMmaWarp + 1, kCodesWarp = kTmaWarp + 1, kHandWarp = kCodesWarp + 1,
              kConvert0 = kHandWarp + 1;
template <bool kDecoded>
constexpr int kThreads = 32 * (kConvert0 + (kDecoded ? 0 : kConvertWarps));
constexpr int kAtom = 1024;                      // 8 rows of 64 columns
constexpr int kChunkBytes = kRowsPerStage * 128; // 64 columns of a stage
constexpr int kHalfBytes = 2 * kChunkBytes;      // 128 columns: one CTA's share of an operand
constexpr int kRawBytes = kRowsPerStage * 128;   // 128 columns of codes
constexpr int kRawSf = kRowsPerStage * 4;        // and their scales
constexpr int kGroups = 3;                       // of converter warps, which take turns at the stages
constexpr int kRowStep = 8 * kConvertWarps / (2 * kGroups);      // between the rows of a converter lane
constexpr int kLaneRows = kRowsPerStage / kRowStep;
constexpr int kSegment = 16;                     // stages of one accumulator, fp32 results
constexpr int kLongSegment = 256;                // bf16 results
constexpr int kMostParts = 16;
constexpr int64_t kLongTerms = 1 << 18;
constexpr int kSplitPairs = 76;                  // CTA pairs that parts are made for; the scratch does not depend on the device
constexpr int kBoxBytes = 32 * 128;              // 32 rows of 128 bytes of results
constexpr size_t kPairSums = size_t(kTile) * kTile * sizeof(float);      // a pair's tile

// kDecoded: x comes in bf16. A stage then takes 1700 cycles from its copies' issue to their landing, and six of them are
// what covers that (four: 800 cycles a stage); without the ring of codes there is room.
template <bool kDecoded>
struct Smem {
  static constexpr int kStages = kDecoded ? 6 : 4;               // of operands
  static constexpr int kBoxes = kDecoded ? 1 : 2;                // of results, of an epilogue warp
  static constexpr int a = 0;
  static constexpr int b = a + kStages * kHalfBytes;
  static constexpr int raw = b + kStages * kHalfBytes;
  static constexpr int raw_sf = raw + (kDecoded ? 0 : kRaw * kRawBytes);
  static constexpr int out = (raw_sf + (kDecoded ? 0 : kRaw * kRawSf) + 1023) / 1024 * 1024;
  static constexpr int bars = out + kEpiWarps * kBoxes * kBoxBytes;
  static constexpr int nbars = 4 * kStages + 2 * kRaw + 5;       // full_a, full_b, full, empty, raw_full, raw_empty, ...
  static constexpr int meta = bars + nbars * 8 + 16;             // blk_off[E + 1], cnt[E]
  __host__ __device__ static constexpr int total(int E) { return meta + (2 * E + 1) * 4 + 1024; }
  static_assert(bars % 8 == 0 && meta + (2 * kMaxE + 1) * 4 + 1024 <= 232448, "shared memory");
};

enum : int {
  kSiteEmpty = 181, kSiteFullA = 182, kSiteFull = 183, kSiteTmemEmpty = 184, kSiteTmemFull = 185, kSiteDrainCopies = 186,
  kSiteDrainMma = 187, kSiteDrainEmpty = 188, kSiteFullB = 189, kSiteRawFull = 190,
  kSiteRawEmpty = 191
};

struct Args {
  int N, C, E, block_m;
  int NT, CT;                // tiles of N and of C
  int tasks, parts;          // E NT CT, and the parts of each
  int whole;                 // (parts 1) tasks from this one on are taken in halves of 128 columns of x; else all
  int rows;                  // of d_y
  const uint32_t* sf;
  int sf_words;              // words from one row of scales to the next
  const int* cnt;            // null: dense
  const int* blk_off;
  char* out;
  int64_t out_pitch;         // bytes of a row of out; [parts][E][N] rows
  float4* sums;              // kLong: kPairSums bytes a pair
  int unreachable;           // the CTA's last stage is not handed over
  int* report;
  uint64_t timeout_ns;
};

// kind::f16: fp32 accumulator (1 in [5:4]), A and B bf16 (1 in [9:7] and [12:10]), both MN-major (bits 15 and 16),
// N >> 3 in [22:17], M >> 4 in [28:24].
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            (static_cast<uint32_t>(kTile >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
constexpr uint32_t kIdescHalf = kIdesc - (static_cast<uint32_t>(kTile / 2 >> 3) << 17);

__device__ __forceinline__ void tc_mma_f16_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive at the same barrier of both CTAs of the pair (bits of their ranks in `ctas`) once this thread's MMAs have completed.
__device__ __forceinline__ void tc_commit_both(uint64_t* bar, uint16_t ctas) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                   smem_u32(bar)),
               "h"(ctas)
               : "memory");
}
// this thread's shared-memory stores before later reads by the tensor cores
__device__ __forceinline__ void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Arrive on the leader's barrier, releasing within this CTA: all that is handed over lies in this CTA's shared memory or
// tensor memory, fenced towards the tensor cores that use it, and no thread of the other CTA looks at it. (Releasing to
// the cluster waits for whatever the SM has in flight, about 2000 cycles a stage.)
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A part of a task: the sum over stages [ks, end) of an expert's rows.
struct Task {
  int slab, n0, c0;          // [part][expert] of out
  int cols;                  // of x: kTile, or half of it
  int row0;                  // first row of the expert
  int rows;                  // its rows
  int ks, end;
};
__device__ __forceinline__ Task task_at(int i, const Args& a, const int* s_blk, const int* s_cnt) {
  Task t;
  const int part = a.parts > 1 ? i / a.tasks : 0;
  i -= part * a.tasks;
  t.cols = kTile;
  int right = 0;
  if (a.parts == 1 && i >= a.whole) {
    t.cols = kTile / 2;
    right = (i - a.whole) & 1;
    i = a.whole + ((i - a.whole) >> 1);
  }
  const int nt = i % a.NT;
  i /= a.NT;
  const int ct = i % a.CT, e = i / a.CT;
  t.slab = part * a.E + e;
  t.n0 = nt * kTile;
  t.c0 = ct * kTile + right * (kTile / 2);
  t.row0 = a.cnt ? s_blk[e] * a.block_m : 0;
  t.rows = a.cnt ? max(0, min(s_cnt[e], a.rows - t.row0)) : a.rows;
  const int nks = (t.rows + kRowsPerStage - 1) / kRowsPerStage;
  t.ks = a.parts > 1 ? static_cast<int>(static_cast<int64_t>(nks) * part / a.parts) : 0;
  t.end = a.parts > 1 ? static_cast<int>(static_cast<int64_t>(nks) * (part + 1) / a.parts) : nks;
  return t;
}

// The stages a pair runs through, task by task.
struct Cursor {
  Task t;                    // t.ks: this stage
  int task, stride, ntasks;
  __device__ __forceinline__ Cursor(int first, int stride, int ntasks) : t{}, task(first - stride), stride(stride), ntasks(ntasks) {}
  // the next task with stages; false past the last
  __device__ __forceinline__ bool next_task(const Args& a, const int* s_blk, const int* s_cnt) {
    do {
      task += stride;
      if (task >= ntasks) return false;
      t = task_at(task, a, s_blk, s_cnt);
    } while (t.ks >= t.end);
    return true;
  }
  __device__ __forceinline__ bool next(const Args& a, const int* s_blk, const int* s_cnt) {
    return ++t.ks < t.end || next_task(a, s_blk, s_cnt);
  }
};

// 32 rows of 128 bytes from shared memory to out, or (kAdd, fp32) added to what is there.
template <bool kAdd>
__device__ __forceinline__ void tma_store_box(const CUtensorMap* m, const void* src, int c, int n, int e) {
  if constexpr (kAdd)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c), "r"(n), "r"(e)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c), "r"(n), "r"(e)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// all but this thread's last kLeft boxes have been read from shared memory; tma_stored: written
template <int kLeft>
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory"); }
__device__ __forceinline__ void tma_stored() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Waits for tensor memory loads; the registers that they fill are the wait's results, so that no use moves before it.
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// One lane of a whole warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A slot of a ring of N, in turn.
template <int N>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++s == N) {
      s = 0;
      phase ^= 1;
    }
  }
};

// Four bytes into shared memory, and (arrive_after_copies) this thread's arrival on a barrier once all such copies of it
// are there.
__device__ __forceinline__ void copy_word_async(uint32_t dst, const uint32_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 codes times 2^(byte - 127) as 16 bf16, exact where bf16 has the value; byte kNoRow: zeros.
// A code's sign, exponent and fraction at bf16's bits 15 and 10 to 4 stand for the same value times 2^-120, bf16's larger
// bias (subnormals too): the high byte is the sign and three bits of the exponent, the low one the other four bits.
// Codes of NaN (0x7F, 0xFF) would come out as +-480 that way: kRare also takes these, bytes of 135 (2^8) and up, whose factor
// is past bf16's range and comes in two, and 255, NaN. is_rare: whether 16 codes and their byte need it.
constexpr uint32_t kNoRow = 0u - 120u;
__device__ __forceinline__ bool is_large(uint32_t byte) { return byte - 135u < 121u; }
// bit 7 of each byte: the code there is NaN
__device__ __forceinline__ uint32_t nan_codes(uint32_t codes) { return ((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ bool is_rare(const uint4& c, uint32_t byte) {
  return is_large(byte) || (nan_codes(c.x) | nan_codes(c.y) | nan_codes(c.z) | nan_codes(c.w)) != 0;
}
template <bool kRare>
__device__ __forceinline__ void to_bf16(const uint4& c, uint32_t byte, uint32_t (&w)[8]) {
  const uint32_t in[4] = {c.x, c.y, c.z, c.w};
  // 2^(byte - 127) 2^120 has the exponent field byte + 120, twice in a word
  uint32_t p1 = (byte + 120u) * 0x00800080u, p2 = 0x3F803F80u;
  if (kRare && is_large(byte)) {
    p1 = byte == 255u ? 0x7FC07FC0u : 254u * 0x00800080u;
    p2 = (byte - 134u + 127u) * 0x00800080u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t high = (((in[i] >> 4) & 0x07070707u) | (in[i] & 0xF8F8F8F8u)) & 0x87878787u;
    const uint32_t low = (in[i] << 4) & 0xF0F0F0F0u;
    w[2 * i] = mul_bf16x2(__byte_perm(low, high, 0x5140), p1);
    w[2 * i + 1] = mul_bf16x2(__byte_perm(low, high, 0x7362), p1);
    if (kRare) {
      const uint32_t nan = byte == kNoRow ? 0u : nan_codes(in[i]) >> 7;        // bits 0, 8, 16 and 24
      w[2 * i] = mul_bf16x2(w[2 * i], p2) | (nan & 1u) * 0x7FC0u | (nan >> 8 & 1u) * 0x7FC00000u;
      w[2 * i + 1] = mul_bf16x2(w[2 * i + 1], p2) | (nan >> 16 & 1u) * 0x7FC0u | (nan >> 24) * 0x7FC00000u;
    }
  }
}

struct Maps {
  CUtensorMap d_y, codes, out;
};

// kTma: out's rows are 16-byte aligned, and results leave by TMA. kDecoded: x comes in bf16. kLong (bf16 results): a sum may
// have more than one accumulator.
template <typename T, bool kTma, bool kDecoded, bool kLong>
__global__ void __launch_bounds__(kThreads<kDecoded>, 1)
    weight_grad_kernel(const __grid_constant__ Maps maps, const Args args) {
  using Smem = Smem<kDecoded>;
  constexpr int kStages = Smem::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_a = reinterpret_cast<uint64_t*>(smem + Smem::bars);   // this CTA's d_y has landed
  uint64_t* full_b = full_a + kStages;           // this CTA's x has been decoded, or has landed in bf16
  uint64_t* full = full_b + kStages;             // leader: both CTAs' operands are there
  uint64_t* empty = full + kStages;              // the stage's MMAs have completed
  uint64_t* raw_full = empty + kStages;          // codes and scales of a stage are there
  uint64_t* raw_empty = raw_full + kRaw;         // and have been read
  uint64_t* tfull = raw_empty + kRaw;
  uint64_t* tempty = tfull + 2;                  // leader: both CTAs have read the accumulator
  uint64_t* drain = tempty + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(full_a + Smem::nbars);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_blk = reinterpret_cast<int*>(smem + Smem::meta);
  int* s_cnt = s_blk + args.E + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const Status st{args.report, args.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_a[i], 1);
      mbar_init(&full_b[i], kDecoded ? 1 : kConvertWarps / kGroups);
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&raw_full[i], 1 + 32);
      mbar_init(&raw_empty[i], kConvertWarps / kGroups);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(s_tmem, 512);
  if (args.cnt) {
    for (int i = threadIdx.x; i <= args.E; i += blockDim.x) s_blk[i] = args.blk_off[i];
    for (int i = threadIdx.x; i < args.E; i += blockDim.x) s_cnt[i] = args.cnt[i];
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();                             // every CTA's barriers exist before anything targets them
  tc_fence_after();
  if (kDecoded) pdl_wait();                      // x has been decoded
  const uint32_t tmem = *s_tmem;
  const int ntasks = args.parts == 1 ? args.tasks + (args.tasks - args.whole) : args.tasks * args.parts;
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  static_assert(sizeof(T) == 2 || !kLong);
  constexpr bool kSeveral = kLong || sizeof(T) == 4;
  constexpr int kMost = sizeof(T) == 4 ? kSegment : kLongSegment;
  auto segments = [](int n) { return kSeveral ? (n + kMost - 1) / kMost : 1; };      // accumulators of a task's n stages

  if (warp == kTmaWarp || (kDecoded && warp == kCodesWarp)) {
    // ------------------------------------------------------------------ d_y by TMA, and x in bf16 by another warp: a copy
    // takes its thread 150 cycles
    if (lane == 0) {
      const bool is_x = kDecoded && warp == kCodesWarp;
      const CUtensorMap* map = is_x ? &maps.codes : &maps.d_y;
      uint64_t* landed = is_x ? full_b : full_a;
      uint8_t* to = smem + (is_x ? Smem::b : Smem::a);
      const uint64_t pol = policy_evict_normal();
      Cursor at(first, stride, ntasks);
      Ring<kStages> ring;
      int steps = 0;                             // stages loaded
      while (at.next(args, s_blk, s_cnt)) {
        const int s = ring.s;
        if (*s_abort || !mbar_wait(&empty[s], ring.phase ^ 1, st, s_abort, kSiteEmpty)) break;
        const int mine = is_x ? at.t.cols / 2 : 128;             // columns
        mbar_arrive_expect_tx(&landed[s], mine * kRowsPerStage * 2);
        const int row = at.t.row0 + at.t.ks * kRowsPerStage;
        const int col = (is_x ? at.t.c0 : at.t.n0) + static_cast<int>(rank) * mine;
        tma_load_2d(to + s * kHalfBytes, map, &landed[s], col, row, pol);
        if (mine == 128) tma_load_2d(to + s * kHalfBytes + kChunkBytes, map, &landed[s], col + 64, row, pol);
        ring.step();
        ++steps;
      }
#pragma unroll 1
      for (int s = 0; s < kStages && s < steps; ++s) {
        const uint32_t last = ((steps - 1 - s) / kStages) & 1;   // its last phase
        mbar_drain(&landed[s], last, st, s_abort, kSiteDrainCopies);
        // the leader's last commit to this CTA's barrier has arrived before the CTA leaves
        if (!*s_abort) mbar_drain(&empty[s], last, st, s_abort, kSiteDrainEmpty);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMAs (leader)
    // the whole warp goes through the loop, and one lane issues: what the instructions take stays in uniform registers
    if (rank == 0) {
      const bool issues = elect_one();
      // 64-column chunks kChunkBytes apart, 8-row groups one atom apart
      const uint64_t da0 = make_smem_desc(smem_u32(smem + Smem::a), kChunkBytes, kAtom, 2);
      const uint64_t db0 = make_smem_desc(smem_u32(smem + Smem::b), kChunkBytes, kAtom, 2);
      const uint16_t both = 3;
      Cursor at(first, stride, ntasks);
      Ring<kStages> ring;
      uint32_t acc = tmem, idesc = kIdesc;
      int it = 0, left = 0, in_acc = 0, rows = 0;     // accumulators so far; of this one: stages left, stages in it; rows left
      bool live = at.next_task(args, s_blk, s_cnt);
      auto wait = [&](uint64_t* bar, uint32_t phase, int where) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(bar, phase, st, s_abort, where));
        tc_fence_after();
        return ok;
      };
      auto start = [&]() {                       // an accumulator
        const int buf = it & 1;
        acc = tmem + buf * kTile;
        if (kDecoded) idesc = at.t.cols == kTile ? kIdesc : kIdescHalf;
        left = at.t.end - at.t.ks;
        if (kSeveral) left = min(left, kMost);
        in_acc = 0;
        rows = at.t.rows - at.t.ks * kRowsPerStage;
        live = !__any_sync(0xffffffffu, *s_abort) && wait(&tempty[buf], ((it >> 1) & 1) ^ 1, kSiteTmemEmpty);
      };
      if (live) start();
      while (live) {
        const int s = ring.s;
        if (!wait(&full[s], ring.phase, kSiteFull)) break;
        const uint64_t da = da0 + ((s * kHalfBytes) >> 4), db = db0 + ((s * kHalfBytes) >> 4);
        if (issues) {
          tc_mma_f16_pair(acc, da, db, idesc, in_acc);
#pragma unroll
          for (int k = 1; k < 4; ++k)            // 16 rows: two atoms
            if (rows > 16 * k) tc_mma_f16_pair(acc, da + k * (2 * kAtom >> 4), db + k * (2 * kAtom >> 4), idesc, 1);
          tc_commit_both(&empty[s], both);
        }
        __syncwarp();
        ring.step();
        in_acc = 1;
        rows -= kRowsPerStage;
        ++at.t.ks;
        if (--left == 0) {
          if (issues) tc_commit_both(&tfull[it & 1], both);
          __syncwarp();
          ++it;
          live = at.t.ks < at.t.end || at.next_task(args, s_blk, s_cnt);
          if (live) start();
        }
      }
      if (issues) {
        tc_commit_pair(map_shared(drain, 0));
        mbar_drain(drain, 0, st, s_abort, kSiteDrainMma);
      }
    }
    __syncwarp();
  } else if (warp == kCodesWarp) {
    // ------------------------------------------------------------------ codes by TMA, scales by loads
    const uint64_t pol = policy_evict_normal();
    Cursor at(first, stride, ntasks);
    Ring<kRaw> ring;
    int steps = 0;                               // stages loaded
    for (; at.next(args, s_blk, s_cnt); ring.step(), ++steps) {
      const int s = ring.s;
      if (!mbar_wait_warp(&raw_empty[s], ring.phase ^ 1, st, s_abort, kSiteRawEmpty)) break;
      const int col = at.t.c0 + static_cast<int>(rank) * 128, row0 = at.t.row0 + at.t.ks * kRowsPerStage;
      if (lane == 0) {
        mbar_arrive_expect_tx(&raw_full[s], kRawBytes);
        tma_load_2d(smem + Smem::raw + s * kRawBytes, &maps.codes, &raw_full[s], col, row0, pol);
      }
      const uint32_t sf = smem_u32(smem + Smem::raw_sf + s * kRawSf) + lane * 4;
      const int word = min(col >> 7, args.sf_words - 1);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        copy_word_async(sf + 128 * i, args.sf + static_cast<int64_t>(min(row0 + lane + 32 * i, args.rows - 1)) * args.sf_words + word);
      arrive_after_copies(&raw_full[s]);
    }
    if (lane == 0)
#pragma unroll 1
      for (int s = 0; s < kRaw && s < steps; ++s)
        mbar_drain(&raw_full[s], ((steps - 1 - s) / kRaw) & 1, st, s_abort, kSiteDrainCopies);
    __syncwarp();
  } else if (warp >= kConvert0) {
    // ------------------------------------------------------------------ x into bf16
    // Three groups of warps take turns at the stages. A warp takes 64 columns (the other 64 in odd rows) of every second
    // group of 8 rows, 4 lanes a row: 8 lanes' 16-byte accesses, two rows, fall into 8 different bank groups, of the codes
    // and of the operand.
    const int cw = warp - kConvert0, group = cw % kGroups, r8 = lane >> 2, q = lane & 3;
    const int chunk = ((cw / kGroups) & 1) ^ (r8 & 1), my_row = cw / (2 * kGroups) * 8 + r8;
    const uint8_t* const raw0 = smem + Smem::raw + my_row * 128 + chunk * 64 + q * 16;
    const uint8_t* const sf0 = smem + Smem::raw_sf + my_row * 4 + chunk * 2 + (q >> 1);
    uint8_t* const b0 = smem + Smem::b + chunk * kChunkBytes + my_row * 128;
    const int lo = ((2 * q) ^ r8) << 4, hi = ((2 * q + 1) ^ r8) << 4;
    Cursor at(first, stride, ntasks);
    Ring<kRaw> raw;
    Ring<kStages> ring;
    int turn = group;
    bool live = at.next(args, s_blk, s_cnt);
    while (live) {
      const int rows = at.t.rows - at.t.ks * kRowsPerStage;      // of the expert from this stage on
      live = at.next(args, s_blk, s_cnt);
      if (turn == 0) {
        if (!mbar_wait_warp(&raw_full[raw.s], raw.phase, st, s_abort, kSiteRawFull)) break;
        uint4 c[kLaneRows];
        uint32_t byte[kLaneRows];
#pragma unroll
        for (int i = 0; i < kLaneRows; ++i) {
          c[i] = *reinterpret_cast<const uint4*>(raw0 + raw.s * kRawBytes + i * kRowStep * 128);
          byte[i] = sf0[raw.s * kRawSf + i * kRowStep * 4];
        }
        bool rare = false;
#pragma unroll
        for (int i = 0; i < kLaneRows; ++i) {
          if (my_row + kRowStep * i >= rows) byte[i] = kNoRow;
          rare = rare || is_rare(c[i], byte[i]);
        }
        if (!mbar_wait_warp(&empty[ring.s], ring.phase ^ 1, st, s_abort, kSiteEmpty)) break;
        auto decode = [&](auto tag) {
#pragma unroll
          for (int i = 0; i < kLaneRows; ++i) {
            uint32_t w[8];
            to_bf16<decltype(tag)::value>(c[i], byte[i], w);
            uint8_t* p = b0 + ring.s * kHalfBytes + i * kRowStep * 128;
            *reinterpret_cast<uint4*>(p + lo) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(p + hi) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        };
        if (__any_sync(0xffffffffu, rare)) decode(std::true_type{});
        else decode(std::false_type{});
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full_b[ring.s]);
          mbar_arrive(&raw_empty[raw.s]);
        }
      }
      turn = turn == 0 ? kGroups - 1 : turn - 1;
      raw.step();
      ring.step();
    }
  } else if (warp == kHandWarp) {
    // ------------------------------------------------------------------ both operands to the leader
    Cursor at(first, stride, ntasks);
    Ring<kStages> ring;
    const uint32_t full0 = map_shared(full, 0);
    bool live = at.next(args, s_blk, s_cnt);
    for (; live; ring.step()) {
      const int s = ring.s, rows = at.t.rows - at.t.ks * kRowsPerStage;      // left from this stage on
      live = at.next(args, s_blk, s_cnt);
      if (!live && args.unreachable) break;
      if (!mbar_wait_warp(&full_a[s], ring.phase, st, s_abort, kSiteFullA) ||
          !mbar_wait_warp(&full_b[s], ring.phase, st, s_abort, kSiteFullB))
        break;
      if (rows < kRowsPerStage && (rows & 15)) {
        // the sum ends inside an MMA: whatever d_y's rows behind it hold becomes zero
        uint8_t* am = smem + Smem::a + s * kHalfBytes;
        const int stop = (rows + 15) & ~15;
        for (int i = rows * 16 + lane; i < stop * 16; i += 32) {
          const int r = i >> 4, p = i & 15;
          *reinterpret_cast<uint4*>(am + (p >> 3) * kChunkBytes + (r >> 3) * kAtom + (r & 7) * 128 + ((p & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) arrive_leader(full0 + s * 8);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3;                   // 32 of the CTA's rows of the tile
    int it = 0, box_turn = 0;
    for (int i = first; i < ntasks; i += stride) {
      const Task t = task_at(i, args, s_blk, s_cnt);
      const int n0 = t.n0 + static_cast<int>(rank) * 128 + quad * 32;
      const int64_t row = static_cast<int64_t>(t.slab) * args.N + n0;
      const int rows = args.N - n0;
      const int nks = t.end - t.ks;              // 0: an expert without rows, or without any for this part
      const int cols = kDecoded ? t.cols : kTile;
      bool ok = true;
      const int segs = max(segments(nks), 1);
      for (int seg = 0; seg < segs && ok; ++seg) {
        const int buf = it & 1;
        ok = nks == 0 || mbar_wait_warp(&tfull[buf], (it >> 1) & 1, st, s_abort, kSiteTmemFull);
        if (!ok) break;
        tc_fence_after();
        it += nks != 0;
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(map_shared(&tempty[buf], 0));
        };
        const uint32_t src0 = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * kTile;
        constexpr int kBox = 128 / sizeof(T);    // columns of a box
        if (kTma && seg > 0 && lane == 0) tma_stored();    // what the boxes are added to
        uint32_t v[kBox];                        // a box's accumulators (kDecoded, which has the registers for it: the
                                                 // next one's are on their way while one is stored)
        auto fetch = [&](int c) {
#pragma unroll
          for (int h = 0; h < kBox; h += 32) tmem_ld_32x32b_x32(src0 + c + h, *reinterpret_cast<uint32_t(*)[32]>(v + h));
        };
        if (kDecoded && nks != 0) fetch(0);
#pragma unroll 1
        for (int c = 0; c < cols; c += kBox) {
          uint32_t w[32];
          if (nks == 0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = 0;
          } else {
            if (!kDecoded) fetch(c);
#pragma unroll
            for (int h = 0; h < kBox; h += 32) tmem_loaded(*reinterpret_cast<uint32_t(*)[32]>(v + h));
            if (kLong && segs > 1) {             // this lane's own sums so far
              float4* sum = args.sums + ((blockIdx.x * kEpiWarps + warp) * (kTile / 4) + c / 4) * 32 + lane;
#pragma unroll
              for (int j = 0; j < kBox; j += 4) {
                float4 f = make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                                       __uint_as_float(v[j + 3]));
                if (seg > 0) {
                  const float4 g = sum[j * 8];
                  f.x += g.x; f.y += g.y; f.z += g.z; f.w += g.w;
                }
                if (seg + 1 < segs) sum[j * 8] = f;
                v[j] = __float_as_uint(f.x); v[j + 1] = __float_as_uint(f.y);
                v[j + 2] = __float_as_uint(f.z); v[j + 3] = __float_as_uint(f.w);
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              w[j] = sizeof(T) == 4 ? v[j] : pack2<T>(v[(2 * j) % kBox], v[(2 * j + 1) % kBox]);
            if (c + kBox == cols) release();
            else if (kDecoded) fetch(c + kBox);
          }
          const int col = t.c0 + c;
          if (rows <= 0 || col >= args.C || (kLong && seg + 1 < segs)) continue;
          uint8_t* box = smem + Smem::out + (warp * Smem::kBoxes + box_turn % Smem::kBoxes) * kBoxBytes;
          ++box_turn;
          if (kTma && lane == 0) tma_store_read<Smem::kBoxes - 1>();       // its last results have left it
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
          if constexpr (kTma) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (sizeof(T) == 4 && seg > 0) tma_store_box<true>(&maps.out, box, col, n0, t.slab);
              else tma_store_box<false>(&maps.out, box, col, n0, t.slab);
            }
          } else {
            // row by row, consecutive lanes consecutive words (44 experts of 3188x2181, unrolled by 4 / whole, us: fp32 618 /
            // 510, bf16 554 / 476)
            __syncwarp();
            const int left = args.C - col - lane * (4 / static_cast<int>(sizeof(T)));      // columns from this lane's on
            char* q = args.out + row * args.out_pitch + col * static_cast<int64_t>(sizeof(T)) + lane * 4;
#pragma unroll
            for (int r = 0; r < 32; ++r, q += args.out_pitch) {
              const uint32_t v = *reinterpret_cast<const uint32_t*>(box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
              if (r >= rows || left <= 0) continue;
              if constexpr (sizeof(T) == 4) {
                float* p = reinterpret_cast<float*>(q);
                *p = seg > 0 ? *p + __uint_as_float(v) : __uint_as_float(v);
              } else if (left >= 2 && (reinterpret_cast<uintptr_t>(q) & 3) == 0) {
                *reinterpret_cast<uint32_t*>(q) = v;
              } else {
                reinterpret_cast<uint16_t*>(q)[0] = static_cast<uint16_t>(v);
                if (left >= 2) reinterpret_cast<uint16_t*>(q)[1] = static_cast<uint16_t>(v >> 16);
              }
            }
            __syncwarp();
          }
        }
      }
      if (!ok) break;
    }
    if (kTma && lane == 0) tma_stored();
    __syncwarp();
  }
  // nothing targets a CTA that has left
  __syncthreads();
  cluster_barrier();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

constexpr int kCopyThreads = 256;
// The rows of x that the sums take in bf16, a warp a row: a pool row's token's (by_token), or its own; zeros where it holds
// no pair (its 16 rows may be an MMA's). Without a routing every row is its own.
__global__ void __launch_bounds__(kCopyThreads)
    decode_rows_kernel(const uint4* __restrict__ codes, int pieces, const uint8_t* __restrict__ sf, int blocks,
                       const int32_t* __restrict__ src, const int32_t* __restrict__ blk_off, int E, int block_m, int K,
                       int by_token, int64_t rows, uint4* __restrict__ out) {
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5);
  if (r >= rows || (src && r >= static_cast<int64_t>(__ldg(blk_off + E)) * block_m)) return;
  const int pair = src ? __ldg(src + r) : 0;
  const int64_t t = by_token ? pair / K : r;
  uint4* o = out + r * pieces * 2;
  constexpr int kFlight = 4;                     // pieces a lane has on their way
  for (int i0 = lane; i0 - lane < pieces; i0 += 32 * kFlight) {
    uint4 c[kFlight];
    uint32_t byte[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int i = i0 + 32 * u;
      const bool in = pair >= 0 && i < pieces;
      c[u] = in ? __ldg(codes + t * pieces + i) : make_uint4(0, 0, 0, 0);
      byte[u] = in ? __ldg(sf + t * blocks + (i >> 1)) : kNoRow;
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      const int i = i0 + 32 * u;
      uint32_t w[8];
      if (__any_sync(0xffffffffu, is_rare(c[u], byte[u]))) to_bf16<true>(c[u], byte[u], w);
      else to_bf16<false>(c[u], byte[u], w);
      if (i < pieces) st_global_v8(reinterpret_cast<float*>(o + 2 * i), w);
    }
  }
}

// Rows of d_y on no 16-byte boundary into rows of whole 16-byte pieces, and rows of scales on no 4-byte boundary into rows
// of whole words: `pieces` a row and a thread each, of T.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads)
    align_rows_kernel(const char* __restrict__ x, int64_t pitch, int64_t rows, int64_t bytes, int64_t pieces,
                      T* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  const int64_t r = i / pieces;
  const int64_t c = (i - r * pieces) * static_cast<int64_t>(sizeof(T)), left = bytes - c;
  if (r >= rows) return;
  const uint4 v = load16_any(x + r * pitch + c, left < static_cast<int64_t>(sizeof(T)) ? static_cast<int>(left) : sizeof(T));
  memcpy(out + i, &v, sizeof(T));                // past the row: columns that no tile stores
}
template <typename T>
cudaError_t align_rows(const void* x, int64_t pitch, int64_t rows, int64_t bytes, void* out, cudaStream_t s) {
  const int64_t pieces = (bytes + static_cast<int64_t>(sizeof(T)) - 1) / static_cast<int64_t>(sizeof(T));
  const int64_t all = rows * pieces;
  align_rows_kernel<T><<<static_cast<unsigned>((all + kCopyThreads - 1) / kCopyThreads), kCopyThreads, 0, s>>>(
      static_cast<const char*>(x), pitch, rows, bytes, pieces, static_cast<T*>(out));
  return cudaGetLastError();
}

// out [rows, C] = the sum over parts, in order, of sums [parts][rows][pitch]; a thread 4 columns.
template <typename T>
__global__ void __launch_bounds__(kCopyThreads)
    add_parts_kernel(const float* __restrict__ sums, int parts, int64_t rows, int C, int pitch, T* __restrict__ out) {
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  const int quads = pitch / 4;
  const int64_t r = i / quads;
  const int c = static_cast<int>(i - r * quads) * 4;
  if (r >= rows) return;
  const float4* p = reinterpret_cast<const float4*>(sums) + i;
  float4 v = __ldg(p);
  for (int k = 1; k < parts; ++k) {
    const float4 w = __ldg(p + k * rows * quads);
    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
  T* o = out + r * C + c;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c + j < C) o[j] = from_float<T>(f[j]);
}
template <typename T>
cudaError_t add_parts(const float* sums, int parts, int64_t rows, int C, int pitch, void* out, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows * (pitch / 4) + kCopyThreads - 1) / kCopyThreads));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_parts_kernel<T>, sums, parts, rows, C, pitch, static_cast<T*>(out));
}

// a.out and a.out_pitch: where the sums go, of T.
template <typename T, bool kDecoded, bool kLong = false>
cudaError_t launch(Args& a, Maps& maps, cudaStream_t s) {
  const bool tma = (reinterpret_cast<uintptr_t>(a.out) | static_cast<uintptr_t>(a.out_pitch)) % 16 == 0;
  if (tma) {
    const uint64_t dims[3] = {static_cast<uint64_t>(a.C), static_cast<uint64_t>(a.N),
                              static_cast<uint64_t>(a.E) * static_cast<uint64_t>(a.parts)};
    const uint64_t strides[2] = {static_cast<uint64_t>(a.out_pitch), static_cast<uint64_t>(a.out_pitch) * a.N};
    const uint32_t box[3] = {128 / sizeof(T), 32, 1};
    if (encode_tmap(&maps.out, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.out,
                    dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  auto kernel = tma ? weight_grad_kernel<T, true, kDecoded, kLong> : weight_grad_kernel<T, false, kDecoded, kLong>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (cudaError_t e = configure_kernel(fn, 0, Smem<kDecoded>::total(kMaxE))) return e;
  int most = 0;
  if (cudaError_t e = max_pair_clusters(fn, kThreads<kDecoded>, Smem<kDecoded>::total(kMaxE), &most)) return e;
  if (most < 1) return cudaErrorInvalidConfiguration;
  if (kLong && most > kSplitPairs) most = kSplitPairs;           // what the scratch is for
  // The tasks past the last whole round are taken in halves where these fit a round (8192x4096x4096, 256 tasks on 76 pairs,
  // 174 us for 177 with all whole; 2048x2560x2560 34 for 36). In parts, whose fp32 sums a kernel adds up, they took 2 us
  // less at 8192 rows and 7 more at 4096.
  const int rest = a.tasks % most, halves = kDecoded && a.parts == 1 && 2 * rest <= most ? rest : 0;
  a.whole = a.tasks - halves;
  const int pairs = a.tasks * a.parts + halves;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (pairs < most ? pairs : most)));
  cfg.blockDim = dim3(kThreads<kDecoded>);
  cfg.dynamicSmemBytes = Smem<kDecoded>::total(a.cnt ? a.E : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2; attr[0].val.clusterDim.y = 1; attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;         // the kernel before is one of this call
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kDecoded ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

// Parts of a task's contraction of `terms` rows: as many as pairs of SMs have room for, of 8 stages at least. (N = 256, one
// part / parts, cold caches, us: 8192 rows, C = 4096 69 / 37, C = 256 69 / 22; 65536 rows, C = 2048 451 / 87; 2048 rows, C =
// 4096 27 / 23; 1024 rows 20 / 21.) Past kLongTerms rows two at least: both types' results are then the same
// fp32 sums.
int parts_of(int64_t tasks, int64_t terms) {
  const int64_t stages = (terms + kRowsPerStage - 1) / kRowsPerStage;
  const int64_t n = kSplitPairs / tasks < stages / 8 ? kSplitPairs / tasks : stages / 8;
  const int64_t least = terms > kLongTerms ? 2 : 1;
  return static_cast<int>(n < least ? least : n > kMostParts ? kMostParts : n);
}
int sums_pitch(int C) { return (C + 3) / 4 * 4; }

// Whether x is decoded into bf16 rows before the product, and not by its converters: where more than 4 tiles of N would
// decode the same codes (8192 rows, C = 4096, first / by converters, us: N 256 61 / 42, 512 63 / 50, 1024 70 / 70, 1280
// 105 / 120, 1792 105 / 124, 4096 184 / 249), and where x's rows are tokens, which some kernel has to bring to their pool
// rows anyhow (copied as codes and left to the converters: 8 experts of 1024 rows, N 256 45 us for 48, 512 63 for 59; 64 of
// 384, C = 2048, N 256 123 for 72, 1408 215 for 142).
constexpr int kDecodeTiles = 4;
bool decodes_first(int N, bool by_token) { return by_token || N > kDecodeTiles * kTile; }

// What a call keeps in its scratch, in this order: x in bf16 (rows of 64 bytes' multiples, stored 32 bytes at a time), a
// copy of d_y, one of the scales, and the sums of parts or of a pair's accumulators. Bytes, 0: none. longest: rows of a sum,
// at most (one expert may take them all).
struct Copies {
  size_t x, d_y, sf, sums;
};
Copies copies_of(const void* d_y, int64_t d_stride, int64_t rows, int N, const void* sf, int C, bool by_token, int E,
                 int64_t terms, int64_t longest) {
  const int blocks = blocks8(C, MM_MOE_VARIANT_MX);
  Copies c{0, 0, 0, 0};
  if (reinterpret_cast<uintptr_t>(d_y) % 16 || d_stride % 8) c.d_y = static_cast<size_t>(rows) * ((N + 7) / 8) * 16;
  if (decodes_first(N, by_token)) c.x = static_cast<size_t>(rows) * blocks * kMxBlock * 2;
  else if (reinterpret_cast<uintptr_t>(sf) % 4 || blocks % 4)
    c.sf = (static_cast<size_t>(rows) * ((blocks + 3) / 4) * 4 + 15) / 16 * 16;
  const int64_t tasks = weight_grad_tasks(E, N, C);
  const int parts = parts_of(tasks, terms);
  if (parts > 1) c.sums = static_cast<size_t>(parts) * E * N * sums_pitch(C) * sizeof(float);
  else if (longest > kLongSegment * kRowsPerStage) c.sums = (2 * tasks < kSplitPairs ? 2 * tasks : kSplitPairs) * kPairSums;
  return c;
}

}  // namespace

int64_t weight_grad_tasks(int E, int N, int C) {
  return static_cast<int64_t>(E) * ((N + kTile - 1) / kTile) * ((C + kTile - 1) / kTile);
}

size_t weight_grad_scratch_bytes(const void* d_y, int64_t d_stride, int64_t rows, int N, const void* sf, int C,
                                 bool by_token, int E, int64_t terms, int64_t longest) {
  const Copies c = copies_of(d_y, d_stride, rows, N, sf, C, by_token, E, terms, longest);
  return c.x + c.d_y + c.sf + c.sums;
}

cudaError_t launch_weight_grad(const WeightGradLaunch& p, cudaStream_t s) {
  Args a{};
  if (cudaError_t e = mx_report(&a.report)) return e;
  a.N = p.N; a.C = p.C; a.E = p.E; a.block_m = p.block_m;
  a.NT = (p.N + kTile - 1) / kTile;
  a.CT = (p.C + kTile - 1) / kTile;
  a.rows = static_cast<int>(p.rows);
  a.cnt = p.cnt; a.blk_off = p.blk_off;
  a.tasks = static_cast<int>(weight_grad_tasks(p.E, p.N, p.C));
  a.parts = parts_of(a.tasks, p.terms);
  a.out = static_cast<char*>(p.out);
  a.out_pitch = static_cast<int64_t>(p.C) * dtype_size(p.dtype);
  a.unreachable = p.unreachable;
  a.timeout_ns = p.timeout_ns;
  const int blocks = blocks8(p.C, MM_MOE_VARIANT_MX);
  const bool decoded = decodes_first(p.N, p.by_token);
  const Copies copies = copies_of(p.d_y, p.d_stride, p.rows, p.N, p.sf, p.C, p.by_token, p.E, p.terms, p.longest);
  const void *d_y = p.d_y, *codes = p.codes, *sf = p.sf;
  uint64_t pitch = static_cast<uint64_t>(p.d_stride) * 2;
  char* to = static_cast<char*>(p.scratch);
  if (decoded) {
    const unsigned per = kCopyThreads / 32, grid = static_cast<unsigned>((p.rows + per - 1) / per);
    decode_rows_kernel<<<grid, kCopyThreads, 0, s>>>(reinterpret_cast<const uint4*>(p.codes), blocks * kMxBlock / 16, p.sf,
                                                     blocks, p.src, p.blk_off, p.E, p.block_m, p.K, p.by_token, p.rows,
                                                     reinterpret_cast<uint4*>(to));
    if (cudaError_t e = cudaGetLastError()) return e;
    codes = to;
    to += copies.x;
  }
  if (copies.d_y) {
    if (cudaError_t e = align_rows<uint4>(p.d_y, p.d_stride * 2, p.rows, static_cast<int64_t>(p.N) * 2, to, s)) return e;
    d_y = to;
    pitch = static_cast<uint64_t>((p.N + 7) / 8) * 16;
    to += copies.d_y;
  }
  if (copies.sf) {
    if (cudaError_t e = align_rows<uint32_t>(p.sf, blocks, p.rows, blocks, to, s)) return e;
    sf = to;
  }
  a.sf = static_cast<const uint32_t*>(sf);
  a.sf_words = (blocks + 3) / 4;
  Maps maps{};
  if (encode_tmap_2d(&maps.d_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d_y, static_cast<uint64_t>(p.N),
                     static_cast<uint64_t>(p.rows), pitch, 64, kRowsPerStage, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const uint64_t cols = static_cast<uint64_t>(blocks) * kMxBlock;
  if ((decoded ? encode_tmap_2d(&maps.codes, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, codes, cols, static_cast<uint64_t>(p.rows),
                                cols * 2, 64, kRowsPerStage, CU_TENSOR_MAP_SWIZZLE_128B)
               : encode_tmap_2d(&maps.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, cols, static_cast<uint64_t>(p.rows), cols,
                                128, kRowsPerStage, CU_TENSOR_MAP_SWIZZLE_NONE)) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  auto go = [&](auto tag) {
    using T = decltype(tag);
    return decoded ? launch<T, true>(a, maps, s) : launch<T, false>(a, maps, s);
  };
  float* sums = reinterpret_cast<float*>(static_cast<char*>(p.scratch) + copies.x + copies.d_y + copies.sf);
  if (a.parts == 1) {
    if (p.dtype == MM_MOE_DTYPE_F32) return go(float{});
    if (!copies.sums) return go(__nv_bfloat16{});
    a.sums = reinterpret_cast<float4*>(sums);
    return decoded ? launch<__nv_bfloat16, true, true>(a, maps, s) : launch<__nv_bfloat16, false, true>(a, maps, s);
  }
  const int pitch_c = sums_pitch(p.C);
  a.out = reinterpret_cast<char*>(sums);
  a.out_pitch = static_cast<int64_t>(pitch_c) * sizeof(float);
  if (cudaError_t e = go(float{})) return e;
  const int64_t rows = static_cast<int64_t>(p.E) * p.N;
  return p.dtype == MM_MOE_DTYPE_F32 ? add_parts<float>(sums, a.parts, rows, p.C, pitch_c, p.out, s)
                                     : add_parts<__nv_bfloat16>(sums, a.parts, rows, p.C, pitch_c, p.out, s);
}

}  // namespace mm

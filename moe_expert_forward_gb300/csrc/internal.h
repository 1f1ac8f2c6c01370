// Internal declarations shared by the host API and the kernel translation units.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mm_moe.h"

namespace mm {

constexpr int kBT = 128;        // tokens per pool block of the token-M kernels (one scale chunk)
constexpr int kBK = 128;        // contraction elements per pipeline stage
constexpr int kSFChunk = 512;   // bytes of one 128-row x 128-K scale chunk (MX)
constexpr int kMaxE = 1024;
constexpr int kMaxK = 16;
constexpr int kSchedCounters = 4;        // tile-group counters after the arrival counters, one per GEMM mode
constexpr int kCombineCounters = 4;      // early combine: tokens taken, deferred, classified, deferred taken

// Byte offsets of every buffer inside the caller's workspace.
struct Layout {
  int T, H, I, E, K, variant, BT;
  int CPB;                   // 128-row scale chunks per pool block: ceil(BT / 128)
  int64_t P;                 // pool row capacity (multiple of BT)
  int64_t nblk_cap;          // P / BT
  int KB1, KB2;              // H/128, I/128
  int part_elem;             // bytes of one partial: 4 (fp32) or 2 (bf16)
  int act_gran;              // F8: intermediate scale block along I (128 or 64); MX: 32
  int S;                     // shared experts (the last S of E and of K; 0 = none)
  int64_t ring;              // intermediate slots (pool blocks) of a wrapping ring; 0 = one per pool block
  size_t ext_idx, ext_w;     // shared experts: the routing extended by S slots, int32 / fp32 [T, K]
  size_t status, cnt, blk_off, dscr, ctr, slot, src, pool_x, pool_x_sf, pool2, pool2_sf, part, dbg, dbg_bytes, prof, total;
};

// E and K count the shared experts: E = routed + S, K = routed slots + S.
Layout make_layout(int T, int H, int I, int E, int K, int variant, int debug_flags = 0, int partials_bf16 = 0,
                   int BT = kBT, int act_gran = 128, int S = 0, int ring = 0);
// The F8 intermediate's scale width by the shape rule of DeepGEMM PR #440 ("Ring
// sizing, recycling, and why that granularity"): 128 when H % 512 == 0 and
// 2I % 512 == 0, else 64.
inline int f8_gran_rule(int H, int I) { return (H % 512 == 0 && (2 * I) % 512 == 0) ? 128 : 64; }

// Byte offset, in a pool scale region laid out [block][kb][CPB chunks][512], of
// the 4-byte word of row r of block b (r < BT) and 128-wide contraction block
// kb: chunk r / 128 of the block, then the tcgen05.cp 32x128b order inside the
// chunk (16-byte line r % 32, word (r % 128) / 32, byte = 32-wide sub-block).
__host__ __device__ __forceinline__ size_t pool_sf_word(int64_t b, int kb, int KB, int CPB, int r) {
  return ((static_cast<size_t>(b) * KB + kb) * CPB + (r >> 7)) * kSFChunk + (r & 31) * 16 + ((r & 127) >> 5) * 4;
}

// Ints of the counter region, zeroed before every forward: [2][nblk_cap]
// per-block arrival counters, kSchedCounters, kCombineCounters, [E] L2
// completions per expert, [T] deferred tokens of the early combine (t + 1),
// [nblk_cap] L2 tiles that have read each block's intermediate (ring reuse).
inline size_t ctr_ints(const Layout& L) {
  return 3 * static_cast<size_t>(L.nblk_cap) + kSchedCounters + kCombineCounters + L.E + L.T;
}

// Device pointers resolved from a workspace.
struct WsPtrs {
  int* status;
  int* cnt;
  int* blk_off;
  int* dscr;
  int* ctr;                  // the counter region (ctr_ints): arrival, tile-group and early-combine counters
  int* slot;
  int* src;
  uint8_t* pool_x;
  uint8_t* pool_x_sf;
  uint8_t* pool2;
  uint8_t* pool2_sf;
  float* part;
  float* dbg;
  unsigned long long* prof;
  int32_t* ext_idx;          // shared experts: extended routing (null without)
  float* ext_w;
};
WsPtrs ws_ptrs(void* ws, const Layout& L);

struct DevInfo {
  int sms;
  int cc_major, cc_minor;
  size_t smem_optin;
};
const DevInfo& dev_info();

// Once per kernel and device (thread-safe): when want_regs > 0, fail with
// cudaErrorInvalidConfiguration unless the kernel was built with exactly that
// many registers a thread (the setmaxnreg splits depend on it); when
// smem_bytes > 0, raise the kernel's dynamic shared-memory limit to it.
cudaError_t configure_kernel(const void* fn, int want_regs, int smem_bytes);
// How many 2-CTA clusters of this kernel (blockDim threads, smem_bytes of dynamic
// shared memory) the current device holds at once; cached per kernel and device.
cudaError_t max_pair_clusters(const void* fn, int threads, int smem_bytes, int* clusters);

// ---- launchers (return cudaError_t of the launch)
cudaError_t launch_dispatch(const int32_t* topk_idx, int T, int K, int E, int block_m, int32_t* cnt,
                            int32_t* blk_off, int32_t* slot, int32_t* src, int32_t* status, int32_t* scratch,
                            int64_t scratch_ints, cudaStream_t s);
constexpr int kDispatchMaxCtas = 256;   // the dispatch scratch holds per-CTA counts [CTAs][E]
// x_bf16: x is bf16 [T, H] and each row is quantised on its way into the pool
cudaError_t launch_gather(const Layout& L, const WsPtrs& W, const uint8_t* x, const void* x_sf, bool x_bf16,
                          cudaStream_t s);
// pdl: programmatic launch after the GEMM (the combine waits for it in-kernel)
cudaError_t launch_combine(const Layout& L, const WsPtrs& W, const int32_t* topk_idx, void* out, bool pdl,
                           cudaStream_t s);
cudaError_t launch_prepare_sf_mx(const uint8_t* w1_sf, const uint8_t* w2_sf, int H, int I, int E,
                                 uint8_t* w1_sfp, uint8_t* w2_sfp, cudaStream_t s);
// topk_idx [T, K] / topk_w -> [T, K + S]: routed slots copied (ids in [E, E+S)
// turned into -2, out of range for the routing kernels), then S slots naming
// experts E .. E+S-1 with weight 1.
cudaError_t launch_extend_routing(const int32_t* topk_idx, const float* topk_w, int T, int K, int E, int S,
                                  int32_t* ext_idx, float* ext_w, cudaStream_t s);
cudaError_t launch_read_intermediate(const Layout& L, const WsPtrs& W, int64_t rows, uint8_t* codes,
                                     void* sf, cudaStream_t s);

struct GemmLaunch {
  const Layout* L;
  const WsPtrs* W;
  const uint8_t* w1;         // e2m1 weights and their prepared scale chunks
  const uint8_t* w1sfp;
  const uint8_t* w2;
  const uint8_t* w2sfp;
  const uint8_t* x;          // activations and scales (in-kernel gather of the fused stream)
  const void* x_sf;
  bool x_bf16;               // x is bf16 [T, H]: the gather quantises (x_sf unused)
  const float* topk_w;
  float* dbg;               // L1 raw accumulators (debug_flags bit 0) or null
  unsigned long long* prof; // per-CTA role timings (debug_flags bit 1) or null
  uint64_t timeout_ns;
  int grid;
  float clamp;              // activation clamp of gate and up (+inf: none)
  int precise;              // SwiGLU with expf and the IEEE division instead of the fast-math form
  bool early_combine;       // fused stream: the epilogue warps combine tokens once their experts are done
  const int32_t* topk_idx;  // early combine: the routing and the bf16 output [T, H]
  void* out;
  bool pdl;                 // programmatic launch after the routing kernel
  bool per_block;           // token-M kernel: deal (weight tile, pool block) pairs as separate groups
  uint8_t* trace;           // token-M kernel: per-task trace records of this launch ([grid][trace_cap] x 64 B) or null
  int trace_cap;            // records per CTA
};
// One per-task trace record (64 bytes; mm_moe.h, Options.trace_buf).
struct TraceRec {
  uint32_t cta, task, type, expert, tile, block, valid, mode;
  uint64_t t_issue, t_mma_done, t_epi_done, reserved;
};
static_assert(sizeof(TraceRec) == 64, "trace record");
// mode 1: L1 tiles, mode 2: L2 tiles, mode 3: gather + lag-ordered L1/L2 stream
cudaError_t launch_gemm_mx(const GemmLaunch& g, int mode, int lag, int l1_extra, cudaStream_t s);
int mx_lag_auto(int E);
// The same modes with the weights as the MMA's M operand and each pool block's
// tokens as N (gemm_mx_sw.cu); g.L->BT must be a supported block size.
cudaError_t launch_gemm_mx_sw(const GemmLaunch& g, int mode, int lag, int l1_extra, cudaStream_t s);
bool mx_sw_block_supported(int bt);
// The swapped form on 2-CTA clusters (gemm_mx_pair.cu): M = 256 weight rows per
// tcgen05 cta_group::2 MMA, half of each block's tokens in each CTA.
cudaError_t launch_gemm_mx_pair(const GemmLaunch& g, int mode, int lag, int l1_extra, cudaStream_t s);
bool mx_pair_block_supported(int bt);

struct GemmLaunchF8 {
  const Layout* L;
  const WsPtrs* W;
  const uint8_t* w;          // e4m3 weights (w1 or w2)
  const float* wsf;          // their fp32 128x128 block scales
  const float* topk_w;
  uint64_t timeout_ns;
  int grid;
  unsigned long long* prof;  // per-CTA role cycles (debug_flags bit 1) or null
  float clamp;               // activation clamp of gate and up (+inf: none)
  int precise;               // SwiGLU with expf and the IEEE division instead of the fast-math form
  bool exact_div;            // L1 requant: divide for every code (debug_flags bit 4), not only near a boundary
  bool unreachable;          // L1: the last stage of each CTA's last task is never loaded (debug_flags bit 2)
};
cudaError_t launch_gemm_f8_l1(const GemmLaunchF8& g, cudaStream_t s);
cudaError_t launch_gemm_f8_l2(const GemmLaunchF8& g, cudaStream_t s);

// The router (route.cu); weights and gradients are fp32, logits any dtype.
struct RouteArgs {
  const void* logits;
  int dtype;
  int64_t stride;            // elements between rows
  int T, E, K;
  const float* bias;         // [E] or null (sigmoid only)
  int score, renorm;
  float scale;
  int32_t* topk_idx;
  float* topk_w;
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t s);
cudaError_t launch_route_backward(const RouteArgs& a, const int32_t* topk_idx, const float* d_w, void* d_logits,
                                  int64_t d_stride, cudaStream_t s);

// The routing in one launch up to so many pairs (sort.cu), by launch_dispatch above;
// status is cleared first.  `scratch` is launch_dispatch's, unused in one launch.
constexpr int64_t kSortOneLaunchPairs = int64_t(3) << 16;
bool sort_in_one_launch(int64_t pairs);
cudaError_t launch_sort(const int32_t* topk_idx, int T, int K, int E, int block_m, int32_t* cnt, int32_t* blk_off,
                        int32_t* slot, int32_t* src, int32_t* status, int32_t* scratch, int64_t scratch_ints,
                        cudaStream_t s);

// Rows sorted by expert and back (rows.cu), over the routing of launch_dispatch.
struct RowsArgs {
  int dtype;
  int64_t T;
  int H, K, E, block_m;
  int64_t num_rows;          // pool rows
  const int32_t* slot;
  const int32_t* src;
  const int32_t* blk_off;
};
cudaError_t launch_permute(const RowsArgs& a, const void* x, int64_t x_stride, void* rows, cudaStream_t s);
// w: weights per pair, or null (ones)
cudaError_t launch_unpermute(const RowsArgs& a, const void* rows, const float* w, void* out, int64_t out_stride,
                             cudaStream_t s);
// d_w: null leaves the weights' gradient out
cudaError_t launch_unpermute_backward(const RowsArgs& a, const void* d_out, int64_t d_stride, const void* rows,
                                      const float* w, void* d_rows, float* d_w, cudaStream_t s);

// Rows in 8 bits (quant8.cu): variant MM_MOE_VARIANT_MX or _F8.
cudaError_t launch_quantize8(const void* x, int dtype, int64_t stride, int64_t R, int C, int variant, void* codes,
                             void* sf, cudaStream_t s);
cudaError_t launch_dequantize8(const void* codes, const void* sf, int64_t R, int C, int variant, int dtype, void* out,
                               int64_t stride, cudaStream_t s);

// The norm (norm.cu).
constexpr int kNormSms = 152;              // its gradient's CTAs do not depend on the device: neither does the scratch
struct NormLaunch {
  const void* x;
  int dtype;
  int64_t x_stride;
  const void* residual;      // or null, then h is null too
  int64_t residual_stride;
  const void* weight;
  int weight_dtype;          // dtype or fp32
  int64_t T;
  int H;
  float eps;
  void* h;
  void* y;                   // or null
  int variant;
  void* codes;               // or null
  void* sf;
  float* rstd;
};
cudaError_t launch_rms_norm(const NormLaunch& n, cudaStream_t s);
struct NormBackLaunch {
  const void* d_y;
  int dtype;
  int64_t d_y_stride;
  const void* h;
  int64_t h_stride;
  const void* weight;
  int weight_dtype;
  const float* rstd;
  const void* d_h;           // or null
  int64_t d_h_stride;
  int64_t T;
  int H;
  void* d_x;
  float* d_weight;
  void* scratch;             // norm_scratch_bytes
};
size_t norm_scratch_bytes(int64_t T, int H);
cudaError_t launch_rms_norm_backward(const NormBackLaunch& n, cudaStream_t s);

// The activation between the experts' products (swiglu.cu).
struct SwigluRows {
  int64_t rows;
  int I;
  const int32_t* slot;       // the routing of launch_sort; all null without one
  const int32_t* src;
  const int32_t* blk_off;
  int E, block_m;
  int64_t pairs;
};
cudaError_t launch_swiglu(const SwigluRows& r, int dtype, const void* h, int64_t stride, const float* w, void* a,
                          void* codes, void* sf, void* kept, void* kept_sf, cudaStream_t s);
cudaError_t launch_swiglu_backward(const SwigluRows& r, int dtype, const void* d_a, int64_t stride, const void* kept,
                                   const void* kept_sf, const float* w, void* d_h, float* d_w, cudaStream_t s);

// Weight gradients from rows in 8 bits (weight_grad.cu).
struct WeightGradLaunch {
  const void* d_y;           // bf16
  int64_t d_stride;
  int64_t rows;
  int N;
  const uint8_t* codes;
  const uint8_t* sf;
  int C;
  const int32_t* cnt;        // null: dense
  const int32_t* blk_off;
  const int32_t* src;
  bool by_token;             // x's rows are tokens
  int K, E, block_m;
  int64_t terms;             // rows of a sum, of an expert on average
  int64_t longest;           // rows of a sum, at most
  int dtype;                 // of out: fp32 or bf16
  void* out;
  void* scratch;             // weight_grad_scratch_bytes
  uint64_t timeout_ns;
  bool unreachable;
};
size_t weight_grad_scratch_bytes(const void* d_y, int64_t d_stride, int64_t rows, int N, const void* sf, int C,
                                 bool by_token, int E, int64_t terms, int64_t longest);
int64_t weight_grad_tasks(int E, int N, int C);
cudaError_t launch_weight_grad(const WeightGradLaunch& p, cudaStream_t s);

// TMA descriptor creation through the driver entry point.
CUresult encode_tmap(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides_bytes, const uint32_t* box, CUtensorMapSwizzle swz);
CUresult encode_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
                        uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
                        CUtensorMapSwizzle swz);

}  // namespace mm

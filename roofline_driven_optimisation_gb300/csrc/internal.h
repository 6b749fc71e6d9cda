// Interface between the C-ABI/dispatcher (gemm_api.cu) and the kernel
// translation units.  Not installed; not part of the public ABI.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace g3 {

// Raises `kernel`'s dynamic shared-memory limit to `bytes` once per device
// (the attribute belongs to the device's context); `done` holds one bit per
// device.  Two threads racing on the first call both set it, which is harmless.
template <class Kernel>
cudaError_t set_smem_once(std::atomic<uint64_t>& done, Kernel kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? (1ull << dev) : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_release);
  return e;
}

enum class Elem : int { F32 = 0, BF16 = 1, FP8 = 2 };

// FP8 formats (values of gemm_fp8_format in the header).
enum Fp8Fmt : int { kE4M3 = 0, kE5M2 = 1 };

// Activations of the fused epilogue (values of gemm_activation in the header).
enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3 };

// One GEMM call after validation: C = alpha*A*B + beta*C, row-major.
struct GemmArgs {
  int M, N, K;
  float alpha, beta;
  const void* A;
  long long lda;
  const void* B;
  long long ldb;
  void* C;
  long long ldc;
  Elem in, out;
  int* status;          // device status word (one int, see report_status)
  uint64_t timeout_ns;  // bound on any single wait inside a kernel
  const float* bias;    // N fp32 values added to every row of C, or null
  int act;              // Act applied last
  const void* B2;       // SwiGLU: the up-projection (K x N, leading dimension ldb), else null
  int swiglu;           // 1: C = silu(A*B) * (A*B2) (alpha 1, beta 0, no bias)
  int fmt_a, fmt_b;     // in == FP8: the formats of A and B (Fp8Fmt)
  int stall;            // test hook: one role of the first CTA (or cluster) waits on a
                        // barrier nothing arrives at, so its bounded wait runs out and
                        // the kernel's abort path runs (tc2, skinny, FP32 SIMT kernels)
};

// Location codes recorded with a device timeout (bits 8 and up of the
// status word; the low 8 bits hold the gemm_status code).
enum WaitSite : int {
  kSiteSelftest = 1,
  kSiteTcProducer = 10,
  kSiteTcMma = 11,
  kSiteTcEpilogue = 12,
  kSiteTcDrain = 13,
  kSiteTc2Producer = 14,
  kSiteTc2Mma = 15,
  kSiteTc2Epilogue = 16,
  kSiteTc2Drain = 17,
  kSiteTc2StreamK = 18,    // a stream-K finisher pair waiting for another pair's partial tile
  kSiteSimtConsumer = 21,
  kSiteSimtDrain = 22,
  kSiteSimtStreamK = 23,   // a stream-K finisher waiting for another CTA's partial tile
  kSiteSkinnyProducer = 30,
  kSiteSkinnyMma = 31,
  kSiteSkinnyEpilogue = 32,
  kSiteSkinnyDrain = 33,
  kSiteW4Producer = 40,
  kSiteW4Mma = 41,
  kSiteW4Epilogue = 42,
  kSiteW4Drain = 43,
  kSiteAttnProducer = 50,
  kSiteAttnMma = 51,
  kSiteAttnSoftmax = 52,
  kSiteAttnDrain = 53,
  kSiteKvAppend = 60,      // a row range, position or page number that does not fit the call
  kSiteKvAttn = 61,        // the same, in attention over the paged cache
  kSiteKvAttnLoad = 62,    // a wait for a tile of the paged cache
  kSiteBlocksProducer = 70,
  kSiteBlocksMma = 71,
  kSiteBlocksScales = 72,
  kSiteBlocksEpilogue = 73,
  kSiteBlocksDrain = 74,
  kSiteWideProducer = 76,
  kSiteWideMma = 77,
  kSiteWideScales = 78,
  kSiteWideEpilogue = 79,
  kSiteWideDrain = 80,
  kSiteWideRows = 81,
  kSiteExperts = 75,       // an expert's slots, or a slot's number, that do not fit the call
};

// Each launcher returns a cudaError_t (as int) from the launch.
int launch_generic(const GemmArgs& a, cudaStream_t s);

// FP32 SIMT kernel: TMA tiles of A (16 k x 128 m, 64-byte swizzle) and
// B (bn n x 16 k), bn = 128 (8 x 8 register tiles, two CTAs per SM) or 256
// (8 x 16 register tiles, one CTA per SM).  plan_f32_simt picks the tile
// width (forced_tn 8 or 16 pins it, 0 lets the wave model choose) and
// whether the tiles of a partial last wave run as a second launch, K split
// over clusters of `split` CTAs (*k_split receives it; 1 otherwise).
struct SimtPlan {
  int tn = 8;     // register-tile width: 8 or 16 (C tiles of 128 x 16*tn)
  int split = 1;  // 1; 4 (narrow: clusters of four share a tile's K range);
                  // 0 (wide: stream-K over the SMs, partial tiles meeting in
                  // a per-device workspace)
};
// Lowers every stream-K flag of the current device's workspace (after a
// device timeout, which may leave flags raised).
void sk_clear_flags();
// The per-device stream-K workspace shared by the FP32 SIMT and CTA-pair
// kernels: stream_k_setup allocates and zeroes it at the first call on a
// device (a device-wide wait); stream_k_slot hands out its four slots in
// turn -- partial tiles (slot_floats floats, num_sms x 65536) and flags
// (slot_flags words, num_sms x 16, zero between calls).
cudaError_t stream_k_setup(int num_sms);
cudaError_t stream_k_slot(int num_sms, float** partials, unsigned** flags, size_t* slot_floats,
                          size_t* slot_flags);
int plan_f32_simt(int M, int N, int K, int num_sms, int forced_tn, SimtPlan* out);
int launch_f32_simt(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB,
                    const SimtPlan& plan, int num_sms, cudaStream_t s, int* k_split);
constexpr int kSimtBM = 128, kSimtBK = 16, kSimtBN8 = 128, kSimtBN16 = 256;

// gemm_f32_noalloc: the FP32 SIMT plan run with the stream-K tail's partial
// tiles and flags in a static device array instead of the workspace, so the
// call allocates nothing.  The array holds the tail of up to
// kStaticScratchCtas CTAs; simt_stream_k_ctas gives the CTAs the tail of
// `plan` needs for this shape (0: the plan has no stream-K tail).
constexpr int kStaticScratchCtas = 152;
int simt_stream_k_ctas(int M, int N, int K, const SimtPlan& plan, int num_sms);
// Bytes of the static array (partial tiles and flags).
size_t simt_static_scratch_bytes();
// Plain GEMMs only (no bias or activation); the caller has checked that
// simt_stream_k_ctas() <= kStaticScratchCtas.
int launch_f32_simt_static(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB,
                           const SimtPlan& plan, int num_sms, cudaStream_t s, int* k_split);

// BF16 tcgen05 kernel: TMA tiles of A (64 k x 128 m) and B (64 n x 64 k),
// 128-byte swizzle; C tiles of 128 x bn with bn from choose_tc_bn().
int choose_tc_bn(int M, int N, int num_sms);
// Single CTA (pair = 1) or CTA pair (pair = 2) and the tile width.
void choose_tc_config(int M, int N, int num_sms, int* pair, int* bn);
int launch_bf16_tc(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, int bn,
                   int num_sms, cudaStream_t s);
constexpr int kTcBM = 128, kTcBK = 64;

// The same GEMM on CTA pairs (clusters of two, cta_group::2): C tiles of
// 256 x bn, bn in {128, 256}; each CTA loads 128 rows of A and bn/2 columns
// of B with the same tensor maps as the single-CTA kernel.
// *schedule receives 2 (whole tiles), 4 (the tiles of a partial last wave
// run as two half-width tiles each) or 6 (they run stream-K over the pairs).
bool split_tiles_enabled();
// gemm_force_split_tiles: 0 forbid, 1 automatic, 2 pin the CTA-pair
// kernel's stream-K tail, 3 pin its half-width tail (where each exists).
int split_tiles_mode();
int launch_bf16_tc_pair(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, int bn,
                        int num_sms, cudaStream_t s, int* schedule);
// SwiGLU on CTA pairs (a.swiglu): C tiles of 256 x 128; each CTA's B operand
// is 64 columns of Bgate (mapB) and the same 64 columns of Bup (mapB2).
// FP8 inputs (in == FP8) on CTA pairs, 256 x 256 C tiles: TMA tiles of A
// (128 k x 128 m bytes) and B (128 n x 128 k bytes), 128-byte swizzle.
// *schedule as for launch_bf16_tc_pair (2 or 6: no half-width tiles).
int launch_fp8_tc_pair(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB,
                       int num_sms, cudaStream_t s, int* schedule);
constexpr int kF8BK = 128;

int launch_bf16_swiglu_pair(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB,
                            const CUtensorMap* mapB2, int num_sms, cudaStream_t s);

// Skinny (M <= 16) split-K kernel: TMA tiles of B (64 n x 64 k) and A
// (64 k x 16 rows), 128-byte swizzle.  mapB2 (the up-projection) is used
// when a.swiglu is set, and may be null otherwise.
// *k_split receives the number of CTAs K was split over.
int launch_skinny(const GemmArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB,
                  const CUtensorMap* mapB2, int num_sms, cudaStream_t s, int* k_split);
constexpr int kSkMaxM = 16, kSkBN = 128, kSkBK = 64;

// INT4 dequantisation W = s[k / G][n] * (q - z) (bf16 or fp32 W);
// *vector_path = 1 when the 32-codes-per-thread kernel ran.
int launch_int4_dequant(const uint8_t* q, int K, int N, int ldq, const void* scales, int lds,
                        int group, int zero, void* w, int ldw, bool out_bf16, int num_sms,
                        cudaStream_t st, int* vector_path);

// INT4 weight-only decode GEMM (bf16 X, M <= 16; codes in the tiled layout
// of 4 KB tiles, 128 columns x 64 rows of K): TMA tiles of X (64 k x 16 rows,
// 128-byte swizzle), bulk copies of the code tiles.  fast = the tcgen05
// kernel (w4_fast_ok and the alignment rules), else a one-thread-per-element
// kernel.
constexpr int kW4BN = 128, kW4BK = 64;
bool w4_fast_ok(int M, int K, int group);
size_t w4_packed_bytes(int K, int N);
int launch_w4_decode(const GemmArgs& a, const void* scales, long long lds, int group, int zero,
                     const CUtensorMap* mapX, const uint8_t* qk, bool fast, int num_sms,
                     cudaStream_t s, int* k_split);
// natural INT4 layout (packed along n) -> tiled layout (w4_packed_bytes)
int launch_int4_repack(const uint8_t* q, long long ldq, uint8_t* qk, int K, int N, int num_sms,
                       cudaStream_t s);

// Attention O = softmax(Q K^T * scale) V, [B][H][S][D] bf16 (K/V with Hkv
// heads).  fast = the tcgen05 kernel (D 64 or 128, 16-byte-aligned tensors;
// 3-D maps of Q with boxes 64 d x 128 rows and of K, V with 64 d x 64 keys),
// else a one-block-per-row kernel.
int launch_attention(int B, int Hq, int Hkv, int Sq, int Sk, int D, const void* Q, const void* K,
                     const void* V, void* O, float scale, int causal, const CUtensorMap* mQ,
                     const CUtensorMap* mK, const CUtensorMap* mV, bool fast, int* status,
                     uint64_t timeout_ns, cudaStream_t s);

// A paged 8-bit key/value cache (gemm_kv_cache) after validation.
struct KvCache {
  uint8_t *k, *v;
  float *ks, *vs;                 // pages x H
  const int* table;
  long long ps, hs, ts, tstride;  // page, head and token strides in bytes; table row stride
  int fmt, pages, P, H, D, seqs, cols;
};

// Appending rotated keys and values (gemm_kv_append).
struct KvAppendArgs {
  KvCache c;
  int tokens, Hq;
  const void *Q, *K, *V;          // bf16 rows, heads side by side
  long long ldq, ldk, ldv, ldqo;  // elements between rows
  void* Qo;
  const float *cos, *sin;         // positions x rot/2
  int positions, rot, interleaved;
  const int *base, *start;
  int max_new;
  int* status;
};
// fast: D 64 or 128, P a power of two 16..128, rot == D, 16-byte-aligned rows.
int launch_kv_append(const KvAppendArgs& a, bool fast, int num_sms, cudaStream_t s);

// Attention over the paged cache (gemm_kv_attention).
struct KvAttnArgs {
  KvCache c;
  int tokens, Hq;
  const void* Q;
  long long ldq;
  void* O;
  long long ldo;
  const int *lengths, *start;
  int max_new;
  float scale;
  void* ws;
  int* status;
  uint64_t timeout_ns;
};
int launch_kv_attention_generic(const KvAttnArgs& a, cudaStream_t s);
// D 64 or 128, P 16, 32, 64 or 128, 16-byte-aligned codes and strides, at most
// kKvMaxSeqs sequences.  mK, mV: 4-D maps (dim, page row, head, page) with boxes of
// D x min(P, 32) codes, swizzle of D bytes.
int launch_kv_attention(const KvAttnArgs& a, const CUtensorMap* mK, const CUtensorMap* mV, int num_sms,
                        cudaStream_t s);
constexpr int kKvMaxSeqs = 8192, kKvSlab = 32;
size_t kv_attention_ws_bytes(int seqs, int heads, int group, int max_new);

// Sampling (gemm_sample_*).
struct SampleArgs {
  int rows, vocab;
  const void* logits;
  long long ld;
  bool bf16;
  const float* temperature;
  const int* top_k;
  const float *top_p, *min_p, *u;
  int* token;
  float* logprob;
};
constexpr int kSampleMaxVocab = 1 << 20;
int launch_sample(const SampleArgs& a, int num_sms, cudaStream_t s);

// Routing of tokens to experts (gemm_route_*).
struct RouteArgs {
  int tokens, experts, top_k;
  const void* logits;
  long long ld;
  bool bf16, softmax, renormalise;
  int groups, top_groups, group_best;
  int group_size, group_lanes;   // experts of a group; lanes that look through one (a power of two)
  bool group_whole;       // a group is group_lanes lanes' experts
  float scale;
  const float* bias;
  int* ids;
  float* weights;
  int *offsets, *order;   // null: the order by expert is not wanted
  int* counts;            // workspace: counts by block and expert
  bool choices;           // a bias or groups: choices are computed, and shared memory has room for a token's in fp64
  bool vec;               // 16-byte-aligned rows
};
constexpr int kRouteMaxExperts = 1024, kRouteMaxTopK = 32, kRouteMaxGroups = 32;
// a power of two: 1 to 32 for up to 1024 experts
constexpr int route_experts_per_lane(int experts) {
  int per = 1;
  while (per * 32 < experts) per *= 2;
  return per;
}
size_t route_ws_bytes(int tokens, int experts);
int launch_route(const RouteArgs& a, int num_sms, cudaStream_t s);

// E4M3 codes with a scale for each block of block_rows (1 or 128) x 128 values.
struct QuantiseArgs {
  int rows, cols;
  const void* x;
  long long ldx;
  bool bf16;
  uint8_t* codes;
  long long ldq;
  float* scales;
  long long lds;
  int block_rows;
  bool vec_x, vec_q;      // rows of 16-byte-aligned vectors of 8 values; of 8-byte-aligned ones
  const int* place = nullptr;   // row r goes to rows place[r * copies + j], j < copies (1 x 128 only)
  int copies = 1;
  const int* order = nullptr;   // what place was made from
  bool units32 = false;         // warps counted in 32 bits
};
int launch_fp8_quantise(const QuantiseArgs& a, cudaStream_t s);
// place[order[p]] = p for p < n
int launch_invert(const int* order, int n, int* place, int* status, cudaStream_t s);

// Block-scaled products of E4M3 codes, for one matrix or for the slots of experts:
// rows [offsets[e], offsets[e+1]) are multiplied with B's e-th matrix.
struct BlocksArgs {
  int experts, rows, N, K;
  const int* offsets;           // null: one matrix, all rows
  const int* order;             // slot number of each row (scatter, gather), or null
  int gather;                   // row p of the product is row order[p] / gather of A; 0: row p
  int scatter;                  // row p of the product is row order[p] of C
  const uint8_t* A;
  long long lda;
  int a_rows;
  const float* sa;              // a_rows x ceil(K/128)
  long long ldsa;
  const uint8_t *B, *B2;        // experts x K x N; B2: the up-projection (SwiGLU), else null
  long long ldb, b_stride;
  const float *sb, *sb2;        // experts x ceil(K/128) x ceil(N/128)
  long long ldsb, sb_stride;
  void* C;
  long long ldc;
  bool out_bf16;
  float alpha, beta;
  // not null (pair kernel): C is fp16 times a power of two for each 128 columns of a row of C
  // (ldys values a row), in whole vectors up to column ldc
  float* ys;
  long long ldys;
  uint8_t* hq;                  // SwiGLU: codes and scales (rows x ceil(N/128)) of silu(A*B) .* (A*B2)
  float* hs;
  long long ldh, ldhs;
  int* status;
  uint64_t timeout_ns;
  int stall;                    // as GemmArgs::stall
  // The kernel before on the stream wrote A and sa alone: B, its scales, offsets and order
  // may be read before it has finished.
  int early;
};
constexpr int kBlocksK = 128, kBlocksN = 128, kBlocksMaxExperts = 1024;
// N and K: a tile of 256 columns and a block behind the last still count in 32 bits
constexpr int kBlocksMaxCols = 0x7fffffff - 255;
// The tcgen05 kernel: row tiles of nt, K split over clusters of `split` CTAs.  Maps: A
// with boxes of 128 k x blocks_box_rows(nt, gather) rows; B and B2 3-D with boxes of 128
// columns x 128 k; 128-byte swizzle.
struct BlocksPlan {
  int nt = 32, split = 1;
};
constexpr int blocks_box_rows(int nt, bool gather) { return gather ? 1 : nt >= 128 ? 64 : 16; }
// The most row tiles that `rows` rows of `experts` experts can make.
constexpr long long blocks_row_tiles(long long rows, int experts, int nt) {
  return experts == 1 ? (rows + nt - 1) / nt : rows / nt + (experts < rows ? experts : rows);
}
int launch_blocks(const BlocksArgs& a, const BlocksPlan& plan, const CUtensorMap* mapA, const CUtensorMap* mapB,
                  const CUtensorMap* mapB2, int num_sms, cudaStream_t s);
// The kernel for many rows, on CTA pairs: items of 256 rows and 256 columns (with B2 128 of
// each); the same maps, A's boxes of blocks_box_rows(kBlocksWide, false) rows.  kBlocksWide in a plan's nt selects it.
constexpr int kBlocksWide = 256;
int launch_blocks_wide(const BlocksArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, const CUtensorMap* mapB2,
                       int num_sms, cudaStream_t s);
int launch_blocks_generic(const BlocksArgs& a, cudaStream_t s);

// O[t] = sum over j of weights[t][j] * Y[t * top_k + j]
struct CombineArgs {
  int tokens, top_k, cols;
  const void* y;                // cols values a row, ldy apart: fp32, or fp16 times ys where that is not null
  const float* ys;              // a scale for each 128 columns, ldys a row
  long long ldys;
  long long ldy;
  const float* weights;
  void* out;
  long long ldo;
  bool vec;
};
int launch_experts_combine(const CombineArgs& a, cudaStream_t s);

int launch_selftest_wait(int* status, uint64_t timeout_ns, cudaStream_t s);

}  // namespace g3

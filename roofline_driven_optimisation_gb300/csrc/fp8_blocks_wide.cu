// Block-scaled products (the formulas are those of fp8_blocks.cu) for calls with many rows,
// on CTA pairs: an item is 256 rows of A and 256 columns of B, or, with gate and up
// weights, 256 rows and 128 columns of each.
//
// Why another kernel.  With many rows the products are compute-bound, and what the
// swapped kernel does a block of 128 k is then too much: a scale of shared memory for each
// column of the accumulator.  Here rows of A are TMEM lanes, so that a drain thread has
// one row and two scales a block.  And a single CTA's 128 x 256 item moves 48 KB a block
// into shared memory and out of it again against 512 tensor cycles: measured 768 cycles
// a block (128 bytes a cycle) without any drain (8192 x 11008 x 4096: 366 us with it, when
// the pairs took 356).  In a pair (cta_group::2, one M = 256 MMA) each CTA holds its 128 rows of A and half
// of B's columns: 32 KB.
//
// What bounds it.  The tensor core's sum of a block of 128 k has to leave TMEM before its
// buffer takes the next block but one, so MMA, its completion, the drain and the buffer's
// return make a chain, and a pair's far barriers are some 300 cycles away.  With one
// 256-wide accumulator a block and two buffers the chain was 950 to 1050 cycles a block;
// so a block is two MMAs of 128 columns (64 of each CTA's half of B), each with its own
// buffers, barriers and four drain warps, and the two chains run beside each other.  The
// drain's 128 x 256 sums a CTA take 256 cycles of fma.rn.f32x2 (64 a warp, two warps a
// scheduler, two cycles each), and 16 sums leave TMEM while the 16 before them are added:
// one after the other cost the chain a quarter (356 us; loads of 32 spill, 350; of 8, 311).
// Measured at 76 pairs x 19 items: 0.38 us a block and 1.7 us an item besides (3.6 where the
// drain warps store the rows of C, as they do in fp32; 8192 x 11008 x 4096 takes 299 us then, and
// with beta, which reads C by rows of a thread each, 383 in bf16 and 506).  Without a drain a block takes 0.36
// us, at the tensor cores' rate alone 0.33.  8192 x 11008 x 4096: 262 us, 2810 TFLOP/s.
//
// Roles (384 threads a CTA, 512 with bf16 rows of C): warp 0 copies (each CTA its rows of A
// and its half of B; all complete on the leader's barrier), warp 1 of the leader issues the
// MMAs, warp 2 copies the scales of its CTA's rows into a ring of eight blocks (cp.async, no
// registers), warp 3 waits for accumulators and scales on behalf of the drain warps, warps
// 4-11 drain: warp w the TMEM lanes 32*(w%4)..+31 of one of the two MMAs, its 128 sums in
// registers for the whole of K.  Warps 12-15 store the rows of C that the drain warps have
// laid into shared memory, so that these go on with the next item (294 to 269 us; the
// experts' down products of 11 blocks an item gain more).
//
// h of gate and up: a thread has 64 columns of its row in both, so the largest magnitude
// of 128 columns is found in registers and one exchange with the thread of the other
// half.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "experts.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

constexpr int BK = kBlocksK, BM = kBlocksWide, BM_CTA = BM / 2;
constexpr int EPI_WARPS = 8, EPI_FIRST = 4, STORE_FIRST = 12;
constexpr int A_BYTES = BM_CTA * BK, B_BYTES = BK * 128;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int TMEM_COLS = 512, COLS = 256, NBUF = 2;
// The ring of scales: a slot holds four blocks of k, four floats for each row and for B's
// one or two column blocks, so that a drain thread waits and reads once in four blocks.
constexpr int RING = 2, RING_BLOCKS = 4, RING_WORDS = RING_BLOCKS * (BM_CTA + 2);
constexpr int BOX = 64;
constexpr int BAR_BYTES = 512;
// What C holds: fp32, bf16, or fp16 times a power of two for each 128 columns of a row (the
// experts' y in large calls).
constexpr int kF32 = 0, kBf16 = 1, kScaled16 = 2;
// Shared memory: the ring of operands, and for each drain warp the rows it is about to
// store (32 rows of 128 bytes of C, or of 64 codes).
template <bool SW, bool OUT_16>
struct Mem {
  // rows of C of 16 bits are stored by four warps of their own, while the next item is multiplied
  static constexpr bool STORERS = !SW && OUT_16;
  static constexpr int THREADS = STORERS ? 512 : 384;
  // registers: 128 threads with few and 256 with many of 384 x 168, or 256 and 256 of 512 x 128
  static constexpr int FEW = STORERS ? 48 : 88, MANY = 208, LAUNCH = STORERS ? 128 : 168;
  static_assert((THREADS - 256) * FEW + 256 * MANY <= THREADS * LAUNCH, "registers that a warp waits for exist");
  static constexpr int STAGES = SW ? 6 : STORERS ? 4 : 5;
  static constexpr int OUT_WARP = 32 * (SW ? 64 : STORERS ? 256 : 128), OUT_BYTES = EPI_WARPS * OUT_WARP;
  static constexpr int BYTES = STAGES * STAGE_BYTES + OUT_BYTES + RING * RING_WORDS * 4 + 2 * BM_CTA * 4 + kListBytes +
                               BAR_BYTES + 1024;
  static_assert(BYTES <= 232448, "shared memory");
  static_assert(8 * (2 * STAGES + 4 * NBUF + 2 * RING + 7 + 2 * EPI_WARPS) <= BAR_BYTES, "barrier area");
};
static_assert(blocks_box_rows(kBlocksWide, false) == BOX, "boxes of A");
constexpr uint64_t kDrainGraceNs = 50000;              // after an abort, time for the other CTA's copies to land
constexpr uint16_t kBothCtas = 0x3;

struct Params {
  BlocksArgs a;
  int kblocks, tiles_n;
  int c_vec;                                           // C's rows are 16-byte-aligned vectors
  int sa_vec;                                          // A's scales: 16-byte-aligned vectors of four blocks
  int c_rows;                                          // and whole ones, and beta is 0: stored row by row
};

// Hardware barriers 1 to 4: accumulator (buffer b, half h) and, every fourth block, its
// scales are there; the signal warp and the half's four drain warps meet there.  (Eight
// warps that poll mbarriers themselves keep the queue to shared memory full.)  All five wait:
// a signal warp that only arrived would run ahead, and its second arrival in a phase (an
// abort comes while the first is pending) would end that phase without one of the drain
// warps, for good.  This way every phase has the same five warps, whatever the signal warp
// has found, and nobody can be left waiting: all go through the same blocks to the end,
// after an abort without results.  It is also faster: the polls for a block stop while the
// drain warps are not back yet (8192 x 11008 x 4096: 262 us, 270 with arrivals).
__device__ __forceinline__ void sync_signal(int b, int h) {
  if (h == 0) {
    if (b == 0) asm volatile("bar.sync 1, 160;" ::: "memory");
    else asm volatile("bar.sync 2, 160;" ::: "memory");
  } else {
    if (b == 0) asm volatile("bar.sync 3, 160;" ::: "memory");
    else asm volatile("bar.sync 4, 160;" ::: "memory");
  }
}
// Barrier 5 of the 256 drain threads; and the same, returning whether any of them has `p`.
__device__ __forceinline__ void sync_drain() { asm volatile("bar.sync 5, 256;" ::: "memory"); }
__device__ __forceinline__ bool any_drain(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 5, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(p ? 1u : 0u)
      : "memory");
  return r != 0;
}

// 32 columns n .. of row m of C from this thread's sums
template <bool OUT_BF16>
__device__ __forceinline__ void store32(const Params& p, long long m, int n, const uint64_t* v) {
  const BlocksArgs& a = p.a;
  if (p.c_vec && n + 32 <= a.N) {
    if constexpr (OUT_BF16) {
      __nv_bfloat16* c = static_cast<__nv_bfloat16*>(a.C) + m * a.ldc + n;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = a.alpha * part2(v[q * 4 + i / 2], i & 1);
        if (a.beta != 0.f) {
          const uint4 o = *reinterpret_cast<const uint4*>(c + q * 8);
          const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f[2 * i] = fmaf(a.beta, __uint_as_float(w[i] << 16), f[2 * i]);
            f[2 * i + 1] = fmaf(a.beta, __uint_as_float(w[i] & 0xffff0000u), f[2 * i + 1]);
          }
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(c + q * 8) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
      float* c = static_cast<float*>(a.C) + m * a.ldc + n;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = a.alpha * part2(v[q * 2 + i / 2], i & 1);
        if (a.beta != 0.f) {
          const float4 o = *reinterpret_cast<const float4*>(c + q * 4);
          f[0] = fmaf(a.beta, o.x, f[0]);
          f[1] = fmaf(a.beta, o.y, f[1]);
          f[2] = fmaf(a.beta, o.z, f[2]);
          f[3] = fmaf(a.beta, o.w, f[3]);
        }
        *reinterpret_cast<float4*>(c + q * 4) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (n + i < a.N) blocks_store(a, m, n + i, part2(v[i / 2], i & 1));
  }
}

// A power of two that takes the sums of a row's 128 columns into fp16.  `scales` is the sum of
// |sa * sb| over the blocks of K; a block's products come to 128 * 448 * 448 < 2^25 at most, so
// with the bound 2^25 * scales below 2^15 none is past 65504, and all down to 2^-29 of that bound
// keep 11 bits (random codes of three in four bits come to 2^-10 of it).  No look at the sums
// is taken: their largest, found in registers, cost 0.9 us an item.  2^113 at most, which takes
// any fp32 number, and 2^-112 at least, so that both it and its reciprocal are normal numbers.
__device__ __forceinline__ float scale_for(float scales) {
  const int e = (int)(__float_as_uint(scales) >> 23 & 255) + 25 - 14;
  return __uint_as_float((uint32_t)min(max(e, 127 - 112), 127 + 113) << 23);
}

// Rows of 128 bytes (64 columns of 16 bits or 32 of fp32) of a warp's 32 rows of C, by way of shared
// memory: a thread has a row, and 32 threads writing 16 bytes each of 32 rows take 32
// wavefronts where four whole rows of 128 bytes take four.  The 16-byte vectors of a row
// are permuted by the row's number, so neither side meets a bank twice.
template <int KIND>
__device__ __forceinline__ void stage_rows(float alpha, uint8_t* out, const uint64_t* v, int lane) {
  const uint64_t f = both(alpha);
  constexpr bool WORD = KIND == kF32;                  // a value fills one
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t x = mul2(v[WORD ? q * 2 + i / 2 : q * 4 + i], f);
      if constexpr (KIND == kBf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(part2(x, 0), part2(x, 1));
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else if constexpr (KIND == kScaled16) {
        const __half2 b = __floats2half2_rn(part2(x, 0), part2(x, 1));
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      } else {
        w[i] = __float_as_uint(part2(x, i & 1));
      }
    }
    *reinterpret_cast<uint4*>(out + lane * 128 + ((q ^ (lane & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The rows, from column n, up to column `end`.  to: this lane's row of C, or -1.
template <int KIND>
__device__ __forceinline__ void send_rows(const Params& p, const uint8_t* out, int to, int n, int end, int lane) {
  const BlocksArgs& a = p.a;
  constexpr int PER = KIND == kF32 ? 4 : 8;            // columns of a vector
  uint8_t* C = static_cast<uint8_t*>(a.C);
  const int c = lane & 7;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int row = q * 4 + lane / 8;
    const long long o = __shfl_sync(0xffffffffu, to, row);
    if (o >= 0 && n + c * PER < end)
      *reinterpret_cast<uint4*>(C + (o * a.ldc + n) * (16 / PER) + c * 16) =
          *reinterpret_cast<const uint4*>(out + row * 128 + ((c ^ (row & 7)) * 16));
  }
}

// SW: gate and up weights, codes out.  KIND: what C holds.
template <bool SW, int KIND>
__global__ void __launch_bounds__(Mem<SW, KIND != kF32>::THREADS, 1)
    blocks_wide_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                       const __grid_constant__ CUtensorMap mapB2, const Params p) {
  constexpr int BN = SW ? 128 : 256;                   // columns of C (or of h) an item
  using M = Mem<SW, KIND != kF32>;
  constexpr int STAGES = M::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;        // the same offset in both CTAs
  uint8_t* base_ptr = smem_raw + (base - raw);
  auto a_tile = [&](int s) { return base + s * STAGE_BYTES; };
  auto b_tile = [&](int s) { return base + s * STAGE_BYTES + A_BYTES; };
  uint8_t* at = base_ptr + STAGES * STAGE_BYTES;
  uint8_t* out = at;                                   // [EPI_WARPS][OUT_WARP]
  at += M::OUT_BYTES;
  float* ring = reinterpret_cast<float*>(at);          // [RING][RING_WORDS]
  at += RING * RING_WORDS * 4;
  float* big = reinterpret_cast<float*>(at);           // [2][BM_CTA]: largest values of halves, or scales
  at += 2 * BM_CTA * 4;
  const uint32_t bar_base = base + (uint32_t)(at - base_ptr);
  uint8_t* bar_ptr = at;
  at += BAR_BYTES;
  int* pre = reinterpret_cast<int*>(at);
  int* beg = pre + kBlocksMaxExperts + 1;
  int* num = beg + kBlocksMaxExperts;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b, int h) { return bar_base + 8u * (2 * STAGES + 2 * b + h); };
  auto tempty_bar = [&](int b, int h) { return bar_base + 8u * (2 * STAGES + 2 * NBUF + 2 * b + h); };
  auto sfull_bar = [&](int r) { return bar_base + 8u * (2 * STAGES + 4 * NBUF + r); };
  auto sempty_bar = [&](int r) { return bar_base + 8u * (2 * STAGES + 4 * NBUF + RING + r); };
  const uint32_t drain_bar = bar_base + 8u * (2 * STAGES + 4 * NBUF + 2 * RING);
  const uint32_t stall_bar = drain_bar + 8u;           // test hook: nothing arrives
  // STORERS: the rows of drain warp w (0 to 7) are there; are stored
  auto ofull_bar = [&](int w) { return stall_bar + 8u * (1 + w); };
  auto oempty_bar = [&](int w) { return stall_bar + 8u * (1 + EPI_WARPS + w); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * (2 * STAGES + 4 * NBUF + 2 * RING + 2 + 2 * EPI_WARPS));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // what may still have to land when a role has given up: stages with copies, the parities
  // of their last ones, and whether an MMA was issued
  volatile uint32_t* landing = tmem_slot + 2;

  const BlocksArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank() & 1u;        // clusters hold one pair
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < NBUF; ++b)
      for (int h = 0; h < 2; ++h) {
        mbar_init(tfull_bar(b, h), 1);
        mbar_init(tempty_bar(b, h), EPI_WARPS);        // four warps of each CTA
      }
    for (int r = 0; r < RING; ++r) {
      mbar_init(sfull_bar(r), 32);
      mbar_init(sempty_bar(r), EPI_WARPS);
    }
    for (int w = 0; w < 2 * EPI_WARPS; ++w) mbar_init(ofull_bar(w), 1);
    mbar_init(drain_bar, 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    for (int q = 0; q < 3; ++q) landing[q] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mapA);
    tma_prefetch_desc(&mapB);
    if (SW) tma_prefetch_desc(&mapB2);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (!a.early) griddep_wait();
  if (warp == 3) list_row_tiles<BM>(a, pre, beg, num, lane);
  tc_fence_before();
  cluster_sync();                                      // barriers, lists and TMEM of both CTAs
  tc_fence_after();
  // the next kernel may take an SM as soon as this one leaves it
  griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  const int items = pre[a.experts] * p.tiles_n;         // in 32 bits: the host has seen to it
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  Walk walk{pre, beg, num, BM, p.tiles_n, 0};
  // a pair without work waits too, so that this kernel never ends before the one before
  if (a.early && first >= items) griddep_wait();

  if (warp < EPI_FIRST) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(M::FEW));
    if (warp == 0) {
      // ------------------------------------------------------------ copies
      if (elect_one_sync()) {
        uint32_t issued = 0, issued_par = 0;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int it = first; ok && it < items; it += step) {
          const Item i = walk.at(it);
          const int mine = min(max(i.rows - (int)rank * BM_CTA, 0), BM_CTA);      // this CTA's rows
          const int other = i.rows - mine;
          const int p0 = i.p0 + (int)rank * BM_CTA;
          // rows that are not there are not copied: what their lanes sum up is not read
          auto copies = [](int rows) { return (rows + BOX - 1) / BOX; };
          const uint32_t bytes = (uint32_t)(2 * B_BYTES + (copies(mine) + copies(other)) * BOX * BK);
          // both CTAs' copies of a stage complete on the leader's barrier
          auto weights = [&](int st, int kb) {
            if (leader) mbar_arrive_expect_tx(full_bar(st), bytes);
            tma_load_3d_pair(b_tile(st), SW && rank == 1 ? &mapB2 : &mapB, map_to_rank(full_bar(st), 0),
                             i.nb * BN + (SW ? 0 : (int)rank * 128), kb * BK, i.e);
          };
          // the ring is empty at first: its weights are on their way while the kernel before
          // writes A
          const int ahead = it == first ? min(STAGES, p.kblocks) : 0;
          for (int st = 0; st < ahead; ++st) weights(st, st);
          if (it == first && a.early) griddep_wait();
          for (int kb = 0; kb < p.kblocks; ++kb) {
            if (kb >= ahead) {
              if (!mbar_wait(empty_bar(stage), phase ^ 1u, a.timeout_ns, abort_flag)) {
                if (!*abort_flag) report_status(a.status, 5, kSiteWideProducer);
                *abort_flag = 1;
                ok = false;
                break;
              }
              weights(stage, kb);
            }
            for (int c = 0; c < copies(mine); ++c)
              tma_load_2d_pair(a_tile(stage) + c * BOX * BK, &mapA, map_to_rank(full_bar(stage), 0), kb * BK, p0 + c * BOX);
            issued |= 1u << stage;
            issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        landing[0] = issued;
        landing[1] = issued_par;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA (leader)
      // The whole warp goes through the loop and one lane issues: descriptors are then the
      // same for all lanes and stay in uniform registers, where the instruction wants them.
      if (leader) {
        constexpr uint32_t idesc = idesc_f8_f32(BM, COLS / 2, kE4M3, kE4M3, /*A K-major*/ 0, /*B MN-major*/ 1);
        const uint64_t a_desc = smem_desc_sw128(a_tile(0), 16, 1024), b_desc = smem_desc_sw128(b_tile(0), B_BYTES, 1024);
        const bool one = elect_one_sync();
        int stage = 0, b = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true, issued_any = false;
        if (a.stall && first == 0 && !__all_sync(0xffffffffu, mbar_wait(stall_bar, 0, a.timeout_ns / 4, abort_flag))) {
          if (!*abort_flag) report_status(a.status, 5, kSiteWideMma);
          *abort_flag = 1;
          ok = false;
        }
        for (int it = first; ok && it < items; it += step) {
          for (int kb = 0; kb < p.kblocks; ++kb) {
            ok = __all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, a.timeout_ns, abort_flag));
            const uint64_t off = (uint64_t)(stage * (STAGE_BYTES >> 4));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok && __all_sync(0xffffffffu, mbar_wait(tempty_bar(b, h), bphase ^ 1u, a.timeout_ns, abort_flag));
              if (!ok) break;
              tc_fence_after();
              const uint32_t d = tmem_base + (uint32_t)(b * COLS + h * (COLS / 2));
              if (one) {
#pragma unroll
                for (int kk = 0; kk < BK / 32; ++kk)
                  tc_mma_f8_pair(d, a_desc + off + (kk * 32 >> 4), b_desc + off + ((kk * 32 * 128 + h * 64) >> 4), idesc,
                                 kk != 0 ? 1u : 0u);
                tc_commit_pair_mc(tfull_bar(b, h), kBothCtas);
                if (h == 1) tc_commit_pair_mc(empty_bar(stage), kBothCtas);
              }
              issued_any = true;
            }
            if (!ok) {
              if (!*abort_flag) report_status(a.status, 5, kSiteWideMma);
              *abort_flag = 1;
              break;
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            if (++b == NBUF) {
              b = 0;
              bphase ^= 1u;
            }
          }
        }
        if (one) landing[2] = issued_any ? 1 : 0;
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ scales
      int r = 0;
      uint32_t rphase = 0;
      bool ok = true;
      for (int it = first; ok && it < items; it += step) {
        const Item i = walk.at(it);
        const float* row[BM_CTA / 32];
#pragma unroll
        for (int q = 0; q < BM_CTA / 32; ++q) {
          const int m = (int)rank * BM_CTA + q * 32 + lane;
          int from = -1, to;
          if (m < i.rows) expert_row(a, i.p0 + m, from, to);
          row[q] = from >= 0 ? a.sa + (long long)from * a.ldsa : nullptr;
        }
        if (it == first && a.early) griddep_wait();
        // B's scales of the item's column blocks: lane 0 the first, lane 1 the second
        const int col = SW ? i.nb : 2 * i.nb + lane;
        const float* sb = nullptr;
        if (lane < 2 && (SW || col * 128 < a.N)) sb = (SW && lane == 1 ? a.sb2 : a.sb) + i.e * a.sb_stride + col;
        for (int kb = 0; kb < p.kblocks; kb += RING_BLOCKS) {
          if (!__all_sync(0xffffffffu, mbar_wait(sempty_bar(r), rphase ^ 1u, a.timeout_ns, abort_flag))) {
            if (!*abort_flag) report_status(a.status, 5, kSiteWideScales);
            *abort_flag = 1;
            ok = false;
            break;
          }
          const uint32_t to = smem_u32(ring + r * RING_WORDS);
#pragma unroll
          for (int q = 0; q < BM_CTA / 32; ++q)
            if (row[q] != nullptr) {
              const uint32_t at_row = to + (q * 32 + lane) * 16;
              if (p.sa_vec && kb + RING_BLOCKS <= p.kblocks) {
                cp_async_16(at_row, row[q] + kb, true);
              } else {
#pragma unroll
                for (int u = 0; u < RING_BLOCKS; ++u)
                  if (kb + u < p.kblocks) cp_async_4(at_row + u * 4, row[q] + kb + u);
              }
            }
          if (sb != nullptr)
#pragma unroll
            for (int u = 0; u < RING_BLOCKS; ++u)
              if (kb + u < p.kblocks) cp_async_4(to + ((BM_CTA + lane) * 4 + u) * 4, sb + (kb + u) * a.ldsb);
          cp_async_arrive(sfull_bar(r));
          if (++r == RING) {
            r = 0;
            rphase ^= 1u;
          }
        }
      }
      cp_async_commit();
      cp_async_wait<0>();                              // none in flight when the CTA leaves
    } else {
      // ------------------------------------------------------------ signals
      int b = 0, r = 0;
      uint32_t bphase = 0, rphase = 0;
      bool ok = true;
      for (int it = first; it < items; it += step)
        for (int kb = 0; kb < p.kblocks; ++kb) {
          const int u = kb % RING_BLOCKS;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (ok) {
              if (lane == 0) {
                ok = (h != 0 || u != 0 || mbar_wait(sfull_bar(r), rphase, a.timeout_ns, abort_flag)) &&
                     mbar_wait(tfull_bar(b, h), bphase, a.timeout_ns, abort_flag);
                if (!ok) {
                  if (!*abort_flag) report_status(a.status, 5, kSiteWideEpilogue);
                  *abort_flag = 1;
                }
              }
              ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            }
            tc_fence_after();
            tc_fence_before();
            sync_signal(b, h);
          }
          if (u == RING_BLOCKS - 1 || kb + 1 == p.kblocks) {
            if (++r == RING) {
              r = 0;
              rphase ^= 1u;
            }
          }
          if (++b == NBUF) {
            b = 0;
            bphase ^= 1u;
          }
        }
    }
  } else if (M::STORERS && warp >= STORE_FIRST) {
    // ------------------------------------------------------------ rows of C
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(M::FEW));
    const int quarter = warp - STORE_FIRST;            // of drain warps quarter and quarter + 4
    uint32_t phase = 0;
    bool ok = p.c_rows != 0;
    for (int it = first; ok && it < items; it += step) {
      const Item i = walk.at(it);
      const int m = (int)rank * BM_CTA + quarter * 32 + lane;
      int from, to = -1;
      if (m < i.rows) expert_row(a, i.p0 + m, from, to);
      for (int half = 0; ok && half < 2; ++half) {
        const int w = half * 4 + quarter;
        ok = __all_sync(0xffffffffu, mbar_wait(ofull_bar(w), phase, a.timeout_ns, abort_flag));
        if (!ok) {
          if (!*abort_flag) report_status(a.status, 5, kSiteWideRows);
          *abort_flag = 1;
          break;
        }
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          const int n = i.nb * BN + c * 128 + half * 64;
          if (n >= a.N) break;
          send_rows<KIND>(p, out + w * M::OUT_WARP + c * 4096, to, n, KIND == kScaled16 ? (int)a.ldc : a.N, lane);
          if (KIND == kScaled16 && half == 0 && to >= 0)
            a.ys[to * a.ldys + n / 128] = big[c * BM_CTA + quarter * 32 + lane];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(oempty_bar(w));
      }
      phase ^= 1u;
    }
  } else {
    // ------------------------------------------------------------ drain and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(M::MANY));
    uint32_t ophase = 0;
    const int quarter = warp % 4, half = (warp - EPI_FIRST) / 4;
    const int lrow = quarter * 32 + lane, m = (int)rank * BM_CTA + lrow;       // row of the CTA, of the item
    const uint32_t t_lane = tmem_base + ((uint32_t)(quarter * 32) << 16);
    const uint32_t lead_tempty = map_to_rank(tempty_bar(0, half), 0);
    int b = 0, r = 0;
    bool ok = true;                                    // not after an abort: then only the barriers count
    for (int it = first; it < items; it += step) {
      const Item i = walk.at(it);
      // this half's columns: 64 from each CTA's part of B (plain: half * 64 .. and 128 + half *
      // 64 .. of the item's; gate and up: half * 64 .. of each)
      int to = -1;                                     // read now, used when K is through
      if (!SW && !(M::STORERS && p.c_rows) && m < i.rows) {
        int from;
        expert_row(a, i.p0 + m, from, to);
      }
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0;
      float scales[2] = {0.f, 0.f};                    // kScaled16: sums of |s0| and |s1|
      for (int kb = 0; kb < p.kblocks; ++kb) {
        const int u = kb % RING_BLOCKS;
        sync_signal(b, half);
        if (*abort_flag) ok = false;
        tc_fence_after();
        const uint32_t sums = t_lane + (uint32_t)(b * COLS + half * (COLS / 2));
        uint32_t v[2][16];
        tmem_ld_32x32b_x16(sums, v[0]);
        const float* slot = ring + r * RING_WORDS + u;
        const float sa = slot[lrow * 4], sb0 = slot[BM_CTA * 4], sb1 = slot[BM_CTA * 4 + 4];
        const float s0 = sa * sb0, s1 = sa * sb1;
        if constexpr (KIND == kScaled16) {
          scales[0] += fabsf(s0);
          scales[1] += fabsf(s1);
        }
        const uint64_t d0 = pack2(__float_as_uint(s0), __float_as_uint(s0));
        const uint64_t d1 = pack2(__float_as_uint(s1), __float_as_uint(s1));
#pragma unroll
        for (int c = 0; c < 8; ++c) {                  // 16 sums are added while the next 16 come
          tc_wait_ld_x16(v[c & 1]);
          if (c < 7) {
            tmem_ld_32x32b_x16(sums + (uint32_t)(c * 16 + 16), v[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote_light(lead_tempty + 16u * b);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) fma2(acc[c * 8 + j], pack2(v[c & 1][2 * j], v[c & 1][2 * j + 1]), c < 4 ? d0 : d1);
        }
        if (u == RING_BLOCKS - 1 || kb + 1 == p.kblocks) {
          if (lane == 0) mbar_arrive(sempty_bar(r));   // its lanes have read: __syncwarp above
          if (++r == RING) r = 0;
        }
        b ^= 1;
      }
      if constexpr (SW) {
        // the eight warps meet below: they go on or give up together
        ok = !any_drain(!ok);
        if (!ok) continue;
        const int n = i.nb * BN + half * 64;
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] = swiglu_near2(acc[j], acc[32 + j]);
        if (n + 64 > a.N) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            acc[j] = pack2(n + 2 * j < a.N ? __float_as_uint(part2(acc[j], 0)) : 0u,
                           n + 2 * j + 1 < a.N ? __float_as_uint(part2(acc[j], 1)) : 0u);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)                   // fmaxf leaves NaN out
          top = fmaxf(top, fmaxf(fabsf(part2(acc[j], 0)), fabsf(part2(acc[j], 1))));
        big[half * BM_CTA + lrow] = top;
        sync_drain();
        const float s = kv_scale_for<kKvE4M3>(fmaxf(top, big[(1 - half) * BM_CTA + lrow]));
        const uint64_t f = both(kv_recip(s));
        // 64 codes of this thread's row, then rows of 64 bytes (as stage_rows)
        uint8_t* mine = out + (warp - EPI_FIRST) * M::OUT_WARP;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t x = mul2(acc[c * 8 + 2 * k], f), y = mul2(acc[c * 8 + 2 * k + 1], f);
            w[k] = kv_code2<kKvE4M3>(part2(x, 0), part2(x, 1)) | (kv_code2<kKvE4M3>(part2(y, 0), part2(y, 1)) << 16);
          }
          *reinterpret_cast<uint4*>(mine + lane * 64 + ((c ^ ((lane >> 1) & 3)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (half == 0 && m < i.rows) a.hs[((long long)i.p0 + m) * a.ldhs + i.nb] = s;
        __syncwarp();
        const int rows = i.rows - ((int)rank * BM_CTA + quarter * 32);         // of this warp
        const int c = lane & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = q * 8 + lane / 4;
          // rows of a.hq are whole vectors; codes past N are 0
          if (row < rows && n + c * 16 < a.ldh)
            *reinterpret_cast<uint4*>(a.hq + ((long long)i.p0 + i.rows - rows + row) * a.ldh + n + c * 16) =
                *reinterpret_cast<const uint4*>(mine + row * 64 + ((c ^ ((row >> 1) & 3)) * 16));
        }
        __syncwarp();
      } else {
        if (!ok) continue;
        const int n = i.nb * BN + half * 64;
        if (p.c_rows) {
          const int w = warp - EPI_FIRST;
          uint8_t* mine = out + w * M::OUT_WARP;
          if constexpr (M::STORERS) {
            if (!__all_sync(0xffffffffu, mbar_wait(oempty_bar(w), ophase ^ 1u, a.timeout_ns, abort_flag))) {
              if (!*abort_flag) report_status(a.status, 5, kSiteWideRows);
              *abort_flag = 1;
              ok = false;
              continue;
            }
            ophase ^= 1u;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float f = a.alpha;
              if constexpr (KIND == kScaled16) {       // 1/s is exact
                const float s = scale_for(scales[c]);
                f = __uint_as_float((254u << 23) - __float_as_uint(s));
                if (half == 0) big[c * BM_CTA + lrow] = s;
              }
              stage_rows<KIND>(f, mine + c * 4096, acc + c * 32, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ofull_bar(w));
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int at = n + c / 2 * 128 + c % 2 * 32;
              if (at >= a.N) break;
              stage_rows<KIND>(a.alpha, mine, acc + c * 16, lane);
              __syncwarp();
              send_rows<KIND>(p, mine, to, at, a.N, lane);
              __syncwarp();                            // read before the next rows are written
            }
          }
        } else if (to >= 0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = n + c / 2 * 128 + c % 2 * 32;
            if (at < a.N) store32<KIND == kBf16>(p, to, at, acc + c * 16);
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  // All roles of both CTAs are through, so the flag is final: whichever of them gave up, and
  // however late, no memory is given back while a copy or an MMA may still write to it.  Both
  // CTAs' copies of a stage complete on the leader's barrier; the peer may have issued some
  // that the leader did not, whose barrier says nothing then.
  if (*abort_flag) {
    if (leader && warp == 0 && lane == 0)
#pragma unroll 1
      for (int st = 0; st < STAGES; ++st)
        if (((landing[0] >> st) & 1u) && !mbar_wait(full_bar(st), (landing[1] >> st) & 1u, kDrainWaitNs, nullptr))
          report_status(a.status, 5, kSiteWideDrain);
    // the thread that issued the MMAs: election gives the same lane again
    if (leader && warp == 1 && elect_one_sync() && landing[2] != 0) {
      tc_commit_pair_mc(drain_bar, 0x1);
      if (!mbar_wait(drain_bar, 0, kDrainWaitNs, nullptr)) report_status(a.status, 5, kSiteWideDrain);
    }
    if (warp == 0) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < kDrainGraceNs) {
      }
    }
    __syncwarp();
  }
  cluster_sync();                                      // both CTAs are done with the pair's TMEM and barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

struct PairInfo {
  std::atomic<bool> ready{false};
  int max_clusters = 0;
};

template <bool SW, int KIND>
int launch_impl(const BlocksArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, const CUtensorMap* mapB2,
                int num_sms, cudaStream_t s) {
  static PairInfo info[64];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = blocks_wide_kernel<SW, KIND>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(Mem<SW, KIND != kF32>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Mem<SW, KIND != kF32>::BYTES;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (!info[dev].ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    if (!info[dev].ready.load(std::memory_order_relaxed)) {
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
      // with fewer registers at launch the warps that take some would wait forever
      if (fa.numRegs < Mem<SW, KIND != kF32>::LAUNCH) return cudaErrorInvalidConfiguration;
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Mem<SW, KIND != kF32>::BYTES)) != cudaSuccess)
        return e;
      int n = 0;
      cfg.gridDim = dim3(2 * (num_sms / 2), 1, 1);
      if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
      info[dev].max_clusters = n > 0 ? n : 1;
      info[dev].ready.store(true, std::memory_order_release);
    }
  }
  Params p;
  p.a = a;
  p.kblocks = (a.K + BK - 1) / BK;
  p.tiles_n = (a.N + (SW ? 128 : 256) - 1) / (SW ? 128 : 256);
  const int osz = KIND == kF32 ? 4 : 2;
  p.sa_vec = ((reinterpret_cast<uintptr_t>(a.sa) & 15u) == 0 && a.ldsa % 4 == 0) ? 1 : 0;
  p.c_vec = ((reinterpret_cast<uintptr_t>(a.C) & 15u) == 0 && (a.ldc * osz) % 16 == 0) ? 1 : 0;
  p.c_rows = p.c_vec != 0 && (KIND == kScaled16 || a.N % (16 / osz) == 0) && a.beta == 0.f ? 1 : 0;
  if (KIND == kScaled16 && (p.c_rows == 0 || a.alpha != 1.f)) return cudaErrorInvalidValue;
  const long long items = blocks_row_tiles(a.rows, a.offsets != nullptr ? a.experts : 1, BM) * p.tiles_n;
  const long long clusters = items < info[dev].max_clusters ? items : info[dev].max_clusters;
  cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, *mapA, *mapB, SW ? *mapB2 : *mapB, p);
}

}  // namespace

int launch_blocks_wide(const BlocksArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, const CUtensorMap* mapB2,
                       int num_sms, cudaStream_t s) {
  if (a.gather != 0) return cudaErrorInvalidValue;
  if (a.B2 != nullptr) return launch_impl<true, kBf16>(a, mapA, mapB, mapB2, num_sms, s);
  if (a.ys != nullptr) return launch_impl<false, kScaled16>(a, mapA, mapB, mapB2, num_sms, s);
  return a.out_bf16 ? launch_impl<false, kBf16>(a, mapA, mapB, mapB2, num_sms, s)
                    : launch_impl<false, kF32>(a, mapA, mapB, mapB2, num_sms, s);
}

}  // namespace g3

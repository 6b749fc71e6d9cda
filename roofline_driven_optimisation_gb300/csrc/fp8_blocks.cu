// Products of E4M3 matrices with a scale for each 1 x 128 block of A and each 128 x 128
// block of B, for one matrix or for the slots of experts, on the tensor cores:
//
//     C[m][n] = alpha * sum over blocks b of sa[m][b] * sb[b][n/128] * S_b[m][n] + beta * C[m][n]
//
// and, for an expert's gate and up weights, silu(A*Bg) .* (A*Bu) as E4M3 codes with a
// scale for each 128 columns (the A of the product that follows).
//
// Operands swapped.  The MMA computes C^T: 128 columns of B are its M = 128 rows
// (N-major in shared memory) and up to NT rows of A its N columns.  A decode step's few
// rows then cost what they are (N is a multiple of 16, set tile by tile at run time, so
// an expert with 5 rows pays for 16), and a tile lies inside one column of B's scales.
// Calls with many rows go to fp8_blocks_wide.cu.
//
// Scales.  The tensor core sums one block of 128 k; its sum S_b is read out of TMEM and
// added with its scale to a sum in registers, so every sum is fp32 and no scale is
// rounded into a code.  With few rows the weights' bytes bound the call, and a block's
// 16 KB arrive every 250 cycles or so: handing one accumulator at a time to the drain
// warps, with their polls, cost 650 cycles a block and was what bounded it.  So TMEM holds two
// groups of up to four blocks' accumulators: MMA, scales and drain meet once a group,
// and the eight drain warps wait at a hardware barrier with a signal warp that polls
// for them.
//
// Roles (384 threads; one CTA an SM, two where K is split over tiles of 32 rows): warp 0
// copies (TMA; the experts' rows of A through tile::gather4, four rows an instruction, so
// that they are never laid out by expert; the first stages' weights before the rows'
// numbers are known), warp 1 issues the MMAs,
// warp 2 multiplies sa with sb for the drain, warp 3 signals, warps 4-11 drain: warp w
// the TMEM lanes 32*(w%4)..+31 (columns of B) and half of the tile's rows of A.
//
// Measured: gate and up of 64 tokens of 64 experts of 4096 and 1376 take 113 us, 0.97 of the
// copy rate; 1 x 11008 x 4096 takes 8.3 us, of which 6.7 are its bytes; 77 x 4096 x 11008
// takes 13 us (7), as each column tile reads the rows again.
//
// Epilogue: the sums go through shared memory, 32 rows of A at a time, and a warp then has
// a whole row's 128 columns: a row of C or of codes leaves as one piece, the largest
// magnitude for h's scale is one warp's, and rows that are not there cost nothing.
//
// Schedule: items (row tile of an expert, column tile) in a line, expert by expert,
// columns outermost inside an expert; CTA c takes items c, c + grid, ...  The counts are
// read on the device, so no launch depends on the routing.  Where a call has fewer items
// than SMs, K is split over a cluster of 2 to 8 CTAs, whose sums meet in distributed
// shared memory in rank order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "experts.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

constexpr int BK = kBlocksK, BN = kBlocksN;
constexpr int THREADS = 384, EPI_WARPS = 8, EPI_FIRST = 4;
constexpr int W_BYTES = BN * BK;               // a weight tile: 128 k rows of 128 columns
constexpr int SMEM_LIMIT = 232448;
constexpr int CHUNK = 32;                      // rows of A that go through shared memory at a time

// SPLIT: K is shared by a cluster, a CTA has one item, and its sums lie over the ring at the
// end.  Tiles of 32 rows then take half of an SM: an SM's copies from HBM come to about 57
// bytes a ns however many are in flight, so a decode step's few items have to reach every
// SM alike, and two CTAs an SM let 86 items be 258 parts (86 CTAs: 9.3 us for the 45 MB of
// a 4096 x 11008 weight).
template <int NT, bool SW, bool SPLIT>
struct Cfg {
  static constexpr int CTAS = SPLIT && NT == 32 ? 2 : 1;      // an SM
  static constexpr int LIMIT = CTAS == 2 ? 115200 : SMEM_LIMIT;
  static constexpr int OPS = SW ? 2 : 1;
  static constexpr int COLS = NT * OPS;                       // TMEM columns of an accumulator
  // blocks that are handed over together; the CTAs of an SM share its 512 TMEM columns
  static constexpr int GROUP = 256 / CTAS / COLS > 4 ? 4 : 256 / CTAS / COLS;
  static constexpr int TMEM_COLS = 2 * GROUP * COLS;
  static constexpr int STAGE_BYTES = OPS * W_BYTES + NT * BK;
  static constexpr int SCALE_BYTES = 2 * GROUP * COLS * 4;
  static constexpr int OUT_BYTES = SPLIT ? 0 : OPS * CHUNK * BN * 4;
  static constexpr int LIST_BYTES = SPLIT ? 64 : kListBytes;
  static constexpr int BAR_BYTES = 512;
  static constexpr int REST = SCALE_BYTES + OUT_BYTES + LIST_BYTES + BAR_BYTES + 1024;
  static constexpr int FIT = (LIMIT - REST) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 10 ? 10 : FIT;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + REST;
  static constexpr int BOX = NT >= 128 ? 64 : 16;             // rows of A in one copy
  static constexpr int CH = NT / 2;                           // rows of A a drain thread holds
  static constexpr int CW = CH >= 32 ? 32 : 16;               // TMEM columns read at a time
  static_assert(TMEM_COLS == 512 || TMEM_COLS == 256, "TMEM allocations are powers of two");
  static_assert(STAGES >= 3, "the ring needs three stages");
  static_assert(!SPLIT || OPS * NT * BN * 4 <= STAGES * STAGE_BYTES, "a split's sums lie over the ring");
  static_assert(8 * (2 * STAGES + 11) <= BAR_BYTES, "barrier area");
};

struct Params {
  BlocksArgs a;
  int kblocks, tiles_n, split;
  int c_vec;                    // four neighbouring columns of C (or codes) are one aligned vector
};

// Hardware barriers: 1 + g the drain warps and the signal warp at group buffer g, 3 the 256
// drain threads.  Nobody can be left waiting: both sides go through the same groups and
// items to the end, after an abort without results.
__device__ __forceinline__ void sync_signal(int g) {
  if (g == 0) asm volatile("bar.sync 1, 288;" ::: "memory");
  else asm volatile("bar.sync 2, 288;" ::: "memory");
}
__device__ __forceinline__ void sync_drain() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

template <int CW>
__device__ __forceinline__ void tmem_read(uint32_t addr, uint32_t (&r)[CW]) {
  if constexpr (CW == 32) tmem_ld_32x32b_x32(addr, r);
  else tmem_ld_32x32b_x16(addr, r);
  tc_wait_ld();
  // no value is used before the wait
#pragma unroll
  for (int i = 0; i < CW; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ int mma_rows(int rows) { return (rows + 15) & ~15; }

// The sums of four neighbouring columns of B for one row of A, over the cluster's ranks
// in order.
__device__ __forceinline__ float4 sum_ranks(uint32_t off, int split) {
  float4 part[8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < split) part[q] = ld_dsmem_f32x4(map_to_rank(off, (uint32_t)q));
  float4 s = part[0];
#pragma unroll
  for (int q = 1; q < 8; ++q)
    if (q < split) {
      s.x += part[q].x;
      s.y += part[q].y;
      s.z += part[q].z;
      s.w += part[q].w;
    }
  return s;
}

// Four neighbouring columns n .. of row p0 + m of the product, by a whole warp: s their sums
// (u the up-projection's).  Columns past N come as zeros.
template <bool SW>
__device__ __forceinline__ void finish_row(const Params& p, const Item& i, int m, float4 s, float4 u, int lane) {
  const BlocksArgs& a = p.a;
  const int n = i.nb * BN + lane * 4;
  const float sv[4] = {s.x, s.y, s.z, s.w};
  if constexpr (SW) {
    const float uv[4] = {u.x, u.y, u.z, u.w};
    float h[4], big = 0.f;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const uint64_t x = swiglu_near2(pack2(__float_as_uint(sv[q]), __float_as_uint(sv[q + 1])),
                                      pack2(__float_as_uint(uv[q]), __float_as_uint(uv[q + 1])));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        h[q + i] = n + q + i < a.N ? part2(x, i) : 0.f;
        big = fmaxf(big, fabsf(h[q + i]));                      // NaN is left out
      }
    }
    // as whole numbers magnitudes order as they are
    const float sc = kv_scale_for<kKvE4M3>(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big))));
    const float r = kv_recip(sc);
    const uint32_t c = kv_code2<kKvE4M3>(__fmul_rn(h[0], r), __fmul_rn(h[1], r)) |
                       (kv_code2<kKvE4M3>(__fmul_rn(h[2], r), __fmul_rn(h[3], r)) << 16);
    const long long row = i.p0 + m;
    // rows of a.hq are whole vectors; codes past N are 0
    if (n < a.ldh) *reinterpret_cast<uint32_t*>(a.hq + row * a.ldh + n) = c;
    if (lane == 0) a.hs[row * a.ldhs + i.nb] = sc;
  } else {
    int from, to;
    expert_row(a, i.p0 + m, from, to);
    if (to < 0) return;
    if (p.c_vec && n + 4 <= a.N) {
      float v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = a.alpha * sv[q];
      if (a.out_bf16) {
        uint2* c = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.C) + (long long)to * a.ldc + n);
        if (a.beta != 0.f) {
          const uint2 o = *c;
          v[0] = fmaf(a.beta, __uint_as_float(o.x << 16), v[0]);
          v[1] = fmaf(a.beta, __uint_as_float(o.x & 0xffff0000u), v[1]);
          v[2] = fmaf(a.beta, __uint_as_float(o.y << 16), v[2]);
          v[3] = fmaf(a.beta, __uint_as_float(o.y & 0xffff0000u), v[3]);
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *c = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        float4* c = reinterpret_cast<float4*>(static_cast<float*>(a.C) + (long long)to * a.ldc + n);
        if (a.beta != 0.f) {
          const float4 o = *c;
          v[0] = fmaf(a.beta, o.x, v[0]);
          v[1] = fmaf(a.beta, o.y, v[1]);
          v[2] = fmaf(a.beta, o.z, v[2]);
          v[3] = fmaf(a.beta, o.w, v[3]);
        }
        *c = make_float4(v[0], v[1], v[2], v[3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (n + q < a.N) blocks_store(a, to, n + q, sv[q]);
    }
  }
}

// GATHER: A's rows through tile::gather4 (mapA has boxes of one row).
template <int NT, bool SW, bool GATHER, bool SPLIT>
__global__ void __launch_bounds__(THREADS, Cfg<NT, SW, SPLIT>::CTAS)
    blocks_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                  const __grid_constant__ CUtensorMap mapB2, const __grid_constant__ Params p) {
  using C = Cfg<NT, SW, SPLIT>;
  constexpr int STAGES = C::STAGES, GROUP = C::GROUP, COLS = C::COLS, CH = C::CH, CW = C::CW;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  auto w_tile = [&](int s) { return base + s * C::STAGE_BYTES; };
  auto t_tile = [&](int s) { return base + s * C::STAGE_BYTES + C::OPS * W_BYTES; };
  uint8_t* at = base_ptr + STAGES * C::STAGE_BYTES;
  float* scales = reinterpret_cast<float*>(at);                  // [2][GROUP][COLS]
  at += C::SCALE_BYTES;
  float* out = reinterpret_cast<float*>(at);                     // [OPS][CHUNK][BN]
  at += C::OUT_BYTES;
  const uint32_t bar_base = base + (uint32_t)(at - base_ptr);
  uint8_t* bar_ptr = at;
  at += C::BAR_BYTES;
  int* pre = reinterpret_cast<int*>(at);                         // [experts + 1]
  int* beg = pre + kBlocksMaxExperts + 1;
  int* num = beg + kBlocksMaxExperts;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (STAGES + s); };
  auto tfull_bar = [&](int g) { return bar_base + 8u * (2 * STAGES + g); };
  auto tempty_bar = [&](int g) { return bar_base + 8u * (2 * STAGES + 2 + g); };
  auto sfull_bar = [&](int g) { return bar_base + 8u * (2 * STAGES + 4 + g); };
  const uint32_t drain_bar = bar_base + 8u * (2 * STAGES + 6);
  const uint32_t stall_bar = drain_bar + 8u;                     // test hook: nothing arrives
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + 8 * (2 * STAGES + 8));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // what may still have to land when a role has given up: stages with copies, the parities
  // of their last ones, and whether an MMA was issued
  volatile uint32_t* landing = tmem_slot + 2;

  const BlocksArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int split = SPLIT ? p.split : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(tfull_bar(g), 1);
      mbar_init(tempty_bar(g), EPI_WARPS);
      mbar_init(sfull_bar(g), 32);
    }
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
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (!a.early) griddep_wait();
  if (warp == 3) {
    if (SPLIT) find_item<NT>(a, p.tiles_n, blockIdx.x / split, pre, lane);
    else list_row_tiles<NT>(a, pre, beg, num, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // the next kernel may take an SM as soon as this one leaves it
  griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  // SPLIT: pre[0..3] is this cluster's item, if it has one; else the lists of all
  const int items = SPLIT ? (pre[2] > 0 ? 1 : 0) : pre[a.experts] * p.tiles_n;   // in 32 bits: the host has seen to it
  const int first = SPLIT ? 0 : blockIdx.x, step = SPLIT ? 1 : gridDim.x;
  // a block without work waits too, so that this kernel never ends before the one before
  if (a.early && first >= items) griddep_wait();
  // blocks of K of this rank
  const int k_lo = (int)((long long)p.kblocks * rank / split), k_hi = (int)((long long)p.kblocks * (rank + 1) / split);
  Walk walk{pre, beg, num, NT, p.tiles_n, 0};
  auto item_at = [&](int it) { return SPLIT ? Item{pre[0], pre[1], pre[2], pre[3]} : walk.at(it); };

  if (warp == 0) {
    // -------------------------------------------------------------- copies
    uint32_t issued = 0, issued_par = 0;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const bool leader = elect_one_sync();
    auto mark = [&](int s) {
      issued |= 1u << s;
      issued_par = (issued_par & ~(1u << s)) | (phase << s);
    };
    for (int it = first; ok && it < items; it += step) {
      const Item i = item_at(it);
      const int n_mma = mma_rows(i.rows);
      const int copies = (n_mma + C::BOX - 1) / C::BOX;
      const uint32_t bytes = (uint32_t)(C::OPS * W_BYTES + (GATHER ? n_mma : copies * C::BOX) * BK);
      auto weights = [&](int s, int kb) {
        mbar_arrive_expect_tx(full_bar(s), bytes);
        tma_load_3d(w_tile(s), &mapB, full_bar(s), i.nb * BN, kb * BK, i.e);
        if (SW) tma_load_3d(w_tile(s) + W_BYTES, &mapB2, full_bar(s), i.nb * BN, kb * BK, i.e);
      };
      // the ring is empty at first: its weights are on their way while `order` is read, and
      // while the kernel before writes A
      const int ahead = it == first ? min(STAGES, k_hi - k_lo) : 0;
      if (leader)
        for (int s = 0; s < ahead; ++s) weights(s, k_lo + s);
      __syncwarp();
      int y[4];
      const int group = lane * 4;                      // GATHER: this lane's four rows
      if (GATHER) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          int from = -1, to;
          if (group + q < i.rows) expert_row(a, i.p0 + group + q, from, to);
          y[q] = from >= 0 ? from : a.a_rows;         // outside: zeros
        }
      }
      if (it == first && a.early) griddep_wait();
      for (int kb = k_lo; kb < k_hi; ++kb) {
        const bool sent = kb - k_lo < ahead;           // its weights are under way
        if (!sent) {
          if ((GATHER || leader) && !mbar_wait(empty_bar(stage), phase ^ 1u, a.timeout_ns, abort_flag)) {
            if (!*abort_flag) report_status(a.status, 5, kSiteBlocksProducer);
            *abort_flag = 1;
            ok = false;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (leader) {
          if (!sent) weights(stage, kb);
          if (!GATHER)
            for (int c = 0; c < copies; ++c)
              tma_load_2d(t_tile(stage) + c * C::BOX * BK, &mapA, full_bar(stage), kb * BK, i.p0 + c * C::BOX);
        }
        if (GATHER) {
          __syncwarp();                                // the bytes are expected before any arrive
          if (group < n_mma)
            tma_gather4(t_tile(stage) + group * BK, &mapA, full_bar(stage), kb * BK, y[0], y[1], y[2], y[3]);
        }
        mark(stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (leader) {
      landing[0] = issued;
      landing[1] = issued_par;
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA
    if (elect_one_sync()) {
      int stage = 0, g = 0;
      uint32_t phase = 0, gphase = 0;
      bool ok = true, issued_any = false;
      if (a.stall && blockIdx.x == 0 && !mbar_wait(stall_bar, 0, a.timeout_ns / 4, abort_flag)) {
        if (!*abort_flag) report_status(a.status, 5, kSiteBlocksMma);
        *abort_flag = 1;
        ok = false;
      }
      for (int it = first; ok && it < items; it += step) {
        const Item i = item_at(it);
        const uint32_t idesc = idesc_f8_f32(BN, (uint32_t)mma_rows(i.rows), kE4M3, kE4M3, /*B^T MN-major*/ 1, /*A K-major*/ 0);
        for (int kb = k_lo; kb < k_hi; ++kb) {
          const int u = (kb - k_lo) % GROUP;
          ok = (u != 0 || mbar_wait(tempty_bar(g), gphase ^ 1u, a.timeout_ns, abort_flag)) &&
               mbar_wait(full_bar(stage), phase, a.timeout_ns, abort_flag);
          if (!ok) {
            if (!*abort_flag) report_status(a.status, 5, kSiteBlocksMma);
            *abort_flag = 1;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)((g * GROUP + u) * COLS);
#pragma unroll
          for (int op = 0; op < C::OPS; ++op)
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              tc_mma_f8(d + op * NT, smem_desc_sw128(w_tile(stage) + op * W_BYTES + kk * 32 * BN, W_BYTES, 1024),
                        smem_desc_sw128(t_tile(stage) + kk * 32, 16, 1024), idesc, kk != 0 ? 1u : 0u);
          issued_any = true;
          tc_commit(empty_bar(stage));
          if (u == GROUP - 1 || kb + 1 == k_hi) {
            tc_commit(tfull_bar(g));
            if (++g == 2) {
              g = 0;
              gphase ^= 1u;
            }
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      landing[2] = issued_any ? 1 : 0;
    }
  } else if (warp == 2) {
    // -------------------------------------------------------------- scales
    constexpr int PER = NT / 32;
    int g = 0;
    uint32_t gphase = 0;
    bool ok = true;
    for (int it = first; ok && it < items; it += step) {
      const Item i = item_at(it);
      const float* row[PER];
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        int from = -1, to;
        if (q * 32 + lane < i.rows) expert_row(a, i.p0 + q * 32 + lane, from, to);
        row[q] = from >= 0 ? a.sa + (long long)from * a.ldsa : nullptr;
      }
      const float* sb = a.sb + i.e * a.sb_stride + i.nb;
      const float* sb2 = SW ? a.sb2 + i.e * a.sb_stride + i.nb : nullptr;
      if (it == first && a.early) griddep_wait();
      // a group ahead: the loads land while the one before is drained (plain loads: read-only
      // ones may be moved before the wait)
      float v[GROUP][PER], w[GROUP], w2[GROUP];
      auto load = [&](int kb) {
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
          const bool in = kb + u < k_hi;
#pragma unroll
          for (int q = 0; q < PER; ++q) v[u][q] = in && row[q] != nullptr ? row[q][kb + u] : 0.f;
          w[u] = in ? sb[(kb + u) * a.ldsb] : 0.f;
          if (SW) w2[u] = in ? sb2[(kb + u) * a.ldsb] : 0.f;
        }
      };
      load(k_lo);
      for (int kb = k_lo; kb < k_hi; kb += GROUP) {
        if (!__all_sync(0xffffffffu, mbar_wait(tempty_bar(g), gphase ^ 1u, a.timeout_ns, abort_flag))) {
          if (!*abort_flag) report_status(a.status, 5, kSiteBlocksScales);
          *abort_flag = 1;
          ok = false;
          break;
        }
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
          float* to = scales + (g * GROUP + u) * COLS + lane;
#pragma unroll
          for (int q = 0; q < PER; ++q) {
            to[q * 32] = v[u][q] * w[u];
            if (SW) to[NT + q * 32] = v[u][q] * w2[u];
          }
        }
        mbar_arrive(sfull_bar(g));
        if (++g == 2) {
          g = 0;
          gphase ^= 1u;
        }
        load(kb + GROUP);
      }
    }
  } else if (warp == 3) {
    // -------------------------------------------------------------- signals
    int g = 0;
    uint32_t gphase = 0;
    bool ok = true;
    for (int it = first; it < items; it += step)
      for (int kb = k_lo; kb < k_hi; kb += GROUP) {
        if (lane == 0 && ok) {
          ok = mbar_wait(sfull_bar(g), gphase, a.timeout_ns, abort_flag) &&
               mbar_wait(tfull_bar(g), gphase, a.timeout_ns, abort_flag);
          if (!ok) {
            if (!*abort_flag) report_status(a.status, 5, kSiteBlocksEpilogue);
            *abort_flag = 1;
          }
        }
        __syncwarp();
        tc_fence_after();
        tc_fence_before();
        sync_signal(g);
        if (++g == 2) {
          g = 0;
          gphase ^= 1u;
        }
      }
  } else {
    // -------------------------------------------------------------- drain and epilogue
    const int quarter = warp % 4, half = (warp - EPI_FIRST) / 4;
    const int nl = quarter * 32 + lane;                          // column of the tile
    const uint32_t t_lane = tmem_base + ((uint32_t)(quarter * 32) << 16);
    int g = 0;
    for (int it = first; it < items; it += step) {
      const Item i = item_at(it);
      const int n_mma = mma_rows(i.rows);
      uint64_t acc[C::OPS][CH / 2];
#pragma unroll
      for (int op = 0; op < C::OPS; ++op)
#pragma unroll
        for (int j = 0; j < CH / 2; ++j) acc[op][j] = 0;
      for (int kb = k_lo; kb < k_hi; kb += GROUP) {
        sync_signal(g);
        tc_fence_after();
#pragma unroll 1
        for (int u = 0; u < GROUP && kb + u < k_hi; ++u) {
          const int buf = (g * GROUP + u) * COLS;
#pragma unroll
          for (int c = 0; c < CH / CW; ++c) {
            const int col = half * CH + c * CW;                  // rows of A: col .. col + CW - 1
            if (col < n_mma) {
#pragma unroll
              for (int op = 0; op < C::OPS; ++op) {
                uint32_t r[CW];
                tmem_read<CW>(t_lane + (uint32_t)(buf + op * NT + col), r);
                const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(scales + buf + op * NT + col);
#pragma unroll
                for (int j = 0; j < CW / 4; ++j) {
                  const ulonglong2 s = sc[j];
                  fma2(acc[op][c * CW / 2 + 2 * j], pack2(r[4 * j], r[4 * j + 1]), s.x);
                  fma2(acc[op][c * CW / 2 + 2 * j + 1], pack2(r[4 * j + 2], r[4 * j + 3]), s.y);
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty_bar(g));
        g ^= 1;
      }
      auto value = [&](int op, int j) { return part2(acc[op][j / 2], j & 1); };
      if constexpr (SPLIT) {
        // this rank's sums, [row of A][column of B], over the ring (every copy has landed
        // and every MMA has read: the last accumulator is complete)
        float* part = reinterpret_cast<float*>(base_ptr);
#pragma unroll
        for (int op = 0; op < C::OPS; ++op)
#pragma unroll
          for (int j = 0; j < CH; ++j)
            if (half * CH + j < i.rows) part[(op * NT + half * CH + j) * BN + nl] = value(op, j);
      } else {
#pragma unroll
        for (int c = 0; c < CH / 16; ++c) {                      // 16 rows of each half
          if (c > 0 || it != first) sync_drain();                // the chunk before is stored
#pragma unroll
          for (int op = 0; op < C::OPS; ++op)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (half * CH + c * 16 + j < i.rows) out[(op * CHUNK + half * 16 + j) * BN + nl] = value(op, c * 16 + j);
          sync_drain();
          if (!*abort_flag)
#pragma unroll 1
            for (int x = warp - EPI_FIRST; x < CHUNK; x += EPI_WARPS) {
              const int m = x / 16 * CH + c * 16 + x % 16;
              if (m < i.rows) {
                const float4 s = *reinterpret_cast<const float4*>(out + x * BN + lane * 4);
                const float4 u = SW ? *reinterpret_cast<const float4*>(out + (CHUNK + x) * BN + lane * 4) : s;
                finish_row<SW>(p, i, m, s, u, lane);
              }
            }
        }
      }
    }
  }

  __syncwarp();
  if constexpr (SPLIT) {
    cluster_sync();                                              // every rank's sums are there
    if (first < items && !*abort_flag && warp >= EPI_FIRST) {
      const Item i = item_at(first);
      const uint32_t part = smem_u32(base_ptr);
#pragma unroll 1
      for (int m = rank + split * (warp - EPI_FIRST); m < i.rows; m += split * EPI_WARPS) {
        const uint32_t off = part + (uint32_t)(m * BN + lane * 4) * 4u;
        const float4 s = sum_ranks(off, split);
        const float4 u = SW ? sum_ranks(off + (uint32_t)(NT * BN) * 4u, split) : s;
        finish_row<SW>(p, i, m, s, u, lane);
      }
    }
    cluster_sync();                                              // no rank leaves while others read its sums
  }
  tc_fence_before();
  __syncthreads();
  // All roles are through, so the flag is final: whichever of them gave up, and however late,
  // no memory is given back while a copy or an MMA may still write to it.
  if (*abort_flag) {
    if (warp == 0 && lane == 0)
#pragma unroll 1
      for (int st = 0; st < STAGES; ++st)
        if (((landing[0] >> st) & 1u) && !mbar_wait(full_bar(st), (landing[1] >> st) & 1u, kDrainWaitNs, nullptr))
          report_status(a.status, 5, kSiteBlocksDrain);
    // the thread that issued the MMAs: election gives the same lane again
    if (warp == 1 && elect_one_sync() && landing[2] != 0) {
      tc_commit(drain_bar);
      if (!mbar_wait(drain_bar, 0, kDrainWaitNs, nullptr)) report_status(a.status, 5, kSiteBlocksDrain);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int NT, bool SW, bool GATHER, bool SPLIT>
int launch_impl(const BlocksArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, const CUtensorMap* mapB2,
                int split, int num_sms, cudaStream_t s) {
  using C = Cfg<NT, SW, SPLIT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_smem_once(done, blocks_kernel<NT, SW, GATHER, SPLIT>, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  Params p;
  p.a = a;
  p.kblocks = (a.K + BK - 1) / BK;
  p.tiles_n = (a.N + BN - 1) / BN;
  p.split = split;
  const int osz = a.out_bf16 ? 2 : 4;
  p.c_vec = reinterpret_cast<uintptr_t>(a.C) % (4 * osz) == 0 && a.ldc % 4 == 0 ? 1 : 0;
  const long long items = blocks_row_tiles(a.rows, a.offsets != nullptr ? a.experts : 1, NT) * p.tiles_n;
  const long long grid = SPLIT ? items * split : items < num_sms ? items : num_sms;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, blocks_kernel<NT, SW, GATHER, SPLIT>, *mapA, *mapB, SW ? *mapB2 : *mapB, p);
}

template <int NT, bool SW, bool GATHER>
int launch_split(const BlocksArgs& a, const CUtensorMap* mapA, const CUtensorMap* mapB, const CUtensorMap* mapB2,
                 int split, int num_sms, cudaStream_t s) {
  return split > 1 ? launch_impl<NT, SW, GATHER, true>(a, mapA, mapB, mapB2, split, num_sms, s)
                   : launch_impl<NT, SW, GATHER, false>(a, mapA, mapB, mapB2, split, num_sms, s);
}

}  // namespace

int launch_blocks(const BlocksArgs& a, const BlocksPlan& plan, const CUtensorMap* mapA, const CUtensorMap* mapB,
                  const CUtensorMap* mapB2, int num_sms, cudaStream_t s) {
  const int split = plan.split;
  if (a.B2 != nullptr)
    return plan.nt == 32 && a.gather != 0 ? launch_split<32, true, true>(a, mapA, mapB, mapB2, split, num_sms, s)
                                          : cudaErrorInvalidValue;
  if (a.gather != 0) return cudaErrorInvalidValue;
  switch (plan.nt) {
    case 32: return launch_split<32, false, false>(a, mapA, mapB, mapB2, split, num_sms, s);
    case 64: return launch_split<64, false, false>(a, mapA, mapB, mapB2, split, num_sms, s);
    case 128: return launch_split<128, false, false>(a, mapA, mapB, mapB2, split, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace g3

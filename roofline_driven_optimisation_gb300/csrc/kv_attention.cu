// Attention of a sequence's newest tokens over its paged 8-bit cache
// (gemm_kv_attention; the header states the mathematics).
//
// A decode step reads every code of the cache once and does 2 * group * n FLOPs with
// each, so for the usual groups it is bound by HBM.  The fast kernel is built to
// keep enough bytes in flight and to do little else:
//   * the unit of work is a slab, 32 keys of one sequence, head and row tile.  All
//     slabs of the call form one line (sequence, head, row tile, keys); every warp of
//     a persistent grid takes an equal, contiguous piece of it, so ragged batches
//     and a single long sequence fill the GPU alike;
//   * a warp is its own producer and consumer: one lane streams the slab's K and V
//     by TMA (4-D map over the page pool) through the warp's ring of stages, so warps
//     never wait for one another;
//   * S^T = K Q^T and O^T = V^T P^T run on mma.m16n8k16 (fp16 in, fp32 out) with keys
//     and values as the 16-row operand and 8 query rows as the columns: 8-bit codes
//     are exact in fp16, and a decode step's 1 to 8 rows fill the tile.  The operand
//     orders are chosen so that ldmatrix on bytes feeds both products (an inner
//     dimension may be summed in any order, if both operands agree);
//   * a page's scale of K multiplies its scores, that of V its probabilities.  P times
//     that scale enters the second product in fp16, 2^-11 off at most, where the codes are
//     exact already: O's own rounding to bf16 is 2^-8, and results stand 0.0016 to 0.0017
//     from the 64-bit ones (2-norm), as an fp32 product's do.  The sum l is of the
//     unrounded P in fp32;
//   * a slab line's piece ends inside an item at most twice a warp; such partial
//     results (running maximum, sum, unnormalised O) meet in shared memory, and what
//     crosses blocks meets in the workspace, where the last block to arrive adds the
//     parts in an order that is the item's own, so that runs repeat bit for bit.
//
// Measured on one GB300 (6.79 TB/s copied), GPU time:
//   128 sequences of about 8192, 32 over 8 heads of 128, E4M3   2152 MB  351 us  6.1 TB/s
//   16 of about 4096, 32 heads of 128, INT8                      537 MB   94 us  5.7 TB/s
//   1 of 131071, 32 over 8 heads of 128, E4M3                    269 MB   55 us  4.9 TB/s
//   24 of about 1500, 5 tokens, 16 over 4 heads of 64, INT8       19 MB   27 us
//   1 of 777, 32 heads of 128, E4M3                               6.4 MB   12 us
// In the first the slabs stream at 6.8 to 7.2 TB/s; blocks on some groups of SMs end
// their equal shares up to 12 % later than the others, and start and end (planning, the
// first tiles, merging) take about 10 us.  In the last two that is nearly all: planning
// 2 us, the first tile 2 us, merging and the exchange between blocks 2 to 8 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace g3 {
namespace {

// The sequence that row `row` belongs to, and its place among the sequence's n
// new rows; false if no sequence holds it.
__device__ __forceinline__ bool find_row(const KvAttnArgs& a, int row, int& b, int& i, int& n) {
  int first;
  if (a.start == nullptr) {
    b = row;
    i = 0;
    n = 1;
    return row < a.c.seqs;
  }
  int lo = 0, hi = a.c.seqs;   // the last b with start[b] <= row
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.start[mid] <= row) lo = mid;
    else hi = mid;
  }
  b = lo;
  kv_rows(a.start, b, a.tokens, a.max_new, a.status, kSiteKvAttn, first, n);
  i = row - first;
  return i >= 0 && i < n;
}

// Tokens of sequence b in the cache, held to what its table row can address.
__device__ __forceinline__ int kv_length(const KvAttnArgs& a, int b) {
  const int len = a.lengths[b];
  const long long most = (long long)a.c.cols * a.c.P;
  if (len < 0 || len > most) {
    report_status(a.status, 1, kSiteKvAttn);
    return len < 0 ? 0 : (int)most;
  }
  return len;
}

// ------------------------------------------------------------------ generic
// Any head width (to 512), page size and stride: one block for each query row
// and head, keys in chunks of one a thread, the softmax online in fp32.  Bound by the
// latency of its loads, a byte each, and it reads a head's keys once for each of its
// query heads: 16 sequences of 4096, 32 over 8 heads, 80 wide 591 us, 96 wide 722, 256
// wide 2747; 128 wide in pages of 256 tokens 1398 (on the fast kernel, in pages of 64, 31
// to 33).
constexpr int GT = 128;   // threads, and keys in a chunk
constexpr int GD = 512;   // widest head

template <int FMT>
__global__ void __launch_bounds__(GT) kv_attention_generic_kernel(const KvAttnArgs a) {
  __shared__ float q[GD], p[GT], red[GT / 32];
  __shared__ long long at[GT];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int D = a.c.D, row = blockIdx.x, hq = blockIdx.y, h = hq / (a.Hq / a.c.H);
  int b, i, n;
  if (!find_row(a, row, b, i, n)) return;
  // keys this row sees; unsigned, since a chunk may end behind 2^31 - 1
  const unsigned keys = (unsigned)max(0, kv_length(a, b) - n + i + 1), P = (unsigned)a.c.P;
  const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.Q) + (long long)row * a.ldq + (long long)hq * D;
  for (int d = threadIdx.x; d < D; d += GT) q[d] = __bfloat162float(qr[d]);
  float acc[GD / GT] = {};
  float m = -INFINITY, l = 0.f;
  for (unsigned j0 = 0; j0 < keys; j0 += GT) {
    const unsigned j = j0 + threadIdx.x;
    float s = -INFINITY, vs = 0.f;
    long long off = -1;
    __syncthreads();   // q is written; the previous chunk's readers are done
    if (j < keys) {
      const int g = kv_page(a.c, b, (int)(j / P), a.status, kSiteKvAttn);
      if (g >= 0) {
        off = (long long)g * a.c.ps + (long long)h * a.c.hs + (long long)(j % P) * a.c.ts;
        const uint8_t* kc = a.c.k + off;
        float dot = 0.f;
        for (int d = 0; d < D; ++d) dot = fmaf(q[d], kv_value2<FMT>(kc[d]).x, dot);
        s = dot * a.c.ks[(long long)g * a.c.H + h] * a.scale;
        vs = a.c.vs[(long long)g * a.c.H + h];
      }
    }
    at[threadIdx.x] = off;
    float mx = s;
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = mx;
    __syncthreads();
    mx = m;
    for (int w = 0; w < GT / 32; ++w) mx = fmaxf(mx, red[w]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    const float e = off >= 0 ? expf(s - mu) : 0.f, alpha = expf(m - mu);
    m = mx;
    p[threadIdx.x] = e * vs;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();   // red has been read
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = sum;
    __syncthreads();
    l *= alpha;
    for (int w = 0; w < GT / 32; ++w) l += red[w];
#pragma unroll
    for (int c = 0; c < GD / GT; ++c) {
      const int d = c * GT + threadIdx.x;
      if (d >= D) break;
      float x = acc[c] * alpha;
      for (int t = 0; t < (int)min((unsigned)GT, keys - j0); ++t)
        if (at[t] >= 0) x = fmaf(p[t], kv_value2<FMT>(a.c.v[at[t] + d]).x, x);
      acc[c] = x;
    }
  }
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.O) + (long long)row * a.ldo + (long long)hq * D;
#pragma unroll
  for (int c = 0; c < GD / GT; ++c) {
    const int d = c * GT + threadIdx.x;
    // l == 0: no key was seen; a NaN sum must come out as NaN
    if (d < D) out[d] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[c] / l);
  }
}


// ------------------------------------------------------------------ fast
using u64 = unsigned long long;
constexpr int NW = 8;                    // warps of a block, one block an SM
constexpr int SLAB = kKvSlab;
constexpr int MAX_CTAS = 160;            // blocks that the workspace has room for
constexpr int MAX_ROWS = 32;             // rows of a tile, at most
constexpr int MAX_TW = 4;                // warps that share a slab's keys, a tile of rows each
constexpr int RING = 3 * 2 * SLAB * 128; // bytes of a warp's ring
constexpr int PV_EXP = 14;               // P times the page's scale is below 2^PV_EXP in fp16
constexpr int MIN_EXP = -112;
constexpr int WHOLE_EXTRA = 6;          // see its use

template <int D, int NT>
struct Cfg {
  static constexpr int TILE = SLAB * D;              // bytes of a slab's keys
  static constexpr int STAGE = 2 * TILE;
  // 24 and 32 rows of 128 values do not fit the registers beside their sums: such
  // queries lie in the last third of the ring, in the order in which lanes read them
  static constexpr bool Q_SHARED = D == 128 && NT > 2;
  static constexpr int Q_BYTES = Q_SHARED ? D / 16 * NT * 32 * 8 : 0;
  static constexpr int STAGES = (RING - (Q_SHARED ? RING / 3 : 0)) / STAGE;   // 3 or 2 (D 128), 6
  static_assert(STAGES * STAGE + Q_BYTES <= RING, "ring");
};

// A partial result: O [rows][D], then m [rows], l [rows].  In the workspace: two of
// every block and tile (its first and last item may go on in other blocks), one of every
// warp (its first item's, while its ring is in use), then a counter for each item.
// The parts' places are of fixed size, so that no call's parts reach another's
// counters.
constexpr int PART_FLOATS = MAX_ROWS * 128 + 2 * MAX_ROWS;
static_assert(PART_FLOATS * 4 <= RING, "a partial result fits in a drained ring");
constexpr size_t PARTS = (size_t)MAX_CTAS * (2 * MAX_TW + NW);
constexpr int MAX_OPENS = NW + MAX_TW;   // a tile's warps meet at one more place than they are

struct StageMeta {
  float ks[2], vs[2];   // scales of the slab's one or two pages
  int ok[2];            // whether the page could be placed
  int pad[2];
};

struct Slot {           // a warp's partial result
  u64 unit;             // first unit of its item (~0: none)
  float* part;          // in shared memory or in the workspace
  int S, rows, h, t, first;   // the item's slabs and rows, head, tile, first row of its sequence
  long long count;      // index of its counter (max_new, so tiles, may be far above what is there)
};

struct Open {           // an item that more than one warp worked on
  u64 unit;
  int e0, e1;           // its parts: slots e0 .. e1 (warp * 2 + slot)
  int S, rows, h, t, first;
  int tl;               // the tile's place in its pass
  long long count;
  bool whole;           // no other block has a part of it
};

struct SeqRec {         // a sequence on the line: units and items before it
  u64 at;
  int items, len, first, n;
};
static_assert(kKvMaxSeqs * sizeof(SeqRec) <= NW * RING, "the records fit in the rings");

struct Shared {
  StageMeta meta[NW][6];
  u64 full[NW][6];
  Slot slot[NW * 2];
  Open open[MAX_OPENS];
  int opens;
  u64 scan[NW];
  int scan_items[NW], scan_longest[NW];
  int last[MAX_OPENS];  // this block finishes the item
  int blocks[MAX_OPENS];   // that have a part of it
  int abort;
};

// Units of sequence b: heads * passes * slabs; a pass is the tiles that the warps of
// a group take side by side
struct Seq {
  int len, first, n, S, tiles, passes;
};

// Slabs of a sequence of len keys; one, of which no row sees a key, where it has none
__device__ __forceinline__ int slabs(int len) { return max(1, (int)(((unsigned)len + SLAB - 1) / SLAB)); }

struct Plan {
  const KvAttnArgs* a;
  int group, rt;        // query heads of a head; rows of a tile
  int tw_log, tl;       // log2 of a group's warps; this warp's place in it
  __device__ __forceinline__ Seq seq(int len, int first, int n) const {
    const int tiles = (n * group + rt - 1) / rt;
    return Seq{len, first, n, slabs(len), tiles, (tiles + (1 << tw_log) - 1) >> tw_log};
  }
  __device__ __forceinline__ Seq seq(int b) const {
    // every load before the first check, which waits for it
    int len = __ldg(a->lengths + b), first = b, end = b + 1;
    if (a->start != nullptr) {
      first = __ldg(a->start + b);
      end = __ldg(a->start + b + 1);
    }
    const long long most = (long long)a->c.cols * a->c.P;
    if (len < 0 || len > most) {
      report_status(a->status, 1, kSiteKvAttn);
      len = len < 0 ? 0 : (int)most;
    }
    if (first < 0 || end < first || end > a->tokens || end - first > a->max_new) {
      report_status(a->status, 1, kSiteKvAttn);
      first = end = 0;
    }
    return seq(len, first, end - first);
  }
  __device__ __forceinline__ u64 units(const Seq& q) const { return (u64)a->c.H * q.passes * q.S; }
  // keys that the last row of tile t sees (none if there is no such tile)
  __device__ __forceinline__ int visible(const Seq& q, int t) const {
    if (t >= q.tiles) return 0;
    if ((t + 1) * rt >= q.n * group) return q.len;
    return q.len - q.n + ((t + 1) * rt - 1) / group + 1;
  }
};

// x / d, by the 32-bit division wherever both fit
__device__ __forceinline__ u64 quotient(u64 x, u64 d) {
  return (x | d) >> 32 ? x / d : (u64)((unsigned)x / (unsigned)d);
}

// A place on the line of slabs
struct Walk {
  int b, idx, s;        // sequence, head * passes + pass, slab
  int h, t, vis;        // head, tile, keys that the tile's last row sees
  Seq q;
  __device__ __forceinline__ void split(const Plan& p) {
    h = q.passes == 1 ? idx : idx / q.passes;
    t = ((idx - h * q.passes) << p.tw_log) + p.tl;
    vis = p.visible(q, t);
  }
  __device__ __forceinline__ void next(const Plan& p) {
    if (++s < q.S) return;
    s = 0;
    if (++idx < p.a->c.H * q.passes) {
      split(p);
      return;
    }
    idx = 0;
    do {
      if (++b >= p.a->c.seqs) return;
      q = p.seq(b);
    } while (q.passes == 0);
    split(p);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }   // -126 <= e <= 127

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes of a register as fp16 pairs.  INT8: the byte plus 128 under the high
// byte of fp16's 1024 is 1024 + 128 + code; subtracting 1152 is exact.
__device__ __forceinline__ uint32_t sub_1152(uint32_t x) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// (bytes 0,1), (bytes 2,3)
template <int FMT>
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kKvE4M3) {
    lo = e4m3x2_to_f16x2(x & 0xffffu);
    hi = e4m3x2_to_f16x2(x >> 16);
  } else {
    x ^= 0x80808080u;
    lo = sub_1152(__byte_perm(x, 0x64646464u, 0x4140));
    hi = sub_1152(__byte_perm(x, 0x64646464u, 0x4342));
  }
}
// (bytes 0,2), (bytes 1,3)
template <int FMT>
__device__ __forceinline__ void widen_pairs(uint32_t x, uint32_t& even, uint32_t& odd) {
  if constexpr (FMT == kKvE4M3) {
    widen<FMT>(__byte_perm(x, 0u, 0x3120), even, odd);
  } else {
    x ^= 0x80808080u;
    even = sub_1152(__byte_perm(x, 0x64646464u, 0x4240));
    odd = sub_1152(__byte_perm(x, 0x64646464u, 0x4341));
  }
}

// fp16 pair mask of keys k0, k0 + 1 below lim
__device__ __forceinline__ uint32_t key_mask(int k0, int lim) {
  return (k0 < lim ? 0xffffu : 0u) | (k0 + 1 < lim ? 0xffff0000u : 0u);
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(NW * 32, 1)
    kv_attention_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ KvAttnArgs a, const int group, const long long max_tiles,
                        const int tw, const int vec) {
  using C = Cfg<D, NT>;
  constexpr int ST = C::STAGES, CH = D / 16, RT = NT * 8;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* base_ptr = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t4 = lane % 4;
  uint8_t* ring_ptr = base_ptr + warp * RING;
  const uint32_t ring = smem_u32(ring_ptr);
  // groups of tw warps walk the same slabs, each for its own tile of rows: what one
  // fetches, the others find in L2.  All are powers of two: the plan's divisions by them
  // in 64 bits took 0.4 us of a call.
  static_assert((NW & (NW - 1)) == 0, "a power of two");
  const int tw_log = 31 - __clz(tw), tl = warp & (tw - 1), worker = warp >> tw_log, workers = NW >> tw_log;
  const int workers_log = 31 - __clz(workers);
  const Plan plan{&a, group, RT, tw_log, tl};
  const int npg = a.c.P < SLAB ? 2 : 1;           // pages of a slab
  const int p_shift = 31 - __clz(a.c.P);          // P is a power of two

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
    for (int w = 0; w < NW; ++w)
      for (int s = 0; s < ST; ++s) mbar_init(smem_u32(&sh.full[w][s]), 2 * npg);
    sh.abort = 0;
    fence_mbar_init();
  }
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();

  // ---- the line of slabs: every sequence's place on it, in the rings' memory
  SeqRec* rec = reinterpret_cast<SeqRec*>(base_ptr);
  const int per = (a.c.seqs + NW * 32 - 1) / (NW * 32);
  const int b_lo = min(a.c.seqs, (int)threadIdx.x * per), b_hi = min(a.c.seqs, b_lo + per);
  u64 mine = 0;
  int items = 0, longest = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq q = plan.seq(b);
    rec[b].at = mine;
    rec[b].items = items;
    rec[b].len = q.len;
    rec[b].first = q.first;
    rec[b].n = q.n;
    mine += plan.units(q);
    items += a.c.H * q.passes;
    if (q.passes > 0) longest = max(longest, q.S);
  }
  u64 incl = mine;
  int item_incl = items;
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
    const int z = __shfl_up_sync(0xffffffffu, item_incl, o);
    if (lane >= o) {
      incl += y;
      item_incl += z;
    }
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    sh.scan[warp] = incl;
    sh.scan_items[warp] = item_incl;
    sh.scan_longest[warp] = longest;
  }
  __syncthreads();
  u64 at = incl - mine, T = 0;
  int item_at = item_incl - items, I = 0;
  for (int w = 0; w < NW; ++w) {
    if (w < warp) {
      at += sh.scan[w];
      item_at += sh.scan_items[w];
    }
    T += sh.scan[w];
    I += sh.scan_items[w];
    longest = max(longest, sh.scan_longest[w]);
  }
  for (int b = b_lo; b < b_hi; ++b) {
    rec[b].at += at;
    rec[b].items += item_at;
  }
  __syncthreads();
  // Blocks take equal shares of the line, or whole items.  Whole items need no exchange
  // between blocks, which costs a call about as much time as WHOLE_EXTRA slabs a warp;
  // so they are taken unless the fullest block's warps get longer than that.  Measured,
  // whole items and shares: 1 x 777 of 32 heads (25 slabs an item) 11.8 and 13.4 us,
  // 60 x 200 of 8 heads 14.6 and 17.6, 32 x 600 of 8 heads 21.9 and 24.9; 1 x 2000 of 8
  // heads (63 slabs) 18.3 and 14.0, 1 x 4000 28.4 and 12.4.
  const u64 share = quotient(T + gridDim.x * workers - 1, gridDim.x * workers);
  const int blocks = min((int)gridDim.x, I);
  const bool by_item = I > 0 && (((u64)((I + blocks - 1) / blocks) * longest + workers - 1) >> workers_log) <= share + WHOLE_EXTRA;
  const u64 G = by_item ? (u64)blocks : T < gridDim.x ? T : gridDim.x;   // every block up to G has a unit
  const u64 cta = blockIdx.x;
  if (cta >= G) return;
  auto record = [&](auto before) {                // the last sequence for which before() holds
    int lo = 0, hi = a.c.seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before(rec[mid])) lo = mid;
      else hi = mid;
    }
    return lo;
  };
  auto item_unit = [&](u64 i) -> u64 {            // first unit of item i
    if (i >= (u64)I) return T;
    const SeqRec& q = rec[record([&](const SeqRec& x) { return x.items <= (int)i; })];
    return q.at + (i - q.items) * (u64)slabs(q.len);
  };
  const u64 A = by_item ? item_unit(quotient(cta * I, G)) : quotient(cta * T, G);
  const u64 B = by_item ? item_unit(quotient((cta + 1) * I, G)) : quotient((cta + 1) * T, G);
  const u64 me = cta * NW + warp;
  const u64 u0 = A + (worker * (B - A) >> workers_log), u1 = A + ((worker + 1) * (B - A) >> workers_log);
  Walk cw;
  if (u0 < u1) {
    cw.b = record([&](const SeqRec& x) { return x.at <= u0; });
    const SeqRec& x = rec[cw.b];
    cw.q = plan.seq(x.len, x.first, x.n);
    const u64 rel = u0 - x.at;
    cw.idx = (int)quotient(rel, cw.q.S);
    cw.s = (int)(rel - (u64)cw.idx * cw.q.S);
    cw.split(plan);
  }
  __syncthreads();                                // the records' memory becomes the rings
  fence_proxy_async_smem();

  // ---- producer side
  const int total = (int)(u1 - u0);
  // the table's entry for the part of a slab that this lane fetches, -1 where no row
  // sees it.  Only loaded here: the check waits for the value, so it comes with the
  // copy, a slab later.
  auto page_of = [&](const Walk& w) -> int {
    const int key = w.s * SLAB + lane * 16;
    if (lane >= npg || key >= w.vis) return -1;
    return __ldg(a.c.table + (long long)w.b * a.c.tstride + (key >> p_shift));
  };
  auto issue = [&](int st, const Walk& w, int p) {
    if (lane < npg) {
      const uint32_t bar = smem_u32(&sh.full[warp][st]);
      StageMeta& m = sh.meta[warp][st];
      const int key = w.s * SLAB + lane * 16, rows = SLAB / npg;
      const bool ok = p >= 0 && p < a.c.pages;
      if (!ok && key < w.vis) report_status(a.status, 1, kSiteKvAttn);
      m.ok[lane] = ok;
      if (ok) {
        const uint32_t dst = ring + st * C::STAGE + lane * 16 * D;
        mbar_arrive_expect_tx(bar, 2 * rows * D);
        tma_load_4d(dst, &mapK, bar, 0, key & (a.c.P - 1), w.h, p);
        tma_load_4d(dst + C::TILE, &mapV, bar, 0, key & (a.c.P - 1), w.h, p);
        cp_async_4(smem_u32(&m.ks[lane]), a.c.ks + (long long)p * a.c.H + w.h);
        cp_async_4(smem_u32(&m.vs[lane]), a.c.vs + (long long)p * a.c.H + w.h);
      } else {
        m.ks[lane] = m.vs[lane] = 0.f;
        mbar_arrive(bar);
      }
      cp_async_arrive(bar);
    }
  };

  const int slot0 = (tl * workers + worker) * 2;    // a tile's warps side by side, in the order of the line
  if (lane < 2) sh.slot[slot0 + lane].unit = ~0ull;
  if (total > 0) {
    Walk pw = cw;                                 // next slab to fetch
    int issued = 0, pg;
    {
      Walk ws[ST];
      int ps[ST];
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        ws[i] = pw;
        ps[i] = i < total ? page_of(pw) : -1;
        if (i < total) pw.next(plan);
      }
#pragma unroll
      for (int i = 0; i < ST; ++i)
        if (i < total) issue(i, ws[i], ps[i]);
      issued = min(ST, total);
      pg = issued < total ? page_of(pw) : -1;
    }

    // ---- consumer state of one item
    uint32_t qf[C::Q_SHARED ? 1 : NT][CH][2];
    uint2* const q_shared = reinterpret_cast<uint2*>(ring_ptr + ST * C::STAGE) + lane;   // [(chunk * NT + nt) * 32]
    float acc[NT][CH][4];
    float m[NT][2], l[NT][2], rs[NT][2];
    int lim[NT][2];                               // keys that this lane's columns see
    int ev = MIN_EXP;                             // V's pages so far have scales below 2^ev
    int lim_min = 0, lim_max = 0;
    bool head = false;                            // the item began before this warp's piece

    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int j = 0; j < total; ++j) {
      const Seq& q = cw.q;
      if (j == 0 || cw.s == 0) {
        // ---- a new item: its query rows, scaled to fp16 by a power of two a row
        head = cw.s != 0;
        const int rows = min(RT, q.n * group - cw.t * RT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = nt * 8 + g, rr = cw.t * RT + r;
          float x[CH][4];
          float mx = 0.f;
          const bool have = r < rows;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) +
                                     (have ? (long long)(q.first + rr / group) * a.ldq +
                                                 (long long)(cw.h * group + rr % group) * D : 0);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            uint2 v = make_uint2(0u, 0u);
            if (have) {
              if (vec) {
                v = *reinterpret_cast<const uint2*>(src + c * 16 + t4 * 4);
              } else {
                const uint16_t* e = reinterpret_cast<const uint16_t*>(src + c * 16 + t4 * 4);
                v = make_uint2(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16));
              }
            }
            x[c][0] = __uint_as_float(v.x << 16);
            x[c][1] = __uint_as_float(v.x & 0xffff0000u);
            x[c][2] = __uint_as_float(v.y << 16);
            x[c][3] = __uint_as_float(v.y & 0xffff0000u);
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fabsf(x[c][k]));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // the largest magnitude of the row lands in [2^14, 2^15)
          const int e = max(-112, (int)(__float_as_uint(mx) >> 23) - 127);
          const float f = pow2i(14 - e);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const uint32_t lo = pack_f16(x[c][0] * f, x[c][1] * f), hi = pack_f16(x[c][2] * f, x[c][3] * f);
            if constexpr (C::Q_SHARED) {
              q_shared[(c * NT + nt) * 32] = make_uint2(lo, hi);
            } else {
              qf[nt][c][0] = lo;
              qf[nt][c][1] = hi;
            }
          }
          const float back = a.scale * 1.4426950408889634f * pow2i(e - 14);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            rs[nt][k] = __shfl_sync(0xffffffffu, back, (2 * t4 + k) * 4);
            const int col = cw.t * RT + nt * 8 + 2 * t4 + k;
            lim[nt][k] = q.len - q.n + min(col / group, q.n - 1) + 1;
            m[nt][k] = -INFINITY;
            l[nt][k] = 0.f;
          }
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[nt][c][k] = 0.f;
        }
        ev = MIN_EXP;
        lim_min = q.len - q.n + cw.t * RT / group + 1;
        lim_max = cw.vis;
      }

      // ---- the slab
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.full[warp][st]), phase, a.timeout_ns, &sh.abort));
      if (!ok) break;
      const int k0 = cw.s * SLAB;
      const StageMeta& meta = sh.meta[warp][st];
      const int ok0 = meta.ok[0], ok1 = npg == 2 ? meta.ok[1] : ok0;
      if (k0 < lim_max && (ok0 | ok1)) {
        const uint32_t kt = ring + st * C::STAGE, vt = kt + C::TILE;
        float ks[2], vs[2];
        ks[0] = meta.ks[0];
        vs[0] = meta.vs[0];
        ks[1] = npg == 2 ? meta.ks[1] : ks[0];
        vs[1] = npg == 2 ? meta.vs[1] : vs[0];
        // every key of the slab is there for every row
        const bool whole = lim_min - SLAB >= k0 && (ok0 & ok1);   // the slab may end at 2^31

        // S^T = K Q^T.  ldmatrix gives lane (g, t4) bytes 4*t4 .. 4*t4+3 of row g of
        // each 16-byte chunk: the first two are the operand's k = 2*t4, 2*t4+1, the
        // others its k + 8; Q is held in the same order.
        float sc[2][NT][4];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[sub][nt][k] = 0.f;
        const int row = lane & 15, sw = D == 128 ? (row & 7) : ((row >> 1) & 3);   // rows 16 apart swizzle alike
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          uint32_t q[2][NT][2];
#pragma unroll
          for (int cc = 0; cc < 2; ++cc)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (C::Q_SHARED) {
                const uint2 v = q_shared[((c + cc) * NT + nt) * 32];
                q[cc][nt][0] = v.x;
                q[cc][nt][1] = v.y;
              } else {
                q[cc][nt][0] = qf[nt][c + cc][0];
                q[cc][nt][1] = qf[nt][c + cc][1];
              }
            }
          const uint32_t at = kt + row * D + (((c + (lane >> 4)) ^ sw) << 4);
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            uint32_t x[4], a0, a1, a2, a3;
            ldsm_x4(at + sub * 16 * D, x);
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              widen<FMT>(x[2 * cc], a0, a2);
              widen<FMT>(x[2 * cc + 1], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(sc[sub][nt], a0, a1, a2, a3, q[cc][nt][0], q[cc][nt][1]);
            }
          }
        }

        // V's scale enters through P; the accumulators' unit is 2^(ev - PV_EXP)
        const int e_new = max(ev, (int)((__float_as_uint(fmaxf(fabsf(vs[0]), fabsf(vs[1]))) >> 23) & 255u) - 126);
        const float grow = pow2i(max(ev - e_new, -126));
        const bool grew = e_new > ev;
        ev = e_new;
        const float unit = pow2i(PV_EXP - ev);
        const float cv[2] = {vs[0] * unit, vs[1] * unit};

        uint32_t pf[2][NT][2];
        float al[NT][2];
        bool rescale = grew;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float x = sc[sub][nt][k] * (rs[nt][k & 1] * ks[sub]);
              if (!whole) {
                const int key = k0 + sub * 16 + g + (k >> 1) * 8;
                if (key >= lim[nt][k & 1] || !(sub ? ok1 : ok0)) x = -INFINITY;
              }
              sc[sub][nt][k] = x;
              mx[k & 1] = fmaxf(mx[k & 1], x);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = mx[k];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float mn = fmaxf(m[nt][k], v), mu = mn == -INFINITY ? 0.f : mn;
            al[nt][k] = ex2(m[nt][k] - mu);
            rescale |= mn != m[nt][k];
            m[nt][k] = mn;
            float sum = 0.f;
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const float p = ex2(sc[sub][nt][hh * 2 + k] - mu);
                sc[sub][nt][hh * 2 + k] = p;
                sum += p;
              }
            l[nt][k] = l[nt][k] * al[nt][k] + sum;
          }
          // P^T as the second operand: transpose 8 x 8 blocks (keys x rows)
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              pf[sub][nt][hh] =
                  movm_t(pack_f16(sc[sub][nt][2 * hh] * cv[sub], sc[sub][nt][2 * hh + 1] * cv[sub]));
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float f0 = al[nt][0] * grow, f1 = al[nt][1] * grow;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              acc[nt][c][0] *= f0;
              acc[nt][c][1] *= f1;
              acc[nt][c][2] *= f0;
              acc[nt][c][3] *= f1;
            }
          }
        }

        // O^T += V^T P^T.  Transposed ldmatrix of byte pairs: lane (g, t4) has values
        // 2g, 2g+1 of keys 2*t4, 2*t4+1; row g of the operand is value 2g, row g + 8
        // value 2g + 1.
        auto products = [&](auto masked, int limit, bool all) {
#pragma unroll
          for (int c = 0; c < CH; c += 2) {
            const uint32_t at = vt + row * D + (((c + (lane >> 4)) ^ sw) << 4);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
              const int kk = k0 + sub * 16 + 2 * t4;
              const bool there = (sub ? ok1 : ok0) != 0;
              const uint32_t mk0 = there ? key_mask(kk, limit) : 0u, mk1 = there ? key_mask(kk + 8, limit) : 0u;
              uint32_t x[4], a0, a1, a2, a3;
              ldsm_x4_t(at + sub * 16 * D, x);
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                widen_pairs<FMT>(x[2 * cc], a0, a1);
                widen_pairs<FMT>(x[2 * cc + 1], a2, a3);
                if constexpr (decltype(masked)::value) {
                  a0 &= mk0;
                  a1 &= mk0;
                  a2 &= mk1;
                  a3 &= mk1;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if constexpr (!decltype(masked)::value) {
                    mma16816(acc[nt][c + cc], a0, a1, a2, a3, pf[sub][nt][0], pf[sub][nt][1]);
                  } else {
                    float y[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816(y, a0, a1, a2, a3, pf[sub][nt][0], pf[sub][nt][1]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[nt][c + cc][k] += all || lim[nt][k & 1] == limit ? y[k] : 0.f;
                  }
                }
              }
            }
          }
        };
        // any INT8 code is finite, so a probability of 0 hides what a row does not see
        if (whole || FMT == kKvInt8) {
          products(std::false_type{}, 0, true);
        } else {
          // A probability of 0 does not hide a NaN.  Keys that no row sees are cut out
          // of V itself; if one that only some rows see holds a NaN, V is cut for each
          // query in turn, and only that query's rows take the product.
          bool nan = false;
          {
            for (int r = max(lim_min - k0, 0); r < min(lim_max - k0, SLAB); ++r)
              if (lane < D / 4) {
                uint32_t x;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(vt + r * D + lane * 4) : "memory");
                nan |= (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
              }
            nan = __any_sync(0xffffffffu, nan);
          }
          const int q_lo = cw.t * RT / group, q_hi = (min(q.n * group, (cw.t + 1) * RT) - 1) / group;
          for (int i = nan ? q_lo : q_hi; i <= q_hi; ++i) {
            const int limit = q.len - q.n + i + 1;
            if (limit > k0) products(std::true_type{}, limit, !nan);
          }
        }
      }
      // ---- the stage is free: fetch ahead
      __syncwarp();
      const Walk done = cw;
      if (issued < total) {
        issue(st, pw, pg);
        if (++issued < total) {
          pw.next(plan);
          pg = page_of(pw);
        }
      }
      if (++st == ST) {
        st = 0;
        phase ^= 1u;
      }
      // ---- the item ends here, or this warp's piece of it
      const bool ends = done.s + 1 == done.q.S;
      if (ends || j + 1 == total) {
        const int rows = min(RT, done.q.n * group - done.t * RT);
        const float unit = pow2i(max(ev - PV_EXP, -126));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float v = l[nt][k];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            l[nt][k] = v;
          }
        if (ends && !head) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int r = nt * 8 + 2 * t4 + k, rr = done.t * RT + r;
              if (r >= rows) continue;
              const float inv = l[nt][k] == 0.f ? 0.f : unit / l[nt][k];
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.O) + (long long)(done.q.first + rr / group) * a.ldo +
                                 (long long)(done.h * group + rr % group) * D + 2 * g;
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                const float lo = acc[nt][c][k] * inv, hi = acc[nt][c][2 + k] * inv;
                if (vec) {
                  *reinterpret_cast<__nv_bfloat162*>(o + c * 16) = __floats2bfloat162_rn(lo, hi);
                } else {
                  o[c * 16] = __float2bfloat16_rn(lo);
                  o[c * 16 + 1] = __float2bfloat16_rn(hi);
                }
              }
            }
        } else if (rows > 0) {
          // into the drained ring, or into the workspace while the ring is in use
          float* part = j + 1 == total
                            ? reinterpret_cast<float*>(ring_ptr)
                            : static_cast<float*>(a.ws) + (MAX_CTAS * 2 * MAX_TW + me) * (size_t)PART_FLOATS;
          if (lane == 0) {
            Slot& s = sh.slot[slot0 + (head ? 0 : 1)];
            s.unit = u0 + j - done.s;
            s.part = part;
            s.S = done.q.S;
            s.rows = rows;
            s.h = done.h;
            s.t = done.t;
            s.first = done.q.first;
            s.count = ((long long)done.b * a.c.H + done.h) * max_tiles + done.t;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int r = nt * 8 + 2 * t4 + k;
              if (r >= rows) continue;
#pragma unroll
              for (int c = 0; c < CH; ++c)
                *reinterpret_cast<float2*>(part + r * D + c * 16 + 2 * g) =
                    make_float2(acc[nt][c][k] * unit, acc[nt][c][2 + k] * unit);
              if (g == 0) {
                part[RT * D + r] = m[nt][k];
                part[RT * D + RT + r] = l[nt][k];
              }
            }
        }
      }
      if (j + 1 < total) cw.next(plan);
    }
    if (!ok) {
      // a copy did not arrive: leave, but not before the copies in flight have landed
      if (lane == 0) report_status(a.status, 5, kSiteKvAttnLoad);
      sh.abort = 1;
      for (int i = 0; i < ST; ++i)
        if (lane == 0) mbar_wait(smem_u32(&sh.full[warp][i]), i < st ? phase ^ 1u : phase, kDrainWaitNs / 8, nullptr);
    }
  }

  // ---- parts of items that more than one warp worked on
  __syncthreads();
  if (sh.abort) return;
  if (warp == 0) {
    // a lane for each slot: an item's first slot makes its entry
    const u64 unit = lane < NW * 2 ? sh.slot[lane].unit : ~0ull;
    const unsigned valid = __ballot_sync(0xffffffffu, unit != ~0ull);
    const unsigned below = valid & ((1u << lane) - 1u);
    const int prev = below ? 31 - __clz(below) : lane;
    const u64 before = __shfl_sync(0xffffffffu, unit, prev);
    const int tile = lane >> (workers_log + 1), tile_before = prev >> (workers_log + 1);
    const bool starts = unit != ~0ull && (below == 0 || before != unit || tile != tile_before);
    const unsigned firsts = __ballot_sync(0xffffffffu, starts);
    if (starts) {
      const Slot& s = sh.slot[lane];
      Open& o = sh.open[__popc(firsts & ((1u << lane) - 1u))];
      const unsigned later = lane < 31 ? firsts & ~((2u << lane) - 1u) : 0u;
      const unsigned own = later ? valid & ((1u << (__ffs(later) - 1)) - 1u) : valid;   // slots before the next item's
      o.unit = unit;
      o.e0 = lane;
      o.e1 = 31 - __clz(own);
      o.S = s.S;
      o.rows = s.rows;
      o.h = s.h;
      o.t = s.t;
      o.first = s.first;
      o.count = s.count;
      o.tl = tile;
      o.whole = unit >= A && unit + s.S <= B;
    }
    if (lane == 0) sh.opens = __popc(firsts);
  }
  __syncthreads();
  float* parts = static_cast<float*>(a.ws);
  int* counters = reinterpret_cast<int*>(parts + PARTS * PART_FLOATS);
  auto store = [&](const Open& o, int r, int d4, float4 x, float sum) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int rr = o.t * RT + r;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.O) + (long long)(o.first + rr / group) * a.ldo +
                         (long long)(o.h * group + rr % group) * D + d4 * 4;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * inv, x.y * inv), hi = __floats2bfloat162_rn(x.z * inv, x.w * inv);
    if (vec) {
      reinterpret_cast<__nv_bfloat162*>(out)[0] = lo;
      reinterpret_cast<__nv_bfloat162*>(out)[1] = hi;
    } else {
      out[0] = lo.x;
      out[1] = lo.y;
      out[2] = hi.x;
      out[3] = hi.y;
    }
  };
  auto add = [](float4& x, float w, const float4& y) {
    x.x = fmaf(w, y.x, x.x);
    x.y = fmaf(w, y.y, x.y);
    x.z = fmaf(w, y.z, x.z);
    x.w = fmaf(w, y.w, x.w);
  };
  const int opens = sh.opens;
  // weights of every slot for every row, behind the part in the first ring
  float* wt = reinterpret_cast<float*>(base_ptr + PART_FLOATS * 4);   // [slot][row]
  float* tops = wt + NW * 2 * MAX_ROWS;                               // [item][row]: maximum
  float* totals = tops + MAX_OPENS * MAX_ROWS;                        // [item][row]: sum
  static_assert((PART_FLOATS + (2 * NW + 2 * MAX_OPENS) * MAX_ROWS) * 4 <= RING, "weights fit behind a part");
  int rmax = 0;
  for (int i = 0; i < opens; ++i) rmax = max(rmax, sh.open[i].rows);
  for (int i = threadIdx.x / 16; i < (opens * rmax + 1) / 2 * 2; i += NW * 2) {
    // half a warp a row, a lane a slot
    const int j = min(i / rmax, opens - 1), r = i - j * rmax, e = lane % 16;
    const Open& o = sh.open[j];
    const Slot& s = sh.slot[e];
    const bool mine = r < o.rows && e >= o.e0 && e <= o.e1 && s.unit == o.unit;
    const float top = mine ? s.part[RT * D + r] : -INFINITY, l = mine ? s.part[RT * D + RT + r] : 0.f;
    float M = top;
    for (int k = 8; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    const float w = mine ? ex2(top - (M == -INFINITY ? 0.f : M)) : 0.f;
    float sum = mine ? w * l : 0.f;
    for (int k = 8; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (mine) wt[e * MAX_ROWS + r] = w;
    if (e == 0 && r < o.rows) {
      tops[j * MAX_ROWS + r] = M;
      totals[j * MAX_ROWS + r] = sum;
    }
  }
  __syncthreads();
  // A warp takes some rows of an item: a lane holds a quad of each of U rows (of U
  // pairs of rows where a row is half a warp wide), whose loads are in flight together.
  constexpr int QUADS = D / 4, RPW = 32 / QUADS;
  const int lane_row = lane / QUADS, lane_quad = lane % QUADS;
  auto merge = [&](auto batch) {
    constexpr int U = decltype(batch)::value;
    const int groups = (rmax + U * RPW - 1) / (U * RPW);
    for (int i = warp; i < opens * groups; i += NW) {
      const int j = i / groups, r0 = (i - j * groups) * U * RPW + lane_row;
      const Open& o = sh.open[j];
      float4 x[U] = {};
      for (int e = o.e0; e <= o.e1; ++e) {
        if (sh.slot[e].unit != o.unit) continue;
        const float* p = sh.slot[e].part + r0 * D + lane_quad * 4;
        const float* w = wt + e * MAX_ROWS + r0;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r0 + u * RPW < o.rows) add(x[u], w[u * RPW], *reinterpret_cast<const float4*>(p + u * RPW * D));
      }
      float* p = parts + ((cta * 2 + (o.unit < A ? 0 : 1)) * MAX_TW + o.tl) * PART_FLOATS;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * RPW;
        if (r >= o.rows) continue;
        if (o.whole) {
          store(o, r, lane_quad, x[u], totals[j * MAX_ROWS + r]);
        } else {
          *reinterpret_cast<float4*>(p + r * D + lane_quad * 4) = x[u];
          if (lane_quad == 0) {
            p[RT * D + r] = tops[j * MAX_ROWS + r];
            p[RT * D + RT + r] = totals[j * MAX_ROWS + r];
          }
        }
      }
    }
  };
  if (opens * rmax <= 2 * NW) merge(std::integral_constant<int, 1>{});
  else merge(std::integral_constant<int, 4>{});
  // ---- and more than one block: the last to arrive adds the blocks' parts in order
  bool any = false;
  for (int i = 0; i < opens; ++i) any |= !sh.open[i].whole;
  if (!any) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x < opens) {
    const Open& o = sh.open[threadIdx.x];
    int last = 0;
    if (!o.whole) {
      const int c0 = (int)quotient((o.unit + 1) * G - 1, T), c1 = (int)quotient((o.unit + o.S) * G - 1, T);
      last = atomicAdd(counters + o.count, 1) == c1 - c0;
      sh.blocks[threadIdx.x] = c1 - c0 + 1;
      if (last) counters[o.count] = 0;             // ready for the next call
    }
    sh.last[threadIdx.x] = last;
  }
  __syncthreads();
  // every part's weight for every row of the items that fall to this block, in the
  // drained rings: [item's rows][its parts], as many items at a time as fit
  constexpr int ROOM = (NW * RING / 4 - MAX_OPENS * MAX_ROWS - NW * 32 * 4) / 2;
  static_assert(MAX_ROWS * MAX_CTAS <= ROOM, "one item always fits");
  float* weight = reinterpret_cast<float*>(base_ptr);
  float* part_sum = weight + ROOM;
  float* item_sum = part_sum + ROOM;                 // [item][row]
  float4* shared_sum = reinterpret_cast<float4*>(item_sum + MAX_OPENS * MAX_ROWS);   // [thread]
  static_assert(ROOM % 2 == 0, "16-byte places");
  auto first_block = [&](const Open& o) { return (int)quotient((o.unit + 1) * G - 1, T); };
  // an item is the last of its first block, and the first of the others
  auto part = [&](const Open& o, int c0, int c) {
    return parts + (((size_t)(c0 + c) * 2 + (c == 0 ? 1 : 0)) * MAX_TW + o.tl) * PART_FLOATS;
  };
  __threadfence();
  for (int from = 0; from < opens;) {
    // items from .. to - 1; each thread finds the same places
    int to = from, used = 0;
    for (; to < opens; ++to) {
      if (!sh.last[to]) continue;
      const int need = sh.open[to].rows * sh.blocks[to];
      if (used + need > ROOM) break;
      used += need;
    }
    auto place = [&](int j) {
      int at = 0;
      for (int i = from; i < j; ++i)
        if (sh.last[i]) at += sh.open[i].rows * sh.blocks[i];
      return at;
    };
    // a warp an item: the rows' maxima and sums in every block, then the weights
    for (int j = from + warp; j < to; j += NW) {
      if (!sh.last[j]) continue;
      const Open& o = sh.open[j];
      const int n = sh.blocks[j], at = place(j), c0 = first_block(o);
#pragma unroll 4
      for (int i = lane; i < o.rows * n; i += 32) {
        const float* p = part(o, c0, i % n) + RT * D + i / n;
        weight[at + i] = __ldcg(p);
        part_sum[at + i] = __ldcg(p + RT);
      }
    }
    __syncthreads();
    for (int j = from; j < to; ++j) {
      if (!sh.last[j]) continue;
      const int n = sh.blocks[j], rows = sh.open[j].rows, at = place(j);
      const int width = n <= 16 ? 16 : 32;           // lanes a row
      for (int r = threadIdx.x / width; r < (rows + 1) / 2 * 2; r += NW * 32 / width) {
        float* w = weight + at + r * n;
        const int lane_c = lane % width, end = r < rows ? n : 0;
        float M = -INFINITY;
        for (int c = lane_c; c < end; c += width) M = fmaxf(M, w[c]);
        for (int k = width / 2; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
        const float Mu = M == -INFINITY ? 0.f : M;
        float sum = 0.f;
        for (int c = lane_c; c < end; c += width) {
          const float x = ex2(w[c] - Mu);
          w[c] = x;
          sum = fmaf(x, part_sum[at + r * n + c], sum);
        }
        for (int k = width / 2; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (lane_c == 0 && r < rows) item_sum[j * MAX_ROWS + r] = sum;
      }
    }
    __syncthreads();
    // As above, in an order of adding that is the item's own: which block is the last to
    // arrive, and so what other items it adds beside this one, changes from run to run.
    // Few rows of many parts leave warps over: 2^ways_log of them share a row's parts
    // (every 2^ways_log-th each) and meet in shared memory.  Up to 4 parts are one warp's
    // loads in flight together.
    auto ways_log = [&](int j) {
      const int pairs = (sh.open[j].rows + RPW - 1) / RPW;
      return sh.blocks[j] <= 4 || pairs > 4 ? 0 : pairs > 2 ? 1 : pairs > 1 ? 2 : 3;
    };
    // the place of the first share behind item j, the items' shares side by side and each
    // item's at a multiple of its ways
    auto shares = [&](int at, int j, int batch) {
      const int w = ways_log(j), rows = w > 0 ? RPW : batch * RPW;
      return ((at + (1 << w) - 1) >> w << w) + ((sh.open[j].rows + rows - 1) / rows << w);
    };
    auto finish = [&](auto batch) {
      constexpr int U = decltype(batch)::value;
      int all = 0;
      bool meet = false;
      for (int j = from; j < to; ++j)
        if (sh.last[j]) {
          all = shares(all, j, U);
          meet |= ways_log(j) > 0;
        }
      // the same number of rounds for every warp: each is at the barrier in each round
      for (int i0 = 0; i0 < all; i0 += NW) {
        int j = from, wl = 0, k = -1;                  // this warp's share of item j
        for (int at = 0; j < to; ++j) {
          if (!sh.last[j]) continue;
          wl = ways_log(j);
          const int end = shares(at, j, U);
          if (i0 + warp < end) {
            k = i0 + warp - ((at + (1 << wl) - 1) >> wl << wl);
            break;
          }
          at = end;
        }
        const bool mine = k >= 0;                      // not between two items' shares, nor behind the last
        const int ways = 1 << wl, s = k & (ways - 1), r0 = (k >> wl) * (wl > 0 ? RPW : U * RPW) + lane_row;
        const Open& o = sh.open[mine ? j : from];
        float4 x[U] = {};
        if (mine) {
          const int n = sh.blocks[j], c0 = first_block(o);
          const float* w = weight + place(j) + r0 * n;
          // part c: the second of block c0, the first of block c0 + c
          const float* p = parts + ((size_t)c0 * 2 * MAX_TW + o.tl) * PART_FLOATS + r0 * D + lane_quad * 4;
          constexpr size_t next = (size_t)2 * MAX_TW * PART_FLOATS;
          const int rows = wl > 0 ? min(o.rows, r0 + 1) : o.rows;   // one row a lane where parts are shared
#pragma unroll 8
          for (int c = s; c < n; c += ways) {
            const float* q = p + (c == 0 ? next / 2 : c * next);
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (r0 + u * RPW < rows)
                add(x[u], w[u * RPW * n + c], __ldcg(reinterpret_cast<const float4*>(q + u * RPW * D)));
          }
        }
        if (meet) {
          shared_sum[threadIdx.x] = x[0];
          __syncthreads();
          if (mine && s == 0)
            for (int q = 1; q < ways; ++q) add(x[0], 1.f, shared_sum[threadIdx.x + q * 32]);
          __syncthreads();
        }
        if (!mine || s != 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r0 + u * RPW < o.rows && (u == 0 || wl == 0))
            store(o, r0 + u * RPW, lane_quad, x[u], item_sum[j * MAX_ROWS + r0 + u * RPW]);
      }
    };
    int one = 0;                                       // shares of a row, or a pair of them
    for (int j = from; j < to; ++j)
      if (sh.last[j]) one = shares(one, j, 1);
    if (one <= NW) finish(std::integral_constant<int, 1>{});
    else finish(std::integral_constant<int, 4>{});
    __syncthreads();                                 // the weights have been read
    from = to;
  }
}

template <int FMT, int D, int NT>
int launch_fast(const KvAttnArgs& a, const CUtensorMap* mK, const CUtensorMap* mV, int group, long long max_tiles,
                int tw, int vec, int num_sms, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  constexpr int smem = NW * RING + 1024;
  cudaError_t e = set_smem_once(smem_set, kv_attention_kernel<FMT, D, NT>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(num_sms < MAX_CTAS ? num_sms : MAX_CTAS));
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<FMT, D, NT>, *mK, *mV, a, group, max_tiles, tw, vec);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// How a call's query rows a head (its longest sequence's) are cut: tiles of 8 NT rows,
// one of each of tw warps side by side.  A tile as high as the rows allow spares
// widening the same codes for another one; beyond 32 rows the warps share evenly.
// Measured: 40 rows of 128 (9 x 20000 x 8 tokens) as three tiles of 16 297 us, two of
// 24 205; 20 rows of 64 (24 x 1500 x 5) as two of 16 35.3, one of 24 28.5.
struct Tiling {
  int nt, tw;
  long long tiles;
};
Tiling tiling(long long rows) {
  const long long eights = (rows + 7) / 8;
  const int tw = eights <= 4 ? 1 : eights <= 8 ? 2 : MAX_TW;
  const int nt = (int)std::min<long long>(4, (eights + tw - 1) / tw);
  return {nt, tw, (eights + nt - 1) / nt};
}

template <class Kernel>
int launch(Kernel kernel, dim3 grid, dim3 block, const KvAttnArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t kv_attention_ws_bytes(int seqs, int heads, int group, int max_new) {
  const size_t tiles = (size_t)tiling((long long)max_new * group).tiles;
  return PARTS * PART_FLOATS * sizeof(float) + ((size_t)seqs * heads * tiles + 3) / 4 * 16;
}

int launch_kv_attention(const KvAttnArgs& a, const CUtensorMap* mK, const CUtensorMap* mV, int num_sms,
                        cudaStream_t s) {
  const int group = a.Hq / a.c.H;
  const Tiling x = tiling((long long)a.max_new * group);
  // pairs of outputs and quads of queries as one access
  const int vec = reinterpret_cast<uintptr_t>(a.Q) % 8 == 0 && a.ldq % 4 == 0 &&
                  reinterpret_cast<uintptr_t>(a.O) % 4 == 0 && a.ldo % 2 == 0;
  auto go = [&](auto fmt, auto dim) -> int {
    constexpr int F = decltype(fmt)::value, D = decltype(dim)::value;
    switch (x.nt) {
      case 1: return launch_fast<F, D, 1>(a, mK, mV, group, x.tiles, x.tw, vec, num_sms, s);
      case 2: return launch_fast<F, D, 2>(a, mK, mV, group, x.tiles, x.tw, vec, num_sms, s);
      case 3: return launch_fast<F, D, 3>(a, mK, mV, group, x.tiles, x.tw, vec, num_sms, s);
      default: return launch_fast<F, D, 4>(a, mK, mV, group, x.tiles, x.tw, vec, num_sms, s);
    }
  };
  using std::integral_constant;
  if (a.c.fmt == kKvE4M3)
    return a.c.D == 128 ? go(integral_constant<int, kKvE4M3>{}, integral_constant<int, 128>{})
                        : go(integral_constant<int, kKvE4M3>{}, integral_constant<int, 64>{});
  return a.c.D == 128 ? go(integral_constant<int, kKvInt8>{}, integral_constant<int, 128>{})
                      : go(integral_constant<int, kKvInt8>{}, integral_constant<int, 64>{});
}

int launch_kv_attention_generic(const KvAttnArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.tokens, (unsigned)a.Hq);
  if (a.c.fmt == kKvE4M3) return launch(kv_attention_generic_kernel<kKvE4M3>, grid, dim3(GT), a, s);
  return launch(kv_attention_generic_kernel<kKvInt8>, grid, dim3(GT), a, s);
}

}  // namespace g3

// Attention of drafted tokens over a paged cache, up to 16 rows a unit, sm_103a.
//
// Sequence b has ctx_b cached tokens and T_b <= 64 drafted ones at positions ctx_b ..
// ctx_b + T_b - 1 of its pages.  Row (t, head) sees every context key, and drafted key u when
// bit u of the token's mask word is set (without masks: u <= t).  A unit is (sequence, K/V
// head, tile of kRows rows): the G = Hq / Hkv query heads of a group and the drafted tokens
// share a unit's rows, row r = t * G + g, so every K/V row is read once for all of them.
//
// Bound: K and V are read once, 4 d (bf16) or 2 d + 2 (e4m3) bytes a key, for 4 d flops a row
// and key; below 274 rows a unit memory is the limit.  Measured on GB300, one token a sequence,
// 32 query and 8 K/V heads, d = 128, sequences of 900 to 16384 tokens: 48 of them in bf16, 1.14 GB
// in 180 us, 6.3 TB/s; 64 in e4m3, 770 MB in 147 us, 5.2 TB/s (there the conversions of K and V
// take half the issue slots, and the latency between dependent steps is the limit: more conversions
// cost little, a third CTA an SM gave an eighth).
//
// Work split: the keys of all units are laid end to end in chunks of 64 or 128 (and some places
// for what a unit costs beside them, see tree_plan) and cut into equal ranges, one a CTA (two
// CTAs an SM, three with e4m3), whatever the lengths are; every CTA finds its range from a
// prefix sum over the sequences, so a captured launch follows the lengths on the device.  A
// CTA's range covers a few whole units and at most two that it shares: its first piece may be
// the rest of a unit begun by an earlier CTA, its last one the front of a unit that goes on in
// the next.  Whole units leave as O and LSE; shared ones as the running state (m, l, o~) in
// one of the CTA's two workspace slots, merged by attn_tree_merge_kernel.
//
// e4m3.  K's codes become f16 pairs (exact, one instruction a pair) against a query row divided by
// the power of two of its largest finite value.  V's become bf16 pairs, exact, and its keys' scales
// go into P, which therefore is bf16: with f16 (three conversions a pair of V less) a key's scale,
// seen by a row or not, would decide how small a weight the other keys may have.
//
// Inside a CTA each warp takes every fourth slice of 16 or 32 keys of the piece on its own: its own ring
// of stages filled by TMA, its own (m, l, o~) in registers, no barrier in the loop.  The four
// states are combined once a piece.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_cache_kernel.cuh"
#include "ptx.cuh"

namespace attn {

constexpr int kTreeMaxNodes = 64;    // bits of a mask word
constexpr int kPlanGroups = 64;      // prefix-sum entries (each over ceil(B / 64) sequences)

struct TreeParams {
  const __nv_bfloat16* q;      // [total_q, Hq, d]
  __nv_bfloat16* o;            // [total_q, Hq, d]
  float* lse;                  // [Hq, total_q]
  const int32_t* table;        // [B, max_pages]
  const int32_t* cu;           // [B + 1]
  const int32_t* ctx;          // [B] or null (no context)
  const unsigned long long* mask;  // [total_q] or null (a chain)
  const void* v;               // the cache's values
  const uint8_t* ks;           // [num_pages, Hkv, page] e4m3 only
  const uint8_t* vs;
  int B, Hq, Hkv, G;
  int max_q, total_q;
  int num_pages, page, max_pages;
  int cap;                     // max_pages * page: positions the table has room for
  int box_rows;                // keys a copy takes (128-row tiles): 16 .. 128, divides the page
  int tok_tile;                // tokens a 128-row tile holds (kRows = 128)
  int fan;                     // CTAs that walk a list of units together, a tile each (1: every tile its own unit)
  int unit_cost;               // what a unit costs beside its chunks, in chunks (see tree_plan)
  float c;                     // scale * log2(e)
  float* st_o;                 // [2 * CTAs, kRows, d] states of shared units
  float* st_m;                 // [2 * CTAs, kRows] log2 units
  float* st_l;
  int4* meta;                  // [2 * CTAs]: (first row, drafted tokens, head, tile), (last CTA, ..) of the unit
                               // whose front is the CTA's slot 1; last CTA < 0: none
  uint32_t* status;            // bounded waits
  uint32_t* page_word;         // bad pages
  unsigned long long timeout_ns;
  int fault_block;             // test hook: the block of 128 keys that is never loaded (-1: none)
};

// One sequence as the kernels see it, every field clamped to what the buffers hold.
struct TreeSeq {
  int q0, T;    // first packed row, drafted tokens
  int ctx, n;   // context keys, keys in all
  int nch;      // chunks of keys (1 at least while there are rows)
  int tiles;    // row tiles of one head (of fan tiles each)
};

template <int kRows, int kChunk>
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  s.q0 = min(max(__ldg(p.cu + b), 0), p.total_q);
  const int q1 = min(max(__ldg(p.cu + b + 1), s.q0), p.total_q);
  s.T = min(q1 - s.q0, p.max_q);
  s.ctx = p.ctx ? min(max(__ldg(p.ctx + b), 0), p.cap) : 0;
  s.n = static_cast<int>(min(static_cast<long long>(s.ctx) + s.T, static_cast<long long>(p.cap)));
  s.nch = s.T > 0 ? max(1, s.n / kChunk + (s.n % kChunk != 0)) : 0;
  s.tiles = kRows == 16 ? (s.T * p.G + kRows - 1) / kRows : (s.T + p.tok_tile * p.fan - 1) / (p.tok_tile * p.fan);
  return s;
}

// Row r of a tile: token and head of the group; false when there is none.  16-row tiles are
// cut from the rows t * G + g; a 128-row tile holds all heads of tok_tile tokens.
template <int kRows>
__device__ __forceinline__ bool tree_row(const TreeParams& p, const TreeSeq& s, int tile, int r, int* tok, int* g) {
  const int rr = kRows == 16 ? tile * kRows + r : r;
  const int t = rr / p.G;
  *g = rr - t * p.G;
  *tok = kRows == 16 ? t : tile * p.tok_tile + t;
  return *tok < s.T && (kRows == 16 || t < p.tok_tile);
}

// A run of chunks of one unit.
struct TreePiece {
  TreeSeq s;
  int b, h, tile;
  int ch0, ch1;       // chunks [ch0, ch1) of the unit's s.nch (none when ch1 <= ch0)
  long long adv;      // places of the list it covers
};

// The list of places the CTAs divide: every unit takes unit_cost places, then one for each of
// its chunks.  The places at the front stand for what a unit costs whatever its length (its
// rows, its start, its states' merge); without them a CTA that falls among many short
// sequences gets as many units as another gets chunks.
// pre[i]: places of all units of the sequences before group i (groups of gs sequences).
// CTA-wide (at least kPlanGroups threads).
template <int kRows, int kChunk>
__device__ __forceinline__ void tree_plan(const TreeParams& p, int gs, long long* pre, long long* warp_sums) {
  const int t = threadIdx.x;
  long long sum = 0;
  if (t < kPlanGroups) {
    const long long first = static_cast<long long>(t) * gs;
    for (long long b = first; b < min(first + gs, static_cast<long long>(p.B)); ++b) {
      const TreeSeq s = tree_seq<kRows, kChunk>(p, static_cast<int>(b));
      sum += (s.nch > 0 ? static_cast<long long>(s.nch) + p.unit_cost : 0ll) * s.tiles * p.Hkv;
      if (blockIdx.x == 0 && s.T > 0 && p.page_word && static_cast<long long>(s.ctx) + s.T > p.cap)
        atomicOr(p.page_word, 1u);
    }
    const int lane = t & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sums[t >> 5] = sum;
  }
  __syncthreads();
  if (t < kPlanGroups) {
    for (int w = 0; w < (t >> 5); ++w) sum += warp_sums[w];
    pre[t + 1] = sum;
    if (t == 0) pre[0] = 0;
  }
  __syncthreads();
}

// x / y for 0 <= x, 0 < y: 32 bits wide where both fit (a 64-bit division costs about as much
// as a global load; out of line, since what runs rarely should not fill the instruction cache).
__device__ __noinline__ long long tree_div_wide(long long x, long long y) { return x / y; }
__device__ __forceinline__ long long tree_div(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return tree_div_wide(x, y);
}

// The places [x0, x1) of CTA `cta` of `grid`: the first `extra` CTAs have per + 1, the others per.
struct TreeRange {
  long long per, extra, x0, x1;
};
__device__ __forceinline__ TreeRange tree_range(long long W, long long cta, long long grid) {
  TreeRange r;
  r.per = tree_div(W, grid);
  r.extra = W - r.per * grid;
  r.x0 = r.per * cta + min(cta, r.extra);
  r.x1 = r.x0 + r.per + (cta < r.extra ? 1 : 0);
  return r;
}
// The CTA whose range holds place x.
__device__ __forceinline__ int tree_owner(const TreeRange& r, long long x) {
  const long long big = r.extra * (r.per + 1);
  return static_cast<int>(x < big ? tree_div(x, r.per + 1) : r.extra + tree_div(x - big, max(r.per, 1ll)));
}

// The piece that starts at place x of the list and ends with its unit or at x_end.
template <int kRows, int kChunk>
__device__ __forceinline__ TreePiece tree_piece(const TreeParams& p, int gs, const long long* pre, long long x,
                                                long long x_end) {
  int lo = 0, hi = kPlanGroups;  // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  TreePiece pc;
  pc.b = lo * gs;
  long long base = pre[lo];
  int len = 1;  // places of a unit of the sequence
  for (;; ++pc.b) {  // ends: x < pre[lo + 1], the places of this group's last sequence
    pc.s = tree_seq<kRows, kChunk>(p, pc.b);
    len = pc.s.nch + p.unit_cost;
    const long long w = pc.s.nch > 0 ? static_cast<long long>(len) * pc.s.tiles * p.Hkv : 0;
    if (x < base + w || pc.b + 1 >= p.B) break;
    base += w;
  }
  const long long y = x - base;
  const int unit = static_cast<int>(tree_div(y, len));
  pc.h = unit / max(pc.s.tiles, 1);
  pc.tile = unit - pc.h * pc.s.tiles;
  const int off = static_cast<int>(y - static_cast<long long>(unit) * len);
  const int end = static_cast<int>(min(static_cast<long long>(len), off + (x_end - x)));
  pc.adv = end - off;
  pc.ch0 = max(0, off - p.unit_cost);
  pc.ch1 = max(0, end - p.unit_cost);
  return pc;
}

// Drafted nodes token t of a sequence sees, as bits.
__device__ __forceinline__ unsigned long long tree_sees(const TreeParams& p, const TreeSeq& s, int t) {
  const unsigned long long all = s.T >= 64 ? ~0ull : (1ull << s.T) - 1ull;
  const unsigned long long w = p.mask ? __ldg(p.mask + s.q0 + t) : (t >= 63 ? ~0ull : (2ull << t) - 1ull);
  return w & all;
}

// ------------------------------------------------------------------ warp-level products

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], fp32 accumulation.
__device__ __forceinline__ void warp_mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void warp_mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Plain bulk copy global -> shared (both addresses and the size multiples of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// e4m3 pair -> bf16 pair, exact (every e4m3 value is a bf16).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t codes) {
  const float2 f = e4m3x2_to_f32(codes);
  return pack_bf16x2(f.x, f.y);
}

constexpr int kTreeRows = 16;
constexpr int kTreeWarps = 4;
constexpr int kTreeThreads = 32 * kTreeWarps;

template <int D, bool kF8>
struct TreeCfg {
  static constexpr int kRowBytes = kF8 ? D : 2 * D;
  // Keys a warp takes at a time.  Every slice pays for its wait, its copies' issue and the
  // maximum's shuffles, so rows of 128 bytes and less go 32 at a time; 256-byte rows at 32 would
  // leave too few stages.
  static constexpr int kSlice = kRowBytes > 128 ? 16 : 32;
  static constexpr int kSubs = kSlice / 16;                      // 16-key boxes of a slice
  static constexpr int kChunk = kTreeWarps * kSlice;             // keys a CTA takes at a time
  static constexpr int kHalf = kSlice * kRowBytes;               // K (or V) of a slice
  static constexpr int kStageBytes = 2 * kHalf;
  static constexpr int kCtas = kF8 ? 3 : 2;                      // an SM
  static constexpr int kRingBytes = (kCtas == 3 ? (D == 64 ? 12 : 16) : 24) * 1024 / kStageBytes * kStageBytes;  // of a warp
  static constexpr int kStages = kRingBytes / kStageBytes;
  static constexpr int kSub = kRowBytes > 128 ? kRowBytes / 128 : 1;  // 128-byte wide sub-tiles
  static constexpr int kSubBytes = kHalf / kSub;
  static constexpr int kCodes = 2 * kSlice;                      // e4m3: scale codes of K, then of V
  static constexpr int kBoxBytes = 2 * 16 * kRowBytes + (kF8 ? 32 : 0);  // what a 16-key box brings
  static constexpr int kOffScale = kTreeWarps * kRingBytes;
  static constexpr int kOffBar = kOffScale + (kF8 ? kTreeWarps * kStages * kCodes : 0);
  static constexpr int kOffMerge = (kOffBar + kTreeWarps * kStages * 8 + 15) / 16 * 16;
  // the warps' states on their way into one, 32 columns at a time; e4m3: the query's fragments before
  static constexpr int kOffStat = kOffMerge + kTreeWarps * kTreeRows * 32 * 4;
  static constexpr int kOffPre = kOffStat + 2 * kTreeWarps * kTreeRows * 4;
  static constexpr int kOffMisc = kOffPre + (kPlanGroups + 1 + 4) * 8;
  static constexpr int kSmem = kOffMisc + 16 + 1024;             // slack to align the base
  static_assert(kSub == 1 || kSubs == 1, "a slice is one box, or its rows lie one after the other");
  static_assert(kStages >= 2 && kStages * kSubs <= 32, "bits");
  static_assert(kSmem <= 228 * 1024 / kCtas - 1024, "CTAs an SM");
};

template <int D, bool kF8>
__global__ void __launch_bounds__(kTreeThreads, TreeCfg<D, kF8>::kCtas)
    attn_tree_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const TreeParams p) {
  using C = TreeCfg<D, kF8>;
  constexpr int kSlice = C::kSlice, kSubs = C::kSubs, kChunk = C::kChunk;
  constexpr int kKeyTiles = kSlice / 8;
  constexpr int kTilesN = D / 8;   // 8-wide column tiles of o~
  constexpr int kSteps = D / 16;   // 16-deep steps of q . k
  constexpr float kTau = 8.f;      // o~ is rescaled when the max rises by more (log2 units)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // fragment row and column pair
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ring = sbase + warp * C::kRingBytes;
  const uint32_t bars = sbase + C::kOffBar + warp * C::kStages * 8;
  uint8_t* scales = smem + C::kOffScale + warp * C::kStages * C::kCodes;
  float* merge = reinterpret_cast<float*>(smem + C::kOffMerge);
  float* stat_m = reinterpret_cast<float*>(smem + C::kOffStat);
  float* stat_l = stat_m + kTreeWarps * kTreeRows;
  long long* pre = reinterpret_cast<long long*>(smem + C::kOffPre);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc);
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
    if (warp == 0) {
      *abort_flag = 0u;
      if (p.num_pages > 0) {  // without pages there are no maps
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
      }
    }
  }
  griddep_wait();
  griddep_launch_dependents();
  const int gs = (p.B + kPlanGroups - 1) / kPlanGroups;
  tree_plan<kTreeRows, kChunk>(p, gs, pre, pre + kPlanGroups + 1);  // its barriers also publish the mbarriers

  const long long W = pre[kPlanGroups];
  const int cta = static_cast<int>(blockIdx.x);
  const TreeRange range = tree_range(W, cta, gridDim.x);
  const long long x0 = range.x0, x1 = range.x1;
  bool has_tail = false;

  // ---- loads: an iterator over this warp's slices, kStages ahead of the products
  const uint64_t pol = policy_evict_first();
  long long px = x0;          // next place to make a piece of
  int ps = 0, ps_end = 0;     // slices [ps, ps_end) step 4 of the piece in hand
  int pbase = 0, pages = 0;   // lane i: the page of box i % kSubs of slice pbase + 4 (i / kSubs)
  int pb = 0, ph = 0, pn = 0;
  uint32_t there = 0;         // bits kSubs * stage ..: boxes that exist and have been asked for
  uint32_t live = 0;          // stages with a copy in flight
  uint32_t phase = 0;         // parity each stage completes next
  int ist = 0;                // stage of the next issue
  auto fetch_pages = [&]() {
    pbase = ps;
    const int s = ps + kTreeWarps * (lane / kSubs);
    const long long pos = static_cast<long long>(s) * kSlice + 16 * (lane % kSubs);
    pages = s < ps_end && pos < pn ? __ldg(p.table + static_cast<long long>(pb) * p.max_pages +
                                           static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page))
                                   : -1;
  };
  auto issue = [&]() {
    while (ps >= ps_end) {
      if (px >= x1) return;
      const TreePiece pc = tree_piece<kTreeRows, kChunk>(p, gs, pre, px, x1);
      px += pc.adv;
      if (pc.ch1 <= pc.ch0) continue;
      pb = pc.b;
      ph = pc.h;
      pn = pc.s.n;
      ps = pc.ch0 * kTreeWarps + warp;
      const long long end = min(static_cast<long long>(pc.ch1) * kChunk, static_cast<long long>(pc.s.n));
      ps_end = static_cast<int>((end + kSlice - 1) / kSlice);
      fetch_pages();
    }
    if (ps - pbase >= (32 / kSubs) * kTreeWarps) fetch_pages();
    // lane i < kSubs looks after box i
    const int pg = __shfl_sync(0xffffffffu, pages, (ps - pbase) / kTreeWarps * kSubs + (lane % kSubs));
    const bool need = lane < kSubs && static_cast<long long>(ps) * kSlice + 16 * lane < pn;
    const bool have = need && static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages);
    if (need && !have && p.page_word) atomicOr(p.page_word, 1u);
    const uint32_t boxes = __ballot_sync(0xffffffffu, have);
    there = (there & ~(((1u << kSubs) - 1u) << (kSubs * ist))) | (boxes << (kSubs * ist));
    if (boxes) {
      const uint32_t bar = bars + 8 * ist;
      const bool withheld = ps * kSlice / 128 == p.fault_block;
      if (!withheld) live |= 1u << ist;
      if (lane == 0 && !withheld) mbar_arrive_expect_tx(bar, __popc(boxes) * C::kBoxBytes);
      __syncwarp();
      if (have && !withheld) {
        const uint32_t dst = ring + ist * C::kStageBytes + 16 * lane * C::kRowBytes;  // lane 0 where kSub > 1
        const int row = static_cast<int>((static_cast<uint32_t>(ps) * kSlice + 16u * lane) % static_cast<uint32_t>(p.page));
#pragma unroll
        for (int s = 0; s < C::kSub; ++s) tma_load_4d(dst + s * C::kSubBytes, &tmK, bar, s * 64, row, ph, pg, pol);
#pragma unroll
        for (int s = 0; s < C::kSub; ++s)
          tma_load_4d(dst + C::kHalf + s * C::kSubBytes, &tmV, bar, s * 64, row, ph, pg, pol);
        if constexpr (kF8) {
          const long long r = (static_cast<long long>(pg) * p.Hkv + ph) * p.page + row;
          const uint32_t sc = smem_u32(scales + ist * C::kCodes) + 16 * lane;
          bulk_load(sc, p.ks + r, 16, bar);
          bulk_load(sc + kSlice, p.vs + r, 16, bar);
        }
      }
    }
    ps += kTreeWarps;
    ist = ist + 1 == C::kStages ? 0 : ist + 1;
  };
#pragma unroll 1
  for (int s = 0; s < C::kStages; ++s) issue();

  bool ok = true;
  int cst = 0;  // stage of the next slice to take
  for (long long x = x0; x < x1;) {
    const TreePiece pc = tree_piece<kTreeRows, kChunk>(p, gs, pre, x, x1);
    x += pc.adv;
    if (pc.ch1 <= pc.ch0) continue;
    // ---- this thread's two rows: g and g + 8
    float cr[2];                    // c, times the power of two the row was divided by (e4m3)
    unsigned long long sees[2];
    const __nv_bfloat16* qrow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int tok, head;
      cr[i] = p.c;
      sees[i] = ~0ull;  // a row that is none: anything
      qrow[i] = nullptr;
      if (tree_row<kTreeRows>(p, pc.s, pc.tile, g + 8 * i, &tok, &head)) {
        sees[i] = tree_sees(p, pc.s, tok);
        qrow[i] = p.q + (static_cast<long long>(pc.s.q0 + tok) * p.Hq + pc.h * p.G + head) * D;
      }
    }
    // The query's fragments: bf16 in registers; e4m3 in shared memory, the same for all four warps,
    // which leaves registers for a third CTA an SM (64 sequences of 1000 to 16384 tokens, d = 128,
    // on GB300: 165 -> 145 us)
    uint32_t qf[kF8 ? 1 : kSteps][4];
    uint4* qs = reinterpret_cast<uint4*>(merge);
    if constexpr (!kF8) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)  // columns 16 k + 8 (j / 2) + 2 t
          qf[k][j] = qrow[j & 1] ? __ldg(reinterpret_cast<const uint32_t*>(qrow[j & 1]) + k * 8 + (j >> 1) * 4 + t) : 0u;
    } else {
      // f16 operands: a row is divided by the power of two of its largest finite value, so its
      // values lie in (-2, 2) and keep all 8 bits down to 2^-14 of the largest.  Columns are
      // taken in the order the codes of K arrive in: 16 k + 4 t .. + 3.
      uint2 w[kSteps][2];
      uint32_t mx[2] = {0, 0};
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[k][i] = qrow[i] ? __ldg(reinterpret_cast<const uint2*>(qrow[i]) + k * 4 + t) : make_uint2(0u, 0u);
          mx[i] = max(mx[i], finite_max(make_uint4(w[k][i].x, w[k][i].y, 0u, 0u)));
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = max(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = max(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
        const uint32_t ef = min(max(mx[i] >> 7, 1u), 253u);  // exponent field of the row's power of two
        const float inv = __uint_as_float((254u - ef) << 23);
        cr[i] = p.c * __uint_as_float(ef << 23);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          w[k][i].x = pack_f16x2(bf16_lo(w[k][i].x) * inv, bf16_hi(w[k][i].x) * inv);
          w[k][i].y = pack_f16x2(bf16_lo(w[k][i].y) * inv, bf16_hi(w[k][i].y) * inv);
        }
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k)  // every warp has them all; each stores its share
        if (k % kTreeWarps == warp) qs[k * 32 + lane] = make_uint4(w[k][0].x, w[k][1].x, w[k][0].y, w[k][1].y);
      __syncthreads();
    }
    float acc[kTilesN][4];
#pragma unroll
    for (int j = 0; j < kTilesN; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // l: this thread's columns only

    const long long end = min(static_cast<long long>(pc.ch1) * kChunk, static_cast<long long>(pc.s.n));
    const int s_end = static_cast<int>((end + kSlice - 1) / kSlice);
#pragma unroll 1
    for (int s = pc.ch0 * kTreeWarps + warp; s < s_end; s += kTreeWarps) {
      const int st = cst;
      cst = cst + 1 == C::kStages ? 0 : cst + 1;
      const uint32_t boxes = (there >> (kSubs * st)) & ((1u << kSubs) - 1u);
      if (boxes) {
        const uint32_t bit = 1u << st;
        const bool got = mbar_wait(bars + 8 * st, (phase & bit) ? 1u : 0u, wc, 32);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;  // the copy stays in flight
          break;
        }
        phase ^= bit;
        live &= ~bit;
        const uint32_t sk = ring + st * C::kStageBytes, sv = sk + C::kHalf;
        const int k0 = s * kSlice;
        const int left = pc.s.n - k0;  // keys from `left` on do not exist: their rows may hold anything
        const bool part = left < kSlice || boxes != (1u << kSubs) - 1u;
        // ---- scores: sc[key tile][row g: 0, 1; row g + 8: 2, 3], keys 8 n + 2 t, + 1
        float sc[kKeyTiles][4];
#pragma unroll
        for (int i = 0; i < 4 * kKeyTiles; ++i) (&sc[0][0])[i] = 0.f;
        float pv[2 * kKeyTiles];  // e4m3: scales of V of this thread's keys
        if constexpr (!kF8) {
          const int key = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
          for (int k = 0; k < kSteps; ++k) {
            const int ch = (k & 3) * 2 + ((lane >> 3) & 1);  // 16-byte chunk of the 128-byte row
#pragma unroll
            for (int b = 0; b < kSubs; ++b) {
              uint32_t w[4];
              ldsm4(w, sk + (k >> 2) * C::kSubBytes + (16 * b + key) * 128 + ((ch ^ (key & 7)) << 4));
              warp_mma_bf16(sc[2 * b], qf[k], w[0], w[1]);
              warp_mma_bf16(sc[2 * b + 1], qf[k], w[2], w[3]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4 * kKeyTiles; ++i) (&sc[0][0])[i] *= p.c;
        } else {
          // chunk ch holds 16 columns; a register of it is 4 codes of a key, two f16 pairs
          const int key = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
          for (int k = 0; k < kSteps; k += 2) {
            const int ch = k + (lane >> 4);
            const uint32_t at = D == 128 ? key * 128 + ((ch ^ (key & 7)) << 4) : key * 64 + ((ch ^ ((key >> 1) & 3)) << 4);
            const uint4 q[2] = {qs[k * 32 + lane], qs[(k + 1) * 32 + lane]};
#pragma unroll
            for (int b = 0; b < kSubs; ++b) {
              uint32_t w[4];
              ldsm4(w, sk + 16 * b * C::kRowBytes + at);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                warp_mma_f16(sc[2 * b], &q[i].x, e4m3x2_to_f16x2(w[2 * i] & 0xffffu), e4m3x2_to_f16x2(w[2 * i] >> 16));
                warp_mma_f16(sc[2 * b + 1], &q[i].x, e4m3x2_to_f16x2(w[2 * i + 1] & 0xffffu),
                             e4m3x2_to_f16x2(w[2 * i + 1] >> 16));
              }
            }
          }
          const uint8_t* kc = scales + st * C::kCodes;
#pragma unroll
          for (int n = 0; n < kKeyTiles; ++n) {
            const uint32_t a = *reinterpret_cast<const uint16_t*>(kc + 8 * n + 2 * t);
            const uint32_t b = *reinterpret_cast<const uint16_t*>(kc + kSlice + 8 * n + 2 * t);
            const float f0 = scale_of(a & 0xffu), f1 = scale_of(a >> 8);
            sc[n][0] *= cr[0] * f0;
            sc[n][1] *= cr[0] * f1;
            sc[n][2] *= cr[1] * f0;
            sc[n][3] *= cr[1] * f1;
            pv[2 * n] = scale_of(b & 0xffu);
            pv[2 * n + 1] = scale_of(b >> 8);
            if (part) {  // a key that does not exist may have any code: 0 keeps 0 * scale from being NaN
              const bool out = !((boxes >> (n / 2)) & 1u);
              if (out || 8 * n + 2 * t >= left) pv[2 * n] = 0.f;
              if (out || 8 * n + 2 * t + 1 >= left) pv[2 * n + 1] = 0.f;
            }
          }
        }
        // ---- masks: every row sees the context; drafted keys go by the row's bits
        const bool draft = k0 + kSlice > pc.s.ctx;
        if (draft || part) {
#pragma unroll
          for (int n = 0; n < kKeyTiles; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int u = k0 + 8 * n + 2 * t + i - pc.s.ctx;
              const bool out = !((boxes >> (n / 2)) & 1u) || u >= 64;
              if (out || (u >= 0 && !((sees[0] >> u) & 1ull))) sc[n][i] = -INFINITY;
              if (out || (u >= 0 && !((sees[1] >> u) & 1ull))) sc[n][2 + i] = -INFINITY;
            }
        }
        // ---- running max (rows g, g + 8) and probabilities
        bool move = false;
        float alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(sc[0][2 * i], sc[0][2 * i + 1]);
#pragma unroll
          for (int n = 1; n < kKeyTiles; ++n) mx = fmaxf(mx, fmaxf(sc[n][2 * i], sc[n][2 * i + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = mx > m[i] + kTau ? mx : m[i];
          const float ref = mn == -INFINITY ? 0.f : mn;
          alpha[i] = ex2_approx(m[i] - ref);
          move |= mn != m[i];
          m[i] = mn;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < kKeyTiles; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float e = ex2_approx(sc[n][2 * i + j] - ref);
              sum += e;
              sc[n][2 * i + j] = e;
            }
          l[i] = l[i] * alpha[i] + sum;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int j = 0; j < kTilesN; ++j) {
            acc[j][0] *= alpha[0];
            acc[j][1] *= alpha[0];
            acc[j][2] *= alpha[1];
            acc[j][3] *= alpha[1];
          }
        }
        uint8_t* vat = smem + (sv - sbase);
        bool odd = false;  // a drafted key's value that is infinite or NaN
        if (draft || part) {
          if (part) {
            // rows of V that do not exist: 0 instead of what is there (0 * NaN is NaN).  Their
            // copies have landed, so plain stores to them stay.
#pragma unroll 1
            for (int i = lane; i < C::kHalf / 16; i += 32) {
              const int key = i % (C::kSubBytes / 16) / (C::kRowBytes / C::kSub / 16);
              if (key >= left || !((boxes >> (key / 16)) & 1u)) reinterpret_cast<uint4*>(vat)[i] = make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          // drafted nodes of this slice, as bits; nothing is masked when every row sees them all
          const int u0 = max(0, k0 - pc.s.ctx), u1 = min(pc.s.T, k0 + kSlice - pc.s.ctx);
          const unsigned long long here = u1 > u0 ? ((~0ull >> (64 - (u1 - u0))) << u0) : 0ull;
          if (__any_sync(0xffffffffu, ((sees[0] & sees[1]) & here) != here)) {
            // A masked probability of 0 times such a value would be NaN in rows that do not see
            // the key: then this slice goes key by key and only to the rows that see it.
            bool bad = false;
            if constexpr (kF8) bad = lane < kSlice && lane < left && scales[st * C::kCodes + kSlice + lane] == 255u;
#pragma unroll 1
            for (int i = lane; i < C::kHalf / 4; i += 32) {  // words, wherever the swizzle put them
              const uint32_t w = reinterpret_cast<const uint32_t*>(vat)[i];
              if constexpr (kF8)
                bad |= any_nonfinite(e4m3x2_to_bf16x2(w & 0xffffu)) || any_nonfinite(e4m3x2_to_bf16x2(w >> 16));
              else
                bad |= any_nonfinite(w);
            }
            odd = __any_sync(0xffffffffu, bad);
          }
        }
        // ---- o~ += P V.  Columns of tile j: bf16 8 j + 2 t, + 1; e4m3 16 (j / 2) + 4 t + (j & 1), + 2.
        const int vkey = ((lane >> 3) & 1) * 8 + (lane & 7);
        if (!odd) {
#pragma unroll
          for (int b = 0; b < kSubs; ++b) {
            // P rounds to bf16 for the product (relative 2^-8 at most; its range keeps small
            // probabilities next to a large one as precise)
            uint32_t pf[4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float a = sc[2 * b + n][2 * i], e = sc[2 * b + n][2 * i + 1];
                pf[2 * n + i] = kF8 ? pack_bf16x2(a * pv[4 * b + 2 * n], e * pv[4 * b + 2 * n + 1]) : pack_bf16x2(a, e);
              }
            if constexpr (!kF8) {
#pragma unroll
              for (int jj = 0; jj < kTilesN / 2; ++jj) {
                const int ch = (jj & 3) * 2 + (lane >> 4);
                uint32_t w[4];
                ldsm4_t(w, sv + (jj >> 2) * C::kSubBytes + (16 * b + vkey) * 128 + ((ch ^ (vkey & 7)) << 4));
                warp_mma_bf16(acc[2 * jj], pf, w[0], w[1]);
                warp_mma_bf16(acc[2 * jj + 1], pf, w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int c0 = 0; c0 < kSteps; c0 += 2) {  // two 16-column chunks: four tiles
                const int ch = c0 + (lane >> 4);
                const uint32_t at =
                    D == 128 ? vkey * 128 + ((ch ^ (vkey & 7)) << 4) : vkey * 64 + ((ch ^ ((vkey >> 1) & 3)) << 4);
                uint32_t w[4];
                ldsm4_t(w, sv + 16 * b * C::kRowBytes + at);  // keys 0-7, 8-15 of chunk c0, then of c0 + 1
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  // codes (key 2t, col 2g), (2t, 2g + 1), (2t + 1, 2g), (2t + 1, 2g + 1) -> pairs of keys
                  const uint32_t y0 = __byte_perm(w[2 * i], 0, 0x3120), y1 = __byte_perm(w[2 * i + 1], 0, 0x3120);
                  warp_mma_bf16(acc[2 * (c0 + i)], pf, e4m3x2_to_bf16x2(y0 & 0xffffu), e4m3x2_to_bf16x2(y1 & 0xffffu));
                  warp_mma_bf16(acc[2 * (c0 + i) + 1], pf, e4m3x2_to_bf16x2(y0 >> 16), e4m3x2_to_bf16x2(y1 >> 16));
                }
              }
            }
          }
        } else {
#pragma unroll 1
          for (int key = 0; key < min(left, kSlice); ++key) {
            const int u = k0 + key - pc.s.ctx;
            // the probabilities of this key sit in lane (key % 8) / 2 of each row's four
            float e[2];
            bool see[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float a = 0.f;
#pragma unroll
              for (int n = 0; n < 2 * kKeyTiles; ++n)
                if ((key >> 3) == n / 2 && (key & 1) == (n & 1)) a = sc[n / 2][2 * i + (n & 1)] * (kF8 ? pv[n] : 1.f);
              e[i] = __shfl_sync(0xffffffffu, a, (lane & ~3) | ((key & 7) >> 1));
              see[i] = ((boxes >> (key / 16)) & 1u) && (u < 0 || (u < 64 && ((sees[i] >> u) & 1ull)));
            }
#pragma unroll
            for (int j = 0; j < kTilesN; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float v;
                if constexpr (!kF8) {
                  const int col = 8 * j + 2 * t + i, ch = (col % 64) / 8;
                  const uint32_t at = (col / 64) * C::kSubBytes + key * 128 + ((ch ^ (key & 7)) << 4) + (col & 7) * 2;
                  v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(vat + at));
                } else {
                  const int col = 16 * (j / 2) + 4 * t + (j & 1) + 2 * i, ch = col / 16;
                  const uint32_t at = (D == 128 ? key * 128 + ((ch ^ (key & 7)) << 4) : key * 64 + ((ch ^ ((key >> 1) & 3)) << 4)) + (col & 15);
                  v = e4m3x2_to_f32(vat[at]).x;
                }
                if (see[0]) acc[j][i] = fmaf(e[0], v, acc[j][i]);
                if (see[1]) acc[j][2 + i] = fmaf(e[1], v, acc[j][2 + i]);
              }
          }
        }
        if (part) fence_proxy_async_smem();  // the plain stores before the next copy into the stage
      }
      __syncwarp();  // every lane has read the stage
      issue();
    }

    // ---- the four warps' states into one
    if (!ok) *abort_flag = 1u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (t == 0) {
        stat_m[warp * kTreeRows + g + 8 * i] = m[i];
        stat_l[warp * kTreeRows + g + 8 * i] = l[i];
      }
    }
    __syncthreads();
    ok = *abort_flag == 0u;  // the same for every thread until the next piece's waits
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float M = stat_m[g + 8 * i];
#pragma unroll
      for (int w = 1; w < kTreeWarps; ++w) M = fmaxf(M, stat_m[w * kTreeRows + g + 8 * i]);
      f[i] = ex2_approx(m[i] - (M == -INFINITY ? 0.f : M));
    }
    const int orow = threadIdx.x >> 3, ocol = (threadIdx.x & 7) * 4;  // of the 16 x 32 quarter
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kTreeWarps; ++w) M = fmaxf(M, stat_m[w * kTreeRows + orow]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kTreeWarps; ++w)
      L = fmaf(stat_l[w * kTreeRows + orow], ex2_approx(stat_m[w * kTreeRows + orow] - ref), L);
    int tok, head;
    const bool row_here = tree_row<kTreeRows>(p, pc.s, pc.tile, orow, &tok, &head);
    const bool whole = pc.ch0 == 0 && pc.ch1 == pc.s.nch;
    const int slot = 2 * cta + (pc.ch0 == 0 ? 1 : 0);
    const long long at = static_cast<long long>(pc.s.q0 + tok) * p.Hq + pc.h * p.G + head;
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      if (q > 0) __syncthreads();  // the quarter before has been read
      float* dst = merge + warp * kTreeRows * 32;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* row = dst + (g + 8 * i) * 32;  // its 4-column groups in the order ^ (row & 7): no bank twice
        if constexpr (!kF8) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float2*>(row + ((2 * j + t / 2) ^ g) * 4 + 2 * (t & 1)) =
                make_float2(acc[4 * q + j][2 * i] * f[i], acc[4 * q + j][2 * i + 1] * f[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float* e = acc[4 * q + 2 * j];
            const float* o = acc[4 * q + 2 * j + 1];
            *reinterpret_cast<float4*>(row + ((4 * j + t) ^ g) * 4) =
                make_float4(e[2 * i] * f[i], o[2 * i] * f[i], e[2 * i + 1] * f[i], o[2 * i + 1] * f[i]);
          }
        }
      }
      __syncthreads();
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kTreeWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(merge + (w * kTreeRows + orow) * 32 + (ocol ^ ((orow & 7) * 4)));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
      }
      if (ok && row_here) {
        if (whole) {
          *reinterpret_cast<uint2*>(p.o + at * D + 32 * q + ocol) =
              make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
        } else {
          *reinterpret_cast<float4*>(p.st_o + (static_cast<long long>(slot) * kTreeRows + orow) * D + 32 * q + ocol) = sum;
        }
      }
    }
    if (ok && row_here && ocol == 0) {
      if (whole) {
        p.lse[static_cast<long long>(pc.h * p.G + head) * p.total_q + pc.s.q0 + tok] =
            L > 0.f || L != L ? M * 0.69314718055994531f + logf(L) : -INFINITY;
      } else {
        p.st_m[slot * kTreeRows + orow] = M;
        p.st_l[slot * kTreeRows + orow] = L;
      }
    }
    if (pc.ch0 == 0 && pc.ch1 < pc.s.nch) {  // goes on in the next CTAs: the last piece of this one
      has_tail = true;
      if (threadIdx.x == 0) {
        // the CTA that holds the unit's last chunk
        p.meta[2 * cta] = make_int4(pc.s.q0, pc.s.T, pc.h, pc.tile);
        p.meta[2 * cta + 1] = make_int4(ok ? tree_owner(range, x + (pc.s.nch - pc.ch1) - 1) : -1, 0, 0, 0);
      }
    }
    __syncthreads();  // the statistics may be overwritten
    if (!ok) break;
  }
  if (!has_tail && threadIdx.x == 0) p.meta[2 * cta + 1] = make_int4(-1, 0, 0, 0);
  // after a failed wait copies may still be in flight: let them land
  if (live) {
#pragma unroll 1
    for (int s = 0; s < C::kStages; ++s)
      if ((live >> s) & 1u) mbar_wait_drain(bars + 8 * s, (phase >> s) & 1u, p.timeout_ns);
  }
}

// Units shared by several CTAs: CTA c's slot 1 holds the front of one, slot 0 of the CTAs after
// it (every fan-th), up to the one in meta, the rest.  A warp merges a row: every state is moved
// to the largest reference, the sums add in CTA order (no atomics: the same bits every time), one
// division.  Eight states are loaded at a time: a unit of one long sequence has some 40, and
// their latency is all there is (11 MB for 8 heads of two 128-row tiles, in L2).
template <int D, int kRows>
__global__ void __launch_bounds__(128) attn_tree_merge_kernel(const TreeParams p) {
  constexpr int kPer = D / 32;
  constexpr int kBatch = 8;  // states loaded together
  griddep_wait();
  griddep_launch_dependents();
  const int cta = static_cast<int>(blockIdx.x);
  const int4 unit = p.meta[2 * cta], last = p.meta[2 * cta + 1];
  if (last.x < 0) return;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  TreeSeq s;
  s.q0 = unit.x;
  s.T = unit.y;
  int tok, g;
  if (!tree_row<kRows>(p, s, unit.w, row, &tok, &g)) return;
  const int count = (last.x - cta) / p.fan + 1;
  float M = -INFINITY, L = 0.f;
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  for (int c0 = 0; c0 < count; c0 += kBatch) {
    float ms[kBatch], ls[kBatch], os[kBatch][kPer];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      ms[i] = -INFINITY;
      ls[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) os[i][k] = 0.f;
      if (c0 + i < count) {
        const long long at = static_cast<long long>(2 * (cta + (c0 + i) * p.fan) + (c0 + i == 0 ? 1 : 0)) * kRows + row;
        ms[i] = p.st_m[at];
        ls[i] = p.st_l[at];
        const float* src = p.st_o + at * D + lane * kPer;
        if constexpr (kPer == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          os[i][0] = v.x;
          os[i][1] = v.y;
          os[i][2] = v.z;
          os[i][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          os[i][0] = v.x;
          os[i][1] = v.y;
        }
      }
    }
    float mc = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) mc = fmaxf(mc, ms[i]);
    const float ref = mc == -INFINITY ? 0.f : mc;
    const float a = ex2_approx(M - ref);
    L *= a;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] *= a;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = ex2_approx(ms[i] - ref);
      L = fmaf(w, ls[i], L);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = fmaf(w, os[i][k], acc[k]);
    }
    M = mc;
  }
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  const int head = unit.z * p.G + g;
  __nv_bfloat16* dst = p.o + (static_cast<long long>(s.q0 + tok) * p.Hq + head) * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
  if (lane == 0)
    p.lse[static_cast<long long>(head) * p.total_q + s.q0 + tok] =
        L > 0.f || L != L ? M * 0.69314718055994531f + logf(L) : -INFINITY;
}

}  // namespace attn

// Attention of drafted tokens over a paged cache, units of up to 128 rows, sm_103a.
//
// The operation, units and work split of attn_tree_kernel.cuh, for calls whose drafted tokens
// and grouped heads make more rows than one 16-row tile: there every further tile reads the
// keys again and its warp-level products become the limit.  Here a tile holds the G heads of
// 128 / G tokens as the 128 lanes of tensor memory, and the products are tcgen05.mma: per
// block of 128 keys S = Q K^T (128 x 128 x d, into one of two or three score buffers) and
// o~ += P V, with P written back over S as bf16.  One CTA an SM, persistent over its range of
// the list of chunks (128 keys each).
//
// Bound: with one tile a head the keys, read once a unit (one sequence of 131072 tokens, 8 K/V
// heads with 4 query heads each, d = 128, 8 drafts, on GB300: bf16 88 us, 6.1 TB/s); with two the
// softmax, 1670 cycles for 128 x 128 scores (64 drafts: 124 us at 2070 MHz, 4.3 TB/s of keys and as
// much again from L2 for the second tile; 130 when calls go on and power holds the clock to 1730 to
// 1910).  e4m3 is bound by latency, 2840 cycles a block in two streams
// beside the widening of V: 95 us with 8 drafts; 24 sequences of 500 to 8192 tokens and up to 24
// drafts, 122 MB of keys, 62 us.
//
// Two streams: blocks of even number go to one group of four softmax warps and accumulator o~,
// odd ones to the other, so that one group's softmax covers the other's products
// and loads; each stream keeps its own (m, l, o~), combined once a piece.
//
// Warps: 0-3 and 8-11 softmax, thread r of a group owns row r (tensor-memory lane r); 4 producer
// (TMA); 5 issues P V; 6 issues S; 7 (bf16) repairs V blocks at a sequence's end, see below, or
// (e4m3) turns the scale codes of K into floats; 12-15 (e4m3) convert Q and V, thread r row r.
//
// e4m3: the codes of K go to the tensor cores as they are.  A query row, divided by the power
// of two that brings its largest finite value into [128, 256), is split into two e4m3 terms,
// q = hi + lo: 8 significant bits are 4 + 4, so the split is exact for values of 2^-9 of the row's
// largest and more, and off by at most 2^-17 of it below; S = hi K^T + lo K^T in fp32.  The row's
// power of two and each key's scale multiply the scores afterwards.  V is widened to bf16 with
// its scale, exact, and P goes in as bf16.  (V as f16 over a running exponent is two conversions
// a pair less; but a key's scale, seen by a row or not, would then decide how small a value the
// other keys may hold.)
//
// K and V blocks are up to eight boxes of 16 keys, each from the page it lies in (larger boxes
// when the page size allows: fewer copies).  A block that holds drafted keys, or keys past the
// end, or a page that does not exist, is "ragged": its V rows that must not count are zeroed
// (0 * NaN is NaN), and infinities and NaN in V of drafted keys are zeroed too and remembered:
// rows that see them get them added in the epilogue, rows that do not never meet them.
#pragma once

#include <type_traits>

#include "attn_tree_kernel.cuh"

namespace attn {

constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kTileWarpTma = 4;
constexpr int kTileWarpPv = 5;
constexpr int kTileWarpS = 6;
constexpr int kTileWarpFix = 7;
constexpr int kTileTags = 16;
// Pieces announced in shared memory.  The producer is at most 7 blocks, so at most 8 pieces, ahead
// of any role, as each is counted in what frees a stage: S in k_free (and through k_ready the
// scales' warp), P V and the repair of V or the converters in v_free, the softmax through P V.  So
// a slot is never overwritten while in use.
constexpr int kTilePieces = 16;

// A piece as the producer announces it to the other roles.
struct TileJob {
  int q0, T, ctx, n;       // the sequence's first row, drafted tokens, context and keys
  int b, h, tile, nch;
  int ch0, ch1;            // blocks; ch1 <= ch0: the end of the list
  int owner;               // the CTA with the unit's last block
  int unused;
};
static_assert(sizeof(TileJob) == 48, "three 16-byte words");

template <int D, bool kF8>
struct TileCfg {
  // (bf16 at d = 128 has no shared memory left for the second stream's statistics, and tensor
  // memory for two score buffers then; through the workspace two streams were slower, 137 us
  // against 124 for 131072 tokens and 64 drafts.)
  static constexpr int kStreams = !kF8 && D == 128 ? 1 : 2;
  static constexpr int kThreads = kF8 ? 512 : kStreams == 2 ? 384 : 256;
  static constexpr int kSub = D / 64;                    // 64-column sub-tiles of a bf16 row
  static constexpr int kSubBytes = 128 * 128;            // 128 rows x 64 bf16
  static constexpr int kTileBytes = kSub * kSubBytes;    // a block of K, V or Q in bf16
  static constexpr int kRawBytes = 128 * D;              // a block in e4m3
  // Rings: K and V blocks as they arrive, and (e4m3) V blocks in bf16
  static constexpr int kRingK = D == 64 ? 4 : 3;
  static constexpr int kRingV = kF8 ? kRingK - 1 : kRingK;
  static constexpr int kWide = kF8 ? (D == 64 ? 3 : 2) : 0;
  static constexpr int kStageK = kF8 ? kRawBytes : kTileBytes;
  static constexpr int kStageV = kStageK;
  static constexpr int kSBufs = kStreams * D + 3 * 128 <= 512 ? 3 : 2;  // what tensor memory has room for
  static constexpr int kOffQ = 0;
  static constexpr int kOffQ8 = kF8 ? kTileBytes : 0;    // e4m3: hi, then lo
  static constexpr int kOffK = kOffQ8 + kTileBytes;
  static constexpr int kOffV = kOffK + kRingK * kStageK;
  static constexpr int kOffWide = kOffV + kRingV * kStageV;
  static constexpr int kOffCodeK = kOffWide + kWide * kTileBytes;       // scale codes, 128 a stage
  static constexpr int kOffCodeV = kOffCodeK + (kF8 ? kRingK * 128 : 0);
  static constexpr int kOffScaleK = kOffCodeV + (kF8 ? kRingV * 128 : 0);  // floats, block g % 8
  static constexpr int kOffScaleQ = kOffScaleK + (kF8 ? 8 * 512 : 0);      // floats, piece u % 8
  static constexpr int kOffStat = kOffScaleQ + (kF8 ? 8 * 512 : 0);   // m, l of each stream, piece u % 2
  static constexpr int kOffBar = kOffStat + (kStreams == 2 ? 2 * 4 * 512 : 0);
  // q_full, q_free, q8_full, {k_full, k_free, k_ready}[RK], {v_full, v_free, v_fixed}[RV],
  // {w_full, w_free}[W], {s_full, pv_done, p_full}[B], drain[2], o_free, q8_free, piece[16]
  static constexpr int kNumBars = 3 + 3 * kRingK + 3 * kRingV + 2 * kWide + 3 * kSBufs + 4 + kTilePieces;
  static constexpr int kOffPieces = (kOffBar + 8 * kNumBars + 15) / 16 * 16;
  static constexpr int kOffPre = kOffPieces + kTilePieces * 48;
  static constexpr int kOffMisc = kOffPre + 8 * (kPlanGroups + 1 + 4);  // tmem base, abort, valid[16], tags[16]
  static constexpr int kSmem = kOffMisc + 8 + 64 + 4 * kTileTags + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA");
  __host__ __device__ static constexpr uint32_t col_s(int b) { return 128u * b; }
  __host__ __device__ static constexpr uint32_t col_o(int b) { return 128u * kSBufs + static_cast<uint32_t>(D) * b; }
  static constexpr uint32_t kIdescS = idesc_bf16_f32(kTileRows, kTileKeys, 0);
  // kind::f8f6f4, e4m3 x e4m3 -> fp32 (the formats' codes are 0)
  static constexpr uint32_t kIdescS8 = (1u << 4) | ((kTileKeys >> 3) << 17) | ((kTileRows >> 4) << 24);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(kTileRows, D, 1);
  static_assert(128 * kSBufs + kStreams * D <= 512, "tensor memory");
};

// mbar_wait with the part that counts time out of line: inlined at some thirty places it fills the
// instruction cache (64 sequences of 500 e4m3 tokens, 8 drafts, d = 128: 64 -> 50 us with this).
__device__ __noinline__ bool tile_wait_on(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag, uint32_t* status,
                                          unsigned long long limit_ns, uint32_t site) {
  return mbar_wait(bar, parity, WaitCtx{abort_flag, status, limit_ns}, site);
}
__device__ __forceinline__ bool tile_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, uint32_t site) {
  return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || tile_wait_on(bar, parity, w.abort_flag, w.status, w.limit_ns, site);
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::f8f6f4 (e4m3 in, fp32 accumulate), k = 32.
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Eight e4m3 codes times the scale (a bf16 pair of it) as four bf16 pairs, exact.
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi, __nv_bfloat162 scale) {
  uint4 r;
  auto one = [&](uint32_t c) {
    const uint32_t w = e4m3x2_to_bf16x2(c);
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), scale);
    return *reinterpret_cast<const uint32_t*>(&v);
  };
  r.x = one(lo & 0xffffu);
  r.y = one(lo >> 16);
  r.z = one(hi & 0xffffu);
  r.w = one(hi >> 16);
  return r;
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Infinities and NaN among the drafted values of a piece, which went into the product as zero,
// to a row that sees their keys: columns col .. col + 31 of its o~ (a positive weight leaves
// them what they are).
template <bool kF8>
__device__ __forceinline__ void tile_add_nonfinite(const TreeParams& p, const TileJob& t, unsigned long long sees, int col,
                                                   int d, uint32_t* o) {
#pragma unroll 1
  for (; sees; sees &= sees - 1) {
    const int pos = t.ctx + __ffsll(static_cast<long long>(sees)) - 1;
    if (pos >= t.n || pos / kTileKeys < t.ch0 || pos / kTileKeys >= t.ch1) continue;
    const int pg = __ldg(p.table + static_cast<long long>(t.b) * p.max_pages + pos / p.page);
    if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) continue;
    const long long at = (static_cast<long long>(pg) * p.Hkv + t.h) * p.page + pos % p.page;
    uint32_t two = 0;
    if constexpr (kF8) two = static_cast<uint32_t>(__ldg(p.vs + at)) * 0x00800080u;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      uint32_t w;
      if constexpr (kF8) {
        const uint32_t cw = e4m3x2_to_bf16x2(__ldg(reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.v) + at * d + col) + k));
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&cw), *reinterpret_cast<const __nv_bfloat162*>(&two));
        w = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.v) + at * d + col) + k);
      }
      if (any_nonfinite(w & 0xffffu)) o[2 * k] = __float_as_uint(__uint_as_float(o[2 * k]) + bf16_lo(w));
      if (any_nonfinite(w & 0xffff0000u)) o[2 * k + 1] = __float_as_uint(__uint_as_float(o[2 * k + 1]) + bf16_hi(w));
    }
  }
}

template <int D, bool kF8>
__global__ void __launch_bounds__(TileCfg<D, kF8>::kThreads, 1)
    attn_tree_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using C = TileCfg<D, kF8>;
  constexpr int RK = C::kRingK, RV = C::kRingV, NB = C::kSBufs, NW = C::kWide;
  constexpr int NWm = NW > 0 ? NW : 1;
  constexpr int ST = C::kStreams;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV;
  const uint32_t bar0 = sbase + C::kOffBar;
  const uint32_t bar_q_full = bar0, bar_q_free = bar0 + 8u, bar_q8_full = bar0 + 16u;
  auto bar_k_full = [&](int s) { return bar0 + 8u * (3 + s); };
  auto bar_k_free = [&](int s) { return bar0 + 8u * (3 + RK + s); };
  auto bar_k_ready = [&](int s) { return bar0 + 8u * (3 + 2 * RK + s); };  // e4m3: its scales are out
  auto bar_v_full = [&](int s) { return bar0 + 8u * (3 + 3 * RK + s); };
  auto bar_v_free = [&](int s) { return bar0 + 8u * (3 + 3 * RK + RV + s); };
  auto bar_v_fixed = [&](int s) { return bar0 + 8u * (3 + 3 * RK + 2 * RV + s); };
  auto bar_w_full = [&](int s) { return bar0 + 8u * (3 + 3 * RK + 3 * RV + s); };
  auto bar_w_free = [&](int s) { return bar0 + 8u * (3 + 3 * RK + 3 * RV + NW + s); };
  constexpr int kB1 = 3 + 3 * RK + 3 * RV + 2 * NW;
  auto bar_s_full = [&](int b) { return bar0 + 8u * (kB1 + b); };
  auto bar_pv_done = [&](int b) { return bar0 + 8u * (kB1 + NB + b); };
  auto bar_p_full = [&](int b) { return bar0 + 8u * (kB1 + 2 * NB + b); };
  auto bar_drain = [&](int i) { return bar0 + 8u * (kB1 + 3 * NB + i); };
  const uint32_t bar_o_free = bar0 + 8u * (kB1 + 3 * NB + 2);  // both groups have read a piece's o~
  const uint32_t bar_q8_free = bar0 + 8u * (kB1 + 3 * NB + 3);  // e4m3: hi and lo have been read
  auto bar_piece = [&](int i) { return bar0 + 8u * (kB1 + 3 * NB + 4 + i); };
  long long* pre = reinterpret_cast<long long*>(smem + C::kOffPre);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 4);
  // valid[g % 16]: which 16-key slices of block g exist (written before the block's copies are
  // announced; the producer is at most 7 blocks ahead of any role)
  volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 8);
  // tag[u % 16] = u + 1 once unit u (of this CTA) has met an infinite or NaN drafted value
  volatile uint32_t* tag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 72);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_free, kF8 ? 4 : 1);
    mbar_init(bar_q8_full, 4);
    mbar_init(bar_q8_free, 1);
    for (int s = 0; s < RK; ++s) {
      mbar_init(bar_k_full(s), 1);
      mbar_init(bar_k_free(s), 1);
      mbar_init(bar_k_ready(s), 1);
    }
    for (int s = 0; s < RV; ++s) {
      mbar_init(bar_v_full(s), 1);
      // bf16: P V, and the repair on every block, ragged or not: a warp that waits by parity must not
      // be passed by two turns of the ring
      mbar_init(bar_v_free(s), kF8 ? 4 : 2);
      mbar_init(bar_v_fixed(s), 1);
    }
    for (int s = 0; s < NW; ++s) {
      mbar_init(bar_w_full(s), 4);
      mbar_init(bar_w_free(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(bar_s_full(b), 1);
      mbar_init(bar_pv_done(b), 1);
      mbar_init(bar_p_full(b), 4);
    }
    mbar_init(bar_drain(0), 1);
    mbar_init(bar_drain(1), 1);
    mbar_init(bar_o_free, 4 * ST);
    for (int i = 0; i < kTilePieces; ++i) mbar_init(bar_piece(i), 1);
    *abort_flag = 0u;
    for (int i = 0; i < kTileTags; ++i) tag[i] = 0u;
    fence_mbar_init();
  }
  if (warp == kTileWarpPv) tmem_alloc<512>(smem_u32(tmem_slot));
  if (warp == kTileWarpTma && lane == 0) {
    tma_prefetch_desc(&tmQ);
    if (p.num_pages > 0) {  // without pages there are no maps
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
  }
  griddep_wait();
  const int gs = (p.B + kPlanGroups - 1) / kPlanGroups;
  tc_fence_before();
  tree_plan<kTileRows, kTileKeys>(p, gs, pre, pre + kPlanGroups + 1);  // ends with a barrier of the CTA
  tc_fence_after();
  // not before this CTA has its tensor memory: a later launch that got there first would hold it
  // until this one ends
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const long long W = pre[kPlanGroups];
  const int cta = static_cast<int>(blockIdx.x);
  // fan > 1: neighbouring CTAs walk the same places, each with its tile of every unit
  const TreeRange range = tree_range(W, cta / p.fan, gridDim.x / p.fan);
  const long long x0 = range.x0, x1 = range.x1;

  // Every role walks the same pieces; g counts their blocks, u the pieces themselves.  The
  // producer finds them (a search and a few global loads) and announces them to the others.
  auto job_at = [&](int u) { return reinterpret_cast<TileJob*>(smem + C::kOffPieces + (u % kTilePieces) * 48); };
  // Waits for piece u; false at the end of the list, or (ok = false too) when the wait ran out.
  auto job = [&](int u, TileJob& t, bool& ok, uint32_t site) {
    ok = tile_wait(bar_piece(u % kTilePieces), (u / kTilePieces) & 1, wc, site);
    if (!ok) return false;
    t = *job_at(u);
    return t.ch1 > t.ch0;
  };
  // The same for a whole warp: one that gives up gives up with all its lanes, whichever of them
  // the wait ran out for, so that none of them waits for another in a vote.
  auto job_warp = [&](int u, TileJob& t, bool& ok, uint32_t site) {
    const bool more = job(u, t, ok, site);
    ok = __all_sync(0xffffffffu, ok);
    return ok && more;
  };
  if (warp == kTileWarpTma) {
    // ================================================================ producer
    // with several tiles a neighbour reads the same keys a little later, or earlier
    const uint64_t pol = p.fan > 1 ? policy_evict_normal() : policy_evict_first();
    const int box16 = p.box_rows / 16;  // slices a box holds
    int g = 0, u = 0;
    uint32_t k_live = 0, k_par = 0, v_live = 0, v_par = 0;
    bool ok = true;
    // The next piece this CTA has rows and keys of, from place x on; lane i < 8 looks after slice i
    // of a block, and has the page of its slice of the piece's first one.  Pages are fetched a block
    // ahead, a piece while the one before is in flight.
    long long x = x0;
    auto page_of = [&](const TreePiece& t, int j) {
      const long long pos = static_cast<long long>(j) * kTileKeys + 16 * lane;
      const bool need = lane < 8 && j < t.ch1 && pos < t.s.n;
      return need ? __ldg(p.table + static_cast<long long>(t.b) * p.max_pages + static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page)) : -1;
    };
    auto find = [&](TreePiece& t, int& owner, int& page) {
      while (x < x1) {
        t = tree_piece<kTileRows, kTileKeys>(p, gs, pre, x, x1);
        x += t.adv;
        t.tile = t.tile * p.fan + cta % p.fan;
        if (t.ch1 <= t.ch0 || t.tile * p.tok_tile >= t.s.T) continue;
        owner = tree_owner(range, x + (t.s.nch - t.ch1) - 1) * p.fan + cta % p.fan;
        page = page_of(t, t.ch0);
        return true;
      }
      return false;
    };
    TreePiece pc, nx;
    int owner = 0, nx_owner = 0, next = -1, nx_page = -1;
    bool more = find(pc, owner, next);
    while (ok && more) {
      if (lane == 0) {
        TileJob t = {};
        t.q0 = pc.s.q0;
        t.T = pc.s.T;
        t.ctx = pc.s.ctx;
        t.n = pc.s.n;
        t.b = pc.b;
        t.h = pc.h;
        t.tile = pc.tile;
        t.nch = pc.s.nch;
        t.ch0 = pc.ch0;
        t.ch1 = pc.ch1;
        t.owner = owner;
        *job_at(u) = t;
        mbar_arrive(bar_piece(u % kTilePieces));
      }
      for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
        const int pg = next;
        next = page_of(pc, j + 1);
        const bool have = static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages);
        if (!have && lane < 8 && static_cast<long long>(j) * kTileKeys + 16 * lane < pc.s.n && p.page_word)
          atomicOr(p.page_word, 1u);
        const uint32_t vm = __ballot_sync(0xffffffffu, have && lane < 8);
        const int row = static_cast<int>((static_cast<uint32_t>(j) * kTileKeys + 16u * lane) % static_cast<uint32_t>(p.page));
        const bool mine = have && lane < 8 && lane % box16 == 0;
        const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
        constexpr int kRowB = kF8 ? D : 128;                 // bytes of a row of a (sub-)tile
        constexpr int kSubs = kF8 ? 1 : C::kSub;
        const uint32_t bytes = boxes * p.box_rows * (kSubs * kRowB + (kF8 ? 1 : 0));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int st = kv ? g % RV : g % RK;
          const uint32_t ph = ((kv ? g / RV : g / RK)) & 1, bit = 1u << st;
          ok = __all_sync(0xffffffffu, tile_wait(kv ? bar_v_free(st) : bar_k_free(st), ph ^ 1, wc, 34 + kv));
          if (!ok) break;
          const uint32_t full = kv ? bar_v_full(st) : bar_k_full(st);
          if (lane == 0 && kv == 0) valid[g & 15] = vm;
          __syncwarp();
          if (kv == 0 && j == p.fault_block) continue;  // withheld: the waits on it run out
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          if (mine) {
            const uint32_t dst = (kv ? sV + st * C::kStageV : sK + st * C::kStageK) + 16 * lane * kRowB;
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
              tma_load_4d(dst + s * C::kSubBytes, kv ? &tmV : &tmK, full, s * 64, row, pc.h, pg, pol);
            if constexpr (kF8) {
              const long long r = (static_cast<long long>(pg) * p.Hkv + pc.h) * p.page + row;
              bulk_load(sbase + (kv ? C::kOffCodeV : C::kOffCodeK) + st * 128 + 16 * lane, (kv ? p.vs : p.ks) + r,
                        p.box_rows, full);
            }
          }
          if (kv == 0) {
            k_live |= bit;
            k_par = (k_par & ~bit) | (ph << st);
          } else {
            v_live |= bit;
            v_par = (v_par & ~bit) | (ph << st);
          }
        }
        // Q after the piece's first block, whose stages depend on earlier blocks only: its K and
        // V are on their way while the last piece's products still read the old Q
        if (ok && j == pc.ch0) {
          if (u > 0) ok = __all_sync(0xffffffffu, tile_wait(bar_q_free, (u - 1) & 1, wc, 33));
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(bar_q_full, C::kSub * p.tok_tile * p.G * 128);
            for (int s = 0; s < C::kSub; ++s)
              tma_load_4d(sQ + s * C::kSubBytes, &tmQ, bar_q_full, s * 64, 0, pc.h, pc.s.q0 + pc.tile * p.tok_tile, pol);
          }
          if (ok) ++u;
        }
        if (!ok) break;
        // once there is something to wait for
        if (j == min(pc.ch0 + 2, pc.ch1 - 1)) more = find(nx, nx_owner, nx_page);
      }
      pc = nx;
      owner = nx_owner;
      next = nx_page;
    }
    if (ok && lane == 0) {  // the end of the list
      job_at(u)->ch0 = 0;
      job_at(u)->ch1 = 0;
      mbar_arrive(bar_piece(u % kTilePieces));
    }
    // let the copies in flight land before this warp leaves
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < RK; ++s)
        if ((k_live >> s) & 1u) mbar_wait_drain(bar_k_full(s), (k_par >> s) & 1u, p.timeout_ns);
#pragma unroll
      for (int s = 0; s < RV; ++s)
        if ((v_live >> s) & 1u) mbar_wait_drain(bar_v_full(s), (v_par >> s) & 1u, p.timeout_ns);
      if (u > 0) mbar_wait_drain(bar_q_full, (u - 1) & 1, p.timeout_ns);
    }
  } else if (warp == kTileWarpPv || warp == kTileWarpS) {
    // ================================================================ products
    if (lane == 0) {
      const uint32_t dhi = (1024u >> 4) | (1u << 14) | (2u << 29);
      int g = 0, u = 0;
      bool ok = true;
      uint32_t fixed_par = 0;  // parity each v_fixed completes next
      TileJob pc;
      while (job(u, pc, ok, 50)) {
        if (warp == kTileWarpS) {
          const uint32_t qlo = ((kF8 ? sbase + C::kOffQ8 : sQ) >> 4) | (1u << 16);
          const uint32_t klo = (sK >> 4) | (1u << 16);
          // e4m3 rows of 64 bytes: 64-byte swizzle, eight rows 512 bytes apart
          const uint32_t dhi8 = D == 128 ? dhi : (512u >> 4) | (1u << 14) | (4u << 29);
          ok = tile_wait(kF8 ? bar_q8_full : bar_q_full, u & 1, wc, 36);
          for (int j = pc.ch0; ok && j < pc.ch1; ++j, ++g) {
            const int st = g % RK, bf = g % NB;
            if (g >= NB) ok = tile_wait(bar_pv_done(bf), ((g - NB) / NB) & 1, wc, 37);
            ok = ok && tile_wait(kF8 ? bar_k_ready(st) : bar_k_full(st), (g / RK) & 1, wc, 38);
            if (!ok) break;
            tc_fence_after();
            const uint32_t blo = klo + st * (C::kStageK >> 4);
            const uint32_t dst = tmem + C::col_s(bf);
            if constexpr (kF8) {
#pragma unroll
              for (int part = 0; part < 2; ++part)  // hi, lo
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks)
                  mma_ss_f8(dst, (static_cast<uint64_t>(dhi8) << 32) | (qlo + part * (C::kRawBytes >> 4) + ks * 2),
                            (static_cast<uint64_t>(dhi8) << 32) | (blo + ks * 2), C::kIdescS8,
                            part + ks > 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks / 4) * (C::kSubBytes >> 4) + (ks % 4) * 2;
                mma_ss(dst, (static_cast<uint64_t>(dhi) << 32) | (qlo + off),
                       (static_cast<uint64_t>(dhi) << 32) | (blo + off), C::kIdescS, ks > 0 ? 1u : 0u);
              }
            }
            mma_commit(bar_s_full(bf));
            mma_commit(bar_k_free(st));
          }
          if (!ok) break;
          mma_commit(kF8 ? bar_q8_free : bar_q_free);
        } else {
          const uint32_t vlo = ((kF8 ? sbase + C::kOffWide : sV) >> 4) | (static_cast<uint32_t>(C::kSubBytes >> 4) << 16);
          if (u > 0) ok = tile_wait(bar_o_free, (u - 1) & 1, wc, 56);
          for (int j = pc.ch0; ok && j < pc.ch1; ++j, ++g) {
            const int st = kF8 ? g % NWm : g % RV;
            ok = kF8 ? tile_wait(bar_w_full(st), (g / NWm) & 1, wc, 39) : tile_wait(bar_v_full(st), (g / RV) & 1, wc, 39);
            if (!kF8 && ok && (static_cast<long long>(j + 1) * kTileKeys > pc.ctx || valid[g & 15] != 0xffu)) {
              ok = tile_wait(bar_v_fixed(st), (fixed_par >> st) & 1u, wc, 40);
              fixed_par ^= 1u << st;
            }
            ok = ok && mbar_wait_poll(bar_p_full(g % NB), (g / NB) & 1, wc, 41);
            if (!ok) break;
            tc_fence_after();
            const uint32_t blo = vlo + st * (C::kTileBytes >> 4);
            const uint32_t a = tmem + C::col_s(g % NB);
#pragma unroll
            for (int ks = 0; ks < kTileKeys / 16; ++ks)
              mma_ts(tmem + C::col_o(g % ST), a + ks * 8, (static_cast<uint64_t>(dhi) << 32) | (blo + ks * (16 * 128 >> 4)),
                     C::kIdescO, (j >= pc.ch0 + ST || ks > 0) ? 1u : 0u);
            mma_commit(bar_pv_done(g % NB));
            mma_commit(kF8 ? bar_w_free(st) : bar_v_free(st));
          }
          if (!ok) break;
        }
        ++u;
      }
      mma_commit(bar_drain(warp == kTileWarpS));
      mbar_wait_drain(bar_drain(warp == kTileWarpS), 0, p.timeout_ns);
    }
  } else if (warp == kTileWarpFix) {
    // ================================================================ ragged blocks of V (bf16)
    if constexpr (kF8) {
      // ---- scales of K's keys as floats, four a lane.  Entry g % 8: block g's stage was freed
      // by S of block g - 4, which is at most 3 blocks ahead of the softmax.
      int g = 0, u = 0;
      bool ok = true;
      TileJob pc;
      while (job_warp(u, pc, ok, 51)) {
        ++u;
        for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
          const int st = g % RK;
          ok = __all_sync(0xffffffffu, tile_wait(bar_k_full(st), (g / RK) & 1, wc, 44));
          if (!ok) break;
          const uint32_t w = *reinterpret_cast<const volatile uint32_t*>(smem + C::kOffCodeK + st * 128 + lane * 4);
          // at least 2^-126: a masked score, -inf, must stay that whatever the code beside it
          reinterpret_cast<float4*>(smem + C::kOffScaleK)[(g & 7) * 32 + lane] =
              make_float4(scale_of(max(w & 0xffu, 1u)), scale_of(max((w >> 8) & 0xffu, 1u)),
                          scale_of(max((w >> 16) & 0xffu, 1u)), scale_of(max(w >> 24, 1u)));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_k_ready(st));
        }
        if (!ok) break;
      }
    } else {
      int g = 0, u = 0;
      bool ok = true;
      TileJob pc;
      while (job_warp(u, pc, ok, 52)) {
        for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
          const int st = g % RV, kb = j * kTileKeys;
          ok = __all_sync(0xffffffffu, tile_wait(bar_v_full(st), (g / RV) & 1, wc, 42));
          if (!ok) break;
          const uint32_t vm = valid[g & 15];
          if (static_cast<long long>(kb) + kTileKeys <= pc.ctx && vm == 0xffu) {
            if (lane == 0) mbar_arrive(bar_v_free(st));
            continue;
          }
          bool odd = false;
          for (int i = lane; i < kTileKeys * (D / 8); i += 32) {
            const int r = i / (D / 8), ch = i % (D / 8);
            const bool here = ((vm >> (r / 16)) & 1u) && kb + r < pc.n;
            if (here && kb + r < pc.ctx) continue;
            uint4* at = reinterpret_cast<uint4*>(smem + C::kOffV + st * C::kTileBytes + (ch / 8) * C::kSubBytes + r * 128 +
                                                 (((ch & 7) ^ (r & 7)) << 4));
            if (!here) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 v = *at;
              if (any_nonfinite(v.x) || any_nonfinite(v.y) || any_nonfinite(v.z) || any_nonfinite(v.w)) {
                *at = make_uint4(finite_only(v.x), finite_only(v.y), finite_only(v.z), finite_only(v.w));
                odd = true;
              }
            }
          }
          if (odd) tag[u % kTileTags] = u + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_v_fixed(st));
            mbar_arrive(bar_v_free(st));
          }
        }
        if (!ok) break;
        ++u;
      }
    }
  } else if (kF8 && warp >= 12) {
    // ================================================================ e4m3 -> bf16
    if constexpr (kF8) {
      // Loops over a row's chunks stay rolled: this role's code next to the softmax's overflows
      // the instruction cache when unrolled (measured on GB300, one sequence of 131072 tokens,
      // d = 128: 144 us with 8 chunks unrolled, a third of the stalls for want of instructions).
      const int r = threadIdx.x - 384;  // row of Q, key of a block
      int g = 0, u = 0;
      bool ok = true;
      TileJob pc;
      while (job_warp(u, pc, ok, 53)) {
        // ---- Q: a row's largest value, then its two terms
        ok = tile_wait(bar_q_full, u & 1, wc, 43) && (u == 0 || tile_wait(bar_q8_free, (u - 1) & 1, wc, 57));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // Four threads a row, 8 columns at a time, rows that exist only; rolled, as the code runs once a
        // piece: unrolled, 8 KB, it took 7000 cycles, most of them waiting for instructions.
        const int rows = min(pc.T - pc.tile * p.tok_tile, p.tok_tile) * p.G;
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += 32) {
          const int qr = r0 + 8 * (warp - 12) + (lane >> 2);
          auto q_at = [&](int ch) {
            return *reinterpret_cast<const uint4*>(smem + C::kOffQ + (ch / 8) * C::kSubBytes + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4));
          };
          uint32_t mx = 0;  // largest finite magnitude; bit 31: one is not
#pragma unroll 1
          for (int ch = lane & 3; ch < D / 8; ch += 4) {
            const uint4 q = q_at(ch);
            mx = max(mx, finite_max(q));
            if (any_nonfinite(q.x) || any_nonfinite(q.y) || any_nonfinite(q.z) || any_nonfinite(q.w)) mx |= 0x80000000u;
          }
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const uint32_t ef = min(max((mx & 0x7fffffffu) >> 7, 8u), 253u);  // exponent field of the row's largest value
          const float up = __uint_as_float((261u - ef) << 23);  // 2^(7 - (ef - 127))
          // The row's factor, finite and more than 0, since a masked score is -inf before it is
          // multiplied: where the product leaves fp32, its least number, off by 2^-149 of a score
          // under 2^128.  Its sign says that the row holds an infinity or NaN.
          if ((lane & 3) == 0) {
            const float f = fmaxf(p.c * __uint_as_float((ef - 7u) << 23), __uint_as_float(1u));
            reinterpret_cast<float*>(smem + C::kOffScaleQ)[(u & 7) * 128 + qr] = (mx >> 31) == 0u ? f : -f;
          }
#pragma unroll 1
          for (int ch = lane & 3; ch < D / 8; ch += 4) {
            const uint4 q = q_at(ch);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // four values each
              const float f0 = bf16_lo(w[2 * i]) * up, f1 = bf16_hi(w[2 * i]) * up;
              const float f2 = bf16_lo(w[2 * i + 1]) * up, f3 = bf16_hi(w[2 * i + 1]) * up;
              const uint32_t h0 = pack_e4m3x2(f0, f1), h1 = pack_e4m3x2(f2, f3);
              const float2 b0 = e4m3x2_to_f32(h0), b1 = e4m3x2_to_f32(h1);
              hi[i] = h0 | (h1 << 16);
              lo[i] = pack_e4m3x2(f0 - b0.x, f1 - b0.y) | (pack_e4m3x2(f2 - b1.x, f3 - b1.y) << 16);
            }
            const int sw = D == 128 ? (ch >> 1) ^ (qr & 7) : (ch >> 1) ^ ((qr >> 1) & 3);
            uint8_t* to = smem + C::kOffQ8 + qr * D + (sw << 4) + (ch & 1) * 8;
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to + C::kRawBytes) = make_uint2(lo[0], lo[1]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_q8_full);
          mbar_arrive(bar_q_free);
        }
        for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
          const int sv = g % RV, sw = g % NWm, kb = j * kTileKeys;
          // ---- V: codes times scale as bf16
          ok = tile_wait(bar_v_full(sv), (g / RV) & 1, wc, 45) && tile_wait(bar_w_free(sw), ((g / NWm) & 1) ^ 1, wc, 46);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t vm = valid[g & 15];
          const bool here = ((vm >> (r / 16)) & 1u) && kb + r < pc.n;
          const bool scan = kb + r >= pc.ctx;
          const uint8_t* src = smem + C::kOffV + sv * C::kStageV + r * D;
          uint8_t* dst = smem + C::kOffWide + sw * C::kTileBytes + r * 128;
          const uint32_t code = smem[C::kOffCodeV + sv * 128 + r];
          const uint32_t two = (code << 7) | (code << 23);  // 2^(code - 127) twice, as bf16
          const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&two);
          const bool ragged = __any_sync(0xffffffffu, !here || scan);
          bool odd = false;
#pragma unroll 2
          for (int c = 0; c < D / 16; ++c) {
            const uint4 raw = *reinterpret_cast<const uint4*>(src + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
            uint4 a = widen8(raw.x, raw.y, scale), b = widen8(raw.z, raw.w, scale);
            if (ragged) {
              // rows that do not exist, and (remembered) what is not finite among the drafted, become 0
              uint32_t* w[2] = {&a.x, &b.x};
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                uint32_t& e = w[i >> 2][i & 3];
                if (here && scan && any_nonfinite(e)) odd = true;
                if (!here) e = 0u;
                if (scan) e = finite_only(e);
              }
            }
            // 16 columns = chunks 2 c, 2 c + 1 of the wide row, in sub-tile c / 4
            uint8_t* to = dst + (c / 4) * C::kSubBytes;
            const int ch = (2 * c) & 7;
            *reinterpret_cast<uint4*>(to + ((ch ^ (r & 7)) << 4)) = a;
            *reinterpret_cast<uint4*>(to + (((ch + 1) ^ (r & 7)) << 4)) = b;
          }
          if (odd) tag[u % kTileTags] = u + 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_w_full(sw));
            mbar_arrive(bar_v_free(sv));
          }
        }
        if (!ok) break;
        ++u;
      }
    }
  } else {
    // ================================================================ softmax
    const int wg = warp >= 8 ? 1 : 0;           // stream: blocks g with g % ST == wg
    const int r = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float c = p.c;  // e4m3: times the row's power of two, piece by piece
    bool odd_q = false;  // e4m3: the row's query is not finite
    constexpr float kTau = 8.f;  // o~ is rescaled when the max rises by more (log2 units)
    int g = 0, u = 0;
    bool ok = true, has_tail = false;
    // The next piece and this thread's row of it are looked up while the last product of the
    // piece in hand runs.
    TileJob pc;
    int tok = 0, head = 0;
    bool row_here = false;
    unsigned long long sees = 0;
    auto look = [&](int v) {
      if (!job_warp(v, pc, ok, 54)) return false;
      const int t = r / p.G;
      head = r - t * p.G;
      tok = pc.tile * p.tok_tile + t;
      row_here = tok < pc.T && t < p.tok_tile;
      TreeSeq sq;
      sq.q0 = pc.q0;
      sq.T = pc.T;
      sees = row_here ? tree_sees(p, sq, tok) : 0ull;
      return true;
    };
    bool more = look(0);
    // warps that gave up here would be missing at the streams' barrier below
    if (ST == 2 && bar_sync_or(1, 256, !ok)) ok = false;
    while (__all_sync(0xffffffffu, ok && more)) {
      const bool idle = !__any_sync(0xffffffffu, row_here);  // no row of this warp exists
      bool any = false;  // this stream has had a block of the piece
      float m = -INFINITY, l = 0.f;
      for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
        if (g % ST != wg) continue;
        const int bf = g % NB;
        const uint32_t colS = C::col_s(bf), colO = C::col_o(wg);
        ok = __all_sync(0xffffffffu, tile_wait(bar_s_full(bf), (g / NB) & 1, wc, 47));
        if (!ok) break;
        const bool first = !any;
        any = true;
        if (kF8 && first) {
          c = reinterpret_cast<const volatile float*>(smem + C::kOffScaleQ)[(u & 7) * 128 + r];
          odd_q = c < 0.f;
          c = fabsf(c);
        }
        if (idle) {  // its lanes of P hold scores: rows nobody reads
          if (lane == 0) mbar_arrive(bar_p_full(bf));
          continue;
        }
        tc_fence_after();
        const int kb = j * kTileKeys;
        const uint32_t vm = valid[g & 15];
        if (static_cast<long long>(kb) + kTileKeys > pc.ctx || vm != 0xffu) {
          // a ragged block: the scores of keys this row does not see become -inf where they lie
          const int off = pc.ctx - kb;  // context keys of the block; the drafted ones follow
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            const int o = off - 32 * w;
            uint32_t see = o >= 32 ? 0xffffffffu : o <= 0 ? 0u : (1u << o) - 1u;
            if (o < 32 && o > -64) see |= static_cast<uint32_t>(o >= 0 ? sees << o : sees >> -o);
            if (!((vm >> (2 * w)) & 1u)) see &= 0xffff0000u;
            if (!((vm >> (2 * w + 1)) & 1u)) see &= 0x0000ffffu;
            uint32_t e[32];
            tmem_ld32(tl + colS + 32 * w, e);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((see >> k) & 1u)) e[k] = 0xff800000u;
            tmem_st32(tl + colS + 32 * w, e);
          }
          tmem_wait_st();
        }
        const float4* ks = reinterpret_cast<const float4*>(smem + C::kOffScaleK + (g & 7) * 512);
        // A row's 128 scores go 32 at a time (64 with one stream, where nothing else covers the
        // loads), loaded twice, for the maximum and for the exponentials, in rolled loops: unrolled
        // they are code enough for the instruction cache to be the limit, cold at a launch's start
        // and beside the converters' code.
        constexpr int CW = ST == 1 ? 64 : 32;
        auto scores = [&](int q, float* s, auto raw) {  // CW scores (raw, e4m3: times their keys' scales)
          uint32_t e[CW];
#pragma unroll
          for (int i = 0; i < CW / 32; ++i) tmem_ld32(tl + colS + q * CW + 32 * i, e + 32 * i);
          if constexpr (kF8 && decltype(raw)::value) {
            float4 f[CW / 4];
#pragma unroll
            for (int k = 0; k < CW / 4; ++k) f[k] = ks[q * (CW / 4) + k];
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < CW / 4; ++k) {
              const float2 a = __fmul2_rn(make_float2(__uint_as_float(e[4 * k]), __uint_as_float(e[4 * k + 1])),
                                          make_float2(f[k].x, f[k].y));
              const float2 b = __fmul2_rn(make_float2(__uint_as_float(e[4 * k + 2]), __uint_as_float(e[4 * k + 3])),
                                          make_float2(f[k].z, f[k].w));
              s[4 * k] = a.x;
              s[4 * k + 1] = a.y;
              s[4 * k + 2] = b.x;
              s[4 * k + 3] = b.y;
            }
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < CW; ++k) s[k] = __uint_as_float(e[k]);
          }
        };
        float mx = -INFINITY;
        float s[CW];
#pragma unroll 1
        for (int q = 0; q < kTileKeys / CW; ++q) {
          scores(q, s, std::true_type{});
          if constexpr (kF8) {  // scaled, for the second pass
            uint32_t e[CW];
#pragma unroll
            for (int k = 0; k < CW; ++k) e[k] = __float_as_uint(s[k]);
#pragma unroll
            for (int i = 0; i < CW / 32; ++i) tmem_st32(tl + colS + q * CW + 32 * i, e + 32 * i);
          }
          float a[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = fmaxf(s[2 * i], s[2 * i + 1]);
#pragma unroll
          for (int k = 8; k < CW; k += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = fmax3(a[i], s[k + 2 * i], s[k + 2 * i + 1]);
          mx = fmax3(mx, fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
        }
        if constexpr (kF8) tmem_wait_st();
        mx *= c;
        const float m_new = mx > m + kTau ? mx : m;
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2_approx(m - ref);
        l *= alpha;
        const bool moved = m_new != m;
        m = m_new;
        const float2 c2 = make_float2(c, c), nm2 = make_float2(-ref, -ref);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int q = 0; q < kTileKeys / CW; ++q) {
          scores(q, s, std::false_type{});
#pragma unroll
          for (int i = 0; i < CW / 32; ++i) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 e = __ffma2_rn(make_float2(s[32 * i + 2 * k], s[32 * i + 2 * k + 1]), c2, nm2);
              e.x = ex2_approx(e.x);
              e.y = ex2_approx(e.y);
              if (k & 1)
                acc1 = __fadd2_rn(acc1, e);
              else
                acc0 = __fadd2_rn(acc0, e);
              pk[k] = pack_bf16x2(e.x, e.y);  // P rounds once, relative 2^-8 at most
            }
            // over S: columns CW / 2 q .. of the buffer held scores that are used by now
            tmem_st16(tl + colS + q * (CW / 2) + 16 * i, pk);
          }
        }
        const float2 acc = __fadd2_rn(acc0, acc1);
        l += acc.x + acc.y;
        if (!first && __any_sync(0xffffffffu, moved)) {
          // o~ may be touched once the stream's last P V, of block g - ST, is in it.  With as many
          // score buffers as streams it is: S of this block came after it.
          if (NB > ST) ok = __all_sync(0xffffffffu, tile_wait(bar_pv_done((g - ST) % NB), ((g - ST) / NB) & 1, wc, 48));
          if (!ok) break;
          if (NB > ST) tc_fence_after();
          const float2 al2 = make_float2(alpha, alpha);
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tl + colO + q * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), al2);
              o[2 * k] = __float_as_uint(v.x);
              o[2 * k + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tl + colO + q * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full(bf));
      }
      // such a row is NaN once it has seen a key (its two terms, saturated, made finite scores)
      if (kF8 && odd_q && m != -INFINITY) l = __uint_as_float(0x7fffffffu);
      const bool whole = pc.ch0 == 0 && pc.ch1 == pc.nch;
      const bool front = pc.ch0 == 0 && !whole;  // goes on in the next CTAs
      const int hq = pc.h * p.G + head;
      const long long orow = static_cast<long long>(pc.q0 + tok) * p.Hq + hq;
      const long long lrow = static_cast<long long>(hq) * p.total_q + pc.q0 + tok;
      const long long at = static_cast<long long>(2 * cta + (pc.ch0 == 0 ? 1 : 0)) * kTileRows + r;
      const TileJob done = pc;
      const bool row_done = row_here;
      const unsigned long long saw = sees;
      const int count = pc.ch1 - pc.ch0, g_end = g;
      if (ok) more = look(u + 1);
      // ---- o~ out: this stream's last P V of the piece has landed
      if (ok && any) {
        const int gl = (g_end - 1) % ST == wg ? g_end - 1 : g_end - 2;
        ok = __all_sync(0xffffffffu, tile_wait(bar_pv_done(gl % NB), (gl / NB) & 1, wc, 49));
      }
      // Both streams' statistics, then every thread has half the columns of its row.  Each of the
      // eight warps comes here once a piece, also after a failed wait, and they leave together.
      float mo = -INFINITY, lo = 0.f;             // the other stream's
      if constexpr (ST == 2) {
        float* stat = reinterpret_cast<float*>(smem + C::kOffStat) + (u & 1) * 512;
        stat[wg * 256 + r] = m;
        stat[wg * 256 + 128 + r] = l;
        if (bar_sync_or(1, 256, !ok || *abort_flag != 0u)) {
          ok = false;
          break;
        }
        mo = stat[(wg ^ 1) * 256 + r];
        lo = stat[(wg ^ 1) * 256 + 128 + r];
      } else if (!ok) {
        break;
      }
      tc_fence_after();
      const float M = fmaxf(m, mo);
      const float refM = M == -INFINITY ? 0.f : M;
      const float fown = ex2_approx(m - refM), foth = ex2_approx(mo - refM);
      const float L = l * fown + lo * foth;
      if (!idle) {
        const float inv = whole ? (L > 0.f || L != L ? 1.f / L : 0.f) : 1.f;
        const float f0 = (wg == 0 ? fown : foth) * inv, f1 = (wg == 0 ? foth : fown) * inv;
        // an accumulator no block has written holds anything
        const bool has0 = count >= ST || (g_end - 1) % ST == 0, has1 = ST == 2 && (count > 1 || ((g_end - 1) & 1) == 1);
        const bool odd = tag[u % kTileTags] == static_cast<uint32_t>(u + 1);
#pragma unroll 1
        for (int q = wg * (D / 32 / ST); q < (wg + 1) * (D / 32 / ST); ++q) {
          uint32_t o[32], w[32];
          tmem_ld32(tl + C::col_o(0) + q * 32, o);
          if constexpr (ST == 2) tmem_ld32(tl + C::col_o(1) + q * 32, w);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            float v = has0 ? __uint_as_float(o[k]) * f0 : 0.f;
            if (ST == 2 && has1) v = fmaf(__uint_as_float(w[k]), f1, v);
            o[k] = __float_as_uint(v);
          }
          if (odd) tile_add_nonfinite<kF8>(p, done, saw, q * 32, D, o);
          if (row_done && whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + orow * D + q * 32);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[i] = pack_bf16x2(__uint_as_float(o[8 * k + 2 * i]), __uint_as_float(o[8 * k + 2 * i + 1]));
              dst[k] = make_uint4(v[0], v[1], v[2], v[3]);
            }
          } else if (row_done) {
            uint4* dst = reinterpret_cast<uint4*>(p.st_o + at * D + q * 32);
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        if (row_done && wg == 0) {
          if (whole) {
            p.lse[lrow] = L > 0.f || L != L ? M * 0.69314718055994531f + logf(L) : -INFINITY;
          } else {
            p.st_m[at] = M;
            p.st_l[at] = L;
          }
        }
      }
      // both accumulators have been read by this warp: the next piece's products may write them
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_o_free);
      if (front) {
        has_tail = true;
        if (wg == 0 && r == 0) {
          p.meta[2 * cta] = make_int4(done.q0, done.T, done.h, done.tile);
          p.meta[2 * cta + 1] = make_int4(done.owner, 0, 0, 0);
        }
      }
      ++u;
    }
    if (!has_tail && wg == 0 && r == 0) p.meta[2 * cta + 1] = make_int4(-1, 0, 0, 0);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kTileWarpPv) {
    tc_fence_after();
    tmem_dealloc<512>(*reinterpret_cast<volatile uint32_t*>(tmem_slot));
  }
}

}  // namespace attn

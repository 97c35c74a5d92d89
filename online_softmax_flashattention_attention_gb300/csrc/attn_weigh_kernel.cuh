// Attention weight that cached keys receive from a call's queries, sm_103a.
//
// Sequence b has ctx_b cached tokens and T_b new ones at positions ctx_b .. ctx_b + T_b - 1, whose
// queries have been through the attention already: LSE is theirs.  Row (t, g) of K/V head h, query
// head h G + g of token t, sees position p <= ctx_b + t, and
//   out[p] = decay * weights[p] + sum over the rows that see p of exp(scale q . k_p - LSE),
// where positions from ctx_b on start from 0.  A row that saw nothing (LSE = -infinity) adds nothing.
//
// Scores are computed with keys as rows, S = K Q^T: 128 keys are the lanes of tensor memory, up to
// 128 query rows its columns.  A thread then owns a key, and the sum it wants runs along its own
// lane: no maximum, no exchange between threads, no second product.  A unit is (sequence, K/V head,
// 128 keys); nobody else touches its keys, so nothing is added atomically.  Its keys are loaded once
// and stay in shared memory while the queries stream by (a prompt), or the keys stream and the few
// queries come along (decoding).
//
// Units lie rank major, a sequence's tiles of keys by position and a tile's heads together: with
// many queries the first keys are seen by most, so each sequence's units go from long to short, and
// the CTAs (one an SM, persistent) take them in a snake.
//
// Warps: 0 finds units, looks their pages up (four units at a time, 8 slices of 16 keys each) and loads
// K; 1 loads Q; 2 issues the products; 4-7 bring the columns' LSE, warp 4 + i for score buffer i;
// 8-15 are two groups of four that take the tiles in turn, thread r of a group key r; 16-19 (e4m3)
// widen K to bf16 with its scale, exact, so that the products are the same for both caches.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tree_tile_kernel.cuh"

namespace attn {

constexpr int kWeighKeys = 128;     // of a unit
constexpr int kWeighCols = 128;     // query rows of a tile, at most
constexpr int kWeighGroups = 64;    // prefix-sum entries (each over ceil(B / 64) sequences)
constexpr int kWeighBufs = 4;       // score buffers of tensor memory
// Units announced in shared memory.  The first warp is at most kRingK + kWide <= 10 units ahead of the
// products; these are at most three tiles, so three units, ahead of the tile that a summing or LSE warp
// is at, and such a warp's last tile lies at most four before: 17 units, so that a slot is never
// overwritten while in use.
constexpr int kWeighJobs = 32;
constexpr int kWeighParts = 8;      // sums on their way from one group to the other

struct WeighParams {
  const float* lse;          // [Hq, total_q]
  const uint8_t* ks;         // the keys' scale codes, e4m3 only
  const float* w;            // [num_pages, Hkv, page]; not read when decay == 0
  float* out;                // the same
  const int32_t* table;      // [B, max_pages]
  const int32_t* cu;         // [B + 1]
  const int32_t* ctx;        // [B] or null
  int B, Hkv, G, total_q;
  int num_pages, page, max_pages, cap;
  int box_rows;              // keys a copy takes: 16 .. 128, divides the page
  int heads;                 // heads of the group in a tile of query rows (G, or 128 of more)
  int tokens;                // tokens of a full tile: 128 / heads
  int small_tokens;          // tokens of a small copy of Q (as many as make whole groups of 8 rows)
  float c;                   // scale * log2(e)
  float decay;
  uint32_t* status;
  uint32_t* page_word;
  unsigned long long timeout_ns;
};

// A sequence, every field clamped to what the buffers hold.
struct WeighSeq {
  int q0, T, ctx, n, tiles;
};
__device__ __forceinline__ WeighSeq weigh_seq(const WeighParams& p, int b) {
  WeighSeq s;
  s.q0 = min(max(__ldg(p.cu + b), 0), p.total_q);
  s.T = min(max(__ldg(p.cu + b + 1), s.q0), p.total_q) - s.q0;
  s.ctx = p.ctx ? min(max(__ldg(p.ctx + b), 0), p.cap) : 0;
  s.n = static_cast<int>(min(static_cast<long long>(s.ctx) + s.T, static_cast<long long>(p.cap)));
  s.tiles = s.T > 0 ? s.n / kWeighKeys + (s.n % kWeighKeys != 0) : 0;
  return s;
}

// A unit as the first warp announces it.
struct WeighJob {
  int q0, T, ctx, n;
  int h, tile;
  int first;               // the first token that sees any key of the unit
  int nq;                  // tiles of query rows; < 0: the end
  int pages[8];            // of the unit's slices of 16 keys, -1 without one
};
static_assert(sizeof(WeighJob) == 64, "four 16-byte words");

// Columns of tile j of a unit: tokens [tok, tok + n) with heads [head, head + p.heads) of the group.
struct WeighCols {
  int tok, head, n;
};
__device__ __forceinline__ WeighCols weigh_cols(const WeighParams& p, const WeighJob& t, int j) {
  WeighCols c;
  if (p.heads == p.G) {
    c.tok = t.first + j * p.tokens;
    c.head = 0;
    c.n = min(p.tokens, t.T - c.tok) * p.heads;
  } else {  // more than 128 heads a group: a token, 128 heads at a time
    const int per = (p.G + p.heads - 1) / p.heads;
    c.tok = t.first + j / per;
    c.head = (j % per) * p.heads;
    c.n = min(p.heads, p.G - c.head);
  }
  return c;
}

template <int D, bool kF8>
struct WeighCfg {
  static constexpr int kThreads = kF8 ? 640 : 512;
  static constexpr int kSub = D / 64;
  static constexpr int kSubBytes = 128 * 128;            // 128 rows x 64 bf16
  static constexpr int kTileBytes = kSub * kSubBytes;    // 128 rows in bf16
  static constexpr int kStageK = kF8 ? 128 * D : kTileBytes;
  static constexpr int kRingK = kF8 ? (D == 128 ? 5 : 8) : (D == 128 ? 3 : 6);
  static constexpr int kWide = kF8 ? 2 : 0;              // widened tiles of keys
  static constexpr int kRingQ = kF8 ? (D == 128 ? 2 : 4) : (D == 128 ? 3 : 5);
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kRingQ * kTileBytes;
  static constexpr int kOffWide = kOffK + kRingK * kStageK;
  static constexpr int kOffCode = kOffWide + kWide * kTileBytes;            // scale codes, 128 a stage
  static constexpr int kOffLse = kOffCode + (kF8 ? kRingK * 128 : 0);       // 128 floats a score buffer
  static constexpr int kOffPart = kOffLse + kWeighBufs * 512;               // 128 floats a part
  static constexpr int kOffJobs = kOffPart + kWeighParts * 512;
  static constexpr int kOffPre = kOffJobs + kWeighJobs * 64;
  static constexpr int kOffBar = kOffPre + 8 * (kWeighGroups + 1 + 3);
  // job[J], {k_full, k_free}[RK], {w_full, w_free}[W], {q_full, q_free}[RQ], {s_full, s_free, lse_full}[4],
  // part_full[P], drain
  static constexpr int kNumBars = kWeighJobs + 2 * kRingK + 2 * kWide + 2 * kRingQ + 3 * kWeighBufs + kWeighParts + 1;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;                   // tmem base, abort, odd[4]
  static constexpr int kSmem = kOffMisc + 24 + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <int D, bool kF8>
__global__ void __launch_bounds__(WeighCfg<D, kF8>::kThreads, 1)
    attn_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQs,
                      const __grid_constant__ CUtensorMap tmK, const WeighParams p) {
  using C = WeighCfg<D, kF8>;
  constexpr int RK = C::kRingK, RQ = C::kRingQ, NW = C::kWide, NWm = NW > 0 ? NW : 1, NB = kWeighBufs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem), sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, bar0 = sbase + C::kOffBar;
  auto bar_job = [&](int i) { return bar0 + 8u * i; };
  auto bar_k_full = [&](int s) { return bar0 + 8u * (kWeighJobs + s); };
  auto bar_k_free = [&](int s) { return bar0 + 8u * (kWeighJobs + RK + s); };
  constexpr int kB1 = kWeighJobs + 2 * RK;
  auto bar_w_full = [&](int s) { return bar0 + 8u * (kB1 + s); };
  auto bar_w_free = [&](int s) { return bar0 + 8u * (kB1 + NW + s); };
  constexpr int kB2 = kB1 + 2 * NW;
  auto bar_q_full = [&](int s) { return bar0 + 8u * (kB2 + s); };
  auto bar_q_free = [&](int s) { return bar0 + 8u * (kB2 + RQ + s); };
  constexpr int kB3 = kB2 + 2 * RQ;
  auto bar_s_full = [&](int b) { return bar0 + 8u * (kB3 + b); };
  auto bar_s_free = [&](int b) { return bar0 + 8u * (kB3 + NB + b); };
  auto bar_lse = [&](int b) { return bar0 + 8u * (kB3 + 2 * NB + b); };
  auto bar_part = [&](int i) { return bar0 + 8u * (kB3 + 3 * NB + i); };
  const uint32_t bar_drain = bar0 + 8u * (kB3 + 3 * NB + kWeighParts);
  long long* pre = reinterpret_cast<long long*>(smem + C::kOffPre);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 4);
  // odd[b]: a column of score buffer b adds nothing whatever its scores are
  volatile uint32_t* odd = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWeighJobs; ++i) mbar_init(bar_job(i), 1);
    for (int s = 0; s < RK; ++s) {
      mbar_init(bar_k_full(s), 1);
      mbar_init(bar_k_free(s), kF8 ? 4 : 1);
    }
    for (int s = 0; s < NW; ++s) {
      mbar_init(bar_w_full(s), 4);
      mbar_init(bar_w_free(s), 1);
    }
    for (int s = 0; s < RQ; ++s) {
      mbar_init(bar_q_full(s), 1);
      mbar_init(bar_q_free(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(bar_s_full(b), 1);
      mbar_init(bar_s_free(b), 4);
      mbar_init(bar_lse(b), 1);
    }
    for (int i = 0; i < kWeighParts; ++i) mbar_init(bar_part(i), 4);
    mbar_init(bar_drain, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc<512>(smem_u32(tmem_slot));
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmQs);
    if (p.num_pages > 0) tma_prefetch_desc(&tmK);  // without pages there is no map
  }
  griddep_wait();
  // units of the sequences before group i (groups of gs sequences)
  const int gs = (p.B + kWeighGroups - 1) / kWeighGroups;
  {
    long long* warp_sums = pre + kWeighGroups + 1;
    long long sum = 0;
    if (threadIdx.x < kWeighGroups) {
      const long long first = static_cast<long long>(threadIdx.x) * gs;
      for (long long b = first; b < min(first + gs, static_cast<long long>(p.B)); ++b) {
        const WeighSeq s = weigh_seq(p, static_cast<int>(b));
        sum += static_cast<long long>(s.tiles) * p.Hkv;
        if (blockIdx.x == 0 && s.T > 0 && p.page_word && static_cast<long long>(s.ctx) + s.T > p.cap) atomicOr(p.page_word, 1u);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) warp_sums[warp] = sum;
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < kWeighGroups) {
      if (warp == 1) sum += warp_sums[0];
      pre[threadIdx.x + 1] = sum;
      if (threadIdx.x == 0) pre[0] = 0;
    }
    __syncthreads();
    tc_fence_after();
  }
  // not before this CTA has its tensor memory: a later launch that got there first would hold it
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  auto job_at = [&](int u) { return reinterpret_cast<WeighJob*>(smem + C::kOffJobs + (u % kWeighJobs) * 64); };
  // Unit u, for a whole warp (one that gives up gives up with all its lanes); false at the end of the
  // list, or (ok = false too) when the wait ran out.
  auto job = [&](int u, WeighJob& t, bool& ok, uint32_t site) {
    ok = __all_sync(0xffffffffu, tile_wait(bar_job(u % kWeighJobs), (u / kWeighJobs) & 1, wc, site));
    if (!ok) return false;
    t = *job_at(u);
    return t.nq >= 0;
  };

  if (warp == 0) {
    // ================================================================ units, K
    const uint64_t pol = policy_evict_first();
    const long long U = pre[kWeighGroups];
    const int box16 = p.box_rows / 16;
    int u = 0;
    uint32_t live = 0, par = 0;
    bool ok = true;
    for (long long r0 = 0; ok; r0 += 4) {
      // lane 8 i + s: unit r0 + i of this CTA, slice s
      const long long r = r0 + lane / 8;
      const long long unit = r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      WeighJob t = {};
      int page = -1, row = 0;
      bool need = false;
      if (unit < U) {
        int lo = 0, hi = kWeighGroups;  // pre[lo] <= unit < pre[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (pre[mid] <= unit)
            lo = mid;
          else
            hi = mid;
        }
        long long y = unit - pre[lo];
        int b = lo * gs;
        WeighSeq s = weigh_seq(p, b);
        while (y >= static_cast<long long>(s.tiles) * p.Hkv && b + 1 < p.B) {
          y -= static_cast<long long>(s.tiles) * p.Hkv;
          s = weigh_seq(p, ++b);
        }
        t.q0 = s.q0;
        t.T = s.T;
        t.ctx = s.ctx;
        t.n = s.n;
        t.tile = static_cast<int>(y / p.Hkv);
        t.h = static_cast<int>(y - static_cast<long long>(t.tile) * p.Hkv);
        t.first = max(0, t.tile * kWeighKeys - s.ctx);
        t.nq = p.heads == p.G ? (s.T - t.first + p.tokens - 1) / p.tokens : (s.T - t.first) * ((p.G + p.heads - 1) / p.heads);
        const int pos = t.tile * kWeighKeys + 16 * (lane & 7);
        need = pos < s.n;
        if (need) {
          const int slot = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page);
          page = __ldg(p.table + static_cast<long long>(b) * p.max_pages + slot);
          row = pos - slot * p.page;
        }
      }
      const bool have = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages);
      if (need && !have && p.page_word) atomicOr(p.page_word, 1u);
      const bool mine = have && (lane & 7) % box16 == 0;
      const uint32_t boxes = __ballot_sync(0xffffffffu, mine);
      const uint32_t units = __ballot_sync(0xffffffffu, unit < U && (lane & 7) == 0);
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        if (!((units >> (8 * i)) & 1u)) break;
        // the slot's last unit is done with: see kWeighJobs
        if (u >= RK) ok = __all_sync(0xffffffffu, tile_wait(bar_k_free(u % RK), ((u - RK) / RK) & 1, wc, 60));
        if (!ok) break;
        if (lane == 8 * i) {
          WeighJob* at = job_at(u);
          at->q0 = t.q0;
          at->T = t.T;
          at->ctx = t.ctx;
          at->n = t.n;
          at->h = t.h;
          at->tile = t.tile;
          at->first = t.first;
          at->nq = t.nq;
        }
        if (lane / 8 == i) job_at(u)->pages[lane & 7] = have ? page : -1;
        __syncwarp();
        const int st = u % RK;
        constexpr int kRowB = kF8 ? D : 128;
        constexpr int kSubs = kF8 ? 1 : C::kSub;
        if (lane == 0) {
          mbar_arrive(bar_job(u % kWeighJobs));
          mbar_arrive_expect_tx(bar_k_full(st), __popc((boxes >> (8 * i)) & 0xffu) * p.box_rows * (kSubs * kRowB + (kF8 ? 1 : 0)));
        }
        __syncwarp();
        if (mine && lane / 8 == i) {
          const uint32_t dst = sK + st * C::kStageK + 16 * (lane & 7) * kRowB;
#pragma unroll
          for (int s = 0; s < kSubs; ++s)
            tma_load_4d(dst + s * C::kSubBytes, &tmK, bar_k_full(st), s * 64, row, t.h, page, pol);
          if constexpr (kF8)
            bulk_load(sbase + C::kOffCode + st * 128 + 16 * (lane & 7),
                      p.ks + (static_cast<long long>(page) * p.Hkv + t.h) * p.page + row, p.box_rows, bar_k_full(st));
        }
        live |= 1u << st;
        par = (par & ~(1u << st)) | (((u / RK) & 1u) << st);
        ++u;
      }
      if (__popc(units) < 4) break;
    }
    if (ok) {  // the end of the list: its slot too must be free
      if (u >= RK) ok = __all_sync(0xffffffffu, tile_wait(bar_k_free(u % RK), ((u - RK) / RK) & 1, wc, 60));
      if (ok && lane == 0) {
        job_at(u)->nq = -1;
        mbar_arrive(bar_job(u % kWeighJobs));
      }
    }
    // let the copies in flight land before this warp leaves
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < RK; ++s)
        if ((live >> s) & 1u) mbar_wait_drain(bar_k_full(s), (par >> s) & 1u, p.timeout_ns);
    }
  } else if (warp == 1) {
    // ================================================================ Q
    const uint64_t pol = policy_evict_normal();
    int g = 0;
    uint32_t live = 0, par = 0;
    bool ok = true;
    WeighJob t;
    for (int u = 0; job(u, t, ok, 61); ++u) {
      for (int j = 0; j < t.nq; ++j, ++g) {
        const int st = g % RQ;
        if (g >= RQ) ok = __all_sync(0xffffffffu, tile_wait(bar_q_free(st), ((g - RQ) / RQ) & 1, wc, 62));
        if (!ok) break;
        const WeighCols c = weigh_cols(p, t, j);
        // few tokens: only as many small copies as hold them
        const int toks = (c.n + p.heads - 1) / p.heads;
        const int small = (toks + p.small_tokens - 1) / p.small_tokens;
        const bool full = 4 * toks > p.tokens || small > 32;
        const int rows = full ? p.tokens * p.heads : p.small_tokens * p.heads;
        if (lane == 0) mbar_arrive_expect_tx(bar_q_full(st), (full ? 1 : small) * rows * C::kSub * 128);
        __syncwarp();
        if (lane < (full ? 1 : small)) {
#pragma unroll
          for (int s = 0; s < C::kSub; ++s)
            tma_load_4d(sQ + st * C::kTileBytes + s * C::kSubBytes + lane * rows * 128, full ? &tmQ : &tmQs, bar_q_full(st), s * 64,
                        t.h * p.G + c.head, t.q0 + c.tok + lane * p.small_tokens, 0, pol);
        }
        live |= 1u << st;
        par = (par & ~(1u << st)) | (((g / RQ) & 1u) << st);
      }
      if (!ok) break;
    }
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < RQ; ++s)
        if ((live >> s) & 1u) mbar_wait_drain(bar_q_full(s), (par >> s) & 1u, p.timeout_ns);
    }
  } else if (warp == 2) {
    // ================================================================ products
    const uint32_t dhi = (1024u >> 4) | (1u << 14) | (2u << 29);
    const uint32_t klo = ((kF8 ? sbase + C::kOffWide : sK) >> 4) | (1u << 16);
    const uint32_t qlo = (sQ >> 4) | (1u << 16);
    int g = 0;
    bool ok = true;
    WeighJob t;
    for (int u = 0; job(u, t, ok, 63); ++u) {
      const int sk = kF8 ? u % NWm : u % RK;
      ok = __all_sync(0xffffffffu, kF8 ? tile_wait(bar_w_full(sk), (u / NWm) & 1, wc, 64) : tile_wait(bar_k_full(sk), (u / RK) & 1, wc, 64));
      for (int j = 0; ok && j < t.nq; ++j, ++g) {
        const int bf = g % NB, sq = g % RQ;
        if (g >= NB) ok = tile_wait(bar_s_free(bf), ((g - NB) / NB) & 1, wc, 65);
        ok = __all_sync(0xffffffffu, ok && tile_wait(bar_q_full(sq), (g / RQ) & 1, wc, 66));
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = idesc_bf16_f32(128, (weigh_cols(p, t, j).n + 15) / 16 * 16, 0);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = (ks / 4) * (C::kSubBytes >> 4) + (ks % 4) * 2;
          mma_ss_elect(tmem + 128u * bf, (static_cast<uint64_t>(dhi) << 32) | (klo + sk * (C::kTileBytes >> 4) + off),
                       (static_cast<uint64_t>(dhi) << 32) | (qlo + sq * (C::kTileBytes >> 4) + off), idesc, ks > 0 ? 1u : 0u);
        }
        mma_commit_elect(bar_s_full(bf));
        mma_commit_elect(bar_q_free(sq));
      }
      if (!ok) break;
      mma_commit_elect(kF8 ? bar_w_free(sk) : bar_k_free(sk));
    }
    // every product issued must finish before tensor memory is released
    mma_commit_elect(bar_drain);
    mbar_wait_drain(bar_drain, 0, p.timeout_ns);
  } else if (warp >= 4 && warp < 8) {
    // ================================================================ LSE of the columns
    const int bf = warp - 4;
    float* to = reinterpret_cast<float*>(smem + C::kOffLse) + bf * 128;
    int g = 0;
    bool ok = true;
    WeighJob t;
    for (int u = 0; job(u, t, ok, 67); ++u) {
      // tiles of this unit for this buffer
      for (int j = (bf - g) & (NB - 1); j < t.nq; j += NB) {
        const WeighCols c = weigh_cols(p, t, j);
        float v[4];
        bool none = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 32 * i + lane;
          v[i] = -INFINITY;
          if (col < c.n) {
            const int tok = col / p.heads, head = c.head + col - tok * p.heads;
            v[i] = -1.4426950408889634f * __ldg(p.lse + static_cast<long long>(t.h * p.G + head) * p.total_q + t.q0 + c.tok + tok);
            if (v[i] == INFINITY) v[i] = -INFINITY;  // a row that saw nothing: exp2(-inf)
            none |= v[i] == -INFINITY;
          }
        }
        const int gg = g + j;
        if (gg >= NB) ok = __all_sync(0xffffffffu, tile_wait(bar_s_free(bf), ((gg - NB) / NB) & 1, wc, 68));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) to[32 * i + lane] = v[i];
        none = __any_sync(0xffffffffu, none);
        if (lane == 0) odd[bf] = none;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_lse(bf));
      }
      if (!ok) break;
      g += t.nq;
    }
  } else if (warp >= 8 && warp < 16) {
    // ================================================================ exponentials and sums
    const int grp = (warp - 8) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float* parts = reinterpret_cast<float*>(smem + C::kOffPart);
    int g = 0;
    bool ok = true;
    WeighJob t;
    for (int u = 0; job(u, t, ok, 69); ++u) {
      const bool last = ((g + t.nq - 1) & 1) == grp;  // this group has the unit's last tile and its result
      const int pos = t.tile * kWeighKeys + r;
      const int page = job_at(u)->pages[r / 16];
      const bool here = page >= 0 && pos < t.n;
      const long long at = here ? (static_cast<long long>(page) * p.Hkv + t.h) * p.page + static_cast<uint32_t>(pos) % static_cast<uint32_t>(p.page) : 0;
      float old = 0.f;
      if (last && here && pos < t.ctx && p.decay != 0.f) old = p.w[at];
      const int sees = max(pos - t.ctx - t.first, 0);  // tokens from t.first + sees on see this key
      float sum = 0.f;
      for (int j = (g ^ grp) & 1; j < t.nq; j += 2) {
        const int gg = g + j, bf = gg % NB;
        const WeighCols c = weigh_cols(p, t, j);
        ok = __all_sync(0xffffffffu, tile_wait(bar_lse(bf), (gg / NB) & 1, wc, 70) && tile_wait(bar_s_full(bf), (gg / NB) & 1, wc, 71));
        if (!ok) break;
        tc_fence_after();
        const float4* nl = reinterpret_cast<const float4*>(smem + C::kOffLse) + bf * 32;
        const int c0 = max(sees - (c.tok - t.first), 0) * p.heads;  // the key's first column of the tile
        const bool ragged = odd[bf] || __any_sync(0xffffffffu, c0 > 0) || (c.n & 31) != 0;
        const float2 cc = make_float2(p.c, p.c);
        float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int q = 0; 32 * q < c.n; ++q) {
          uint32_t s[32];
          tmem_ld32(tl + 128u * bf + 32 * q, s);
          float4 n4[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) n4[k] = nl[8 * q + k];
          tmem_wait_ld();
          if (!ragged) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 x = __ffma2_rn(make_float2(__uint_as_float(s[4 * k]), __uint_as_float(s[4 * k + 1])), cc, make_float2(n4[k].x, n4[k].y));
              float2 y = __ffma2_rn(make_float2(__uint_as_float(s[4 * k + 2]), __uint_as_float(s[4 * k + 3])), cc, make_float2(n4[k].z, n4[k].w));
              x.x = ex2_approx(x.x);
              x.y = ex2_approx(x.y);
              y.x = ex2_approx(y.x);
              y.y = ex2_approx(y.y);
              a0 = __fadd2_rn(a0, x);
              a1 = __fadd2_rn(a1, y);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int col = 32 * q + 4 * k;
              if (col < c.n) {
                auto one = [&](int i, float n) {
                  const float e = ex2_approx(fmaf(__uint_as_float(s[4 * k + i]), p.c, n));
                  return col + i >= c0 && col + i < c.n && n != -INFINITY ? e : 0.f;
                };
                a0 = __fadd2_rn(a0, make_float2(one(0, n4[k].x), one(1, n4[k].y)));
                a1 = __fadd2_rn(a1, make_float2(one(2, n4[k].z), one(3, n4[k].w)));
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_s_free(bf));
        sum += (a0.x + a0.y) + (a1.x + a1.y);
      }
      if (!ok) break;
      // the sum of the even tiles and of the odd ones: the same two whichever group has which
      const int slot = u % kWeighParts;
      if (!last) {
        parts[slot * 128 + r] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_part(slot));
      } else {
        if (t.nq > 1) {
          ok = __all_sync(0xffffffffu, tile_wait(bar_part(slot), (u / kWeighParts) & 1, wc, 72));
          if (!ok) break;
          sum += parts[slot * 128 + r];
        }
        if (here) p.out[at] = fmaf(p.decay, old, sum);
      }
      g += t.nq;
    }
  } else if (kF8 && warp >= 16) {
    // ================================================================ K: e4m3 -> bf16
    if constexpr (kF8) {
      const int r = threadIdx.x - 512;
      bool ok = true;
      WeighJob t;
      for (int u = 0; job(u, t, ok, 73); ++u) {
        const int st = u % RK, sw = u % NWm;
        ok = tile_wait(bar_k_full(st), (u / RK) & 1, wc, 74) && (u < NWm || tile_wait(bar_w_free(sw), ((u - NWm) / NWm) & 1, wc, 75));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint8_t* src = smem + C::kOffK + st * C::kStageK + r * D;
        uint8_t* dst = smem + C::kOffWide + sw * C::kTileBytes + r * 128;
        const uint32_t code = smem[C::kOffCode + st * 128 + r];
        const uint32_t two = (code << 7) | (code << 23);  // 2^(code - 127) twice, as bf16
        const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&two);
#pragma unroll 2
        for (int c = 0; c < D / 16; ++c) {
          const uint4 raw = *reinterpret_cast<const uint4*>(src + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
          uint8_t* to = dst + (c / 4) * C::kSubBytes;
          const int ch = (2 * c) & 7;
          *reinterpret_cast<uint4*>(to + ((ch ^ (r & 7)) << 4)) = widen8(raw.x, raw.y, scale);
          *reinterpret_cast<uint4*>(to + (((ch + 1) ^ (r & 7)) << 4)) = widen8(raw.z, raw.w, scale);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_w_full(sw));
          mbar_arrive(bar_k_free(st));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<512>(*reinterpret_cast<volatile uint32_t*>(tmem_slot));
  }
}

}  // namespace attn

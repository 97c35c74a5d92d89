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
// some blocks of 128 keys); nobody else touches its keys, so nothing is added atomically.  It goes in
// steps of two blocks and one tile of query rows:
//   one tile for the sequence's queries (decoding): the tile stays, 2 or 8 blocks of keys pass by;
//   several (a prompt): two blocks of keys stay, the tiles pass by.  Two, as the tiles come from L2:
//   with one block the copies alone were 7 TB/s.
//
// Shared memory's bandwidth is what a prompt is bound by, before exponentials (1130 cycles for 256 x
// 128 scores) and the tensor pipe (1090): both operands of a product come from there.  So the columns'
// LSE does not: it enters the product as one more step of 16, K's side 1, 1, 1, 0 ..., Q's side -LSE /
// scale as three bf16 terms (24 bits), and what a thread reads is ready for exp2.
//
// Units lie rank major, a sequence's runs of keys by position and a run's heads together: with many
// queries the first keys are seen by most, so each sequence's units go from long to short, and the
// CTAs (one an SM, persistent) take them in a snake.
//
// Warps: 0 loads K; 1 loads Q; 2 and 7 issue the products, a block of the step each (a warp beside busy
// ones gets an instruction every ten cycles or so: one issuer took 3500 cycles a step); 3 and 6 find
// units and look their pages up in turn (a unit is three dependent global loads away, some 3000
// cycles); 4 and 5 bring the columns' LSE, of even and odd tiles; 8-23 are four groups of four, two for
// the blocks of even steps and two for those of odd ones, thread r of a group key r of its block; 24-27
// (e4m3) convert.
//
// e4m3.  A unit with several tiles of queries widens its keys to bf16 with their scales, exact, once.
// One with a single tile would pay that for every key it sees: there the codes go to the tensor cores
// as they are and the queries are split into two e4m3 terms, as attn_tree_tile_kernel.cuh describes;
// the query row's power of two and the key's scale multiply the score afterwards.
//
// Turns.  A parity tells a turn of a stage from the next one, not from the one after it: who skips a turn
// of a barrier needs something else to say that it has ended before the next.
//   LSE: a warp has every other tile.  For tile t it waits until all four groups are done with the tile kLse
//   before t; the tile before that one at its place is done too, as the warp waited for a later tile's when it
//   had tile t - 2, and groups go in order.  The query stage of that tile has been given back as well: a group is
//   done with a tile after its scores have come, and an issuer gives stages back in order, before later scores.
//   Products: an issuer has every turn of its own stages of K and of its score buffers.  Where it skips q_full
//   or k_full it waits for w_full, which comes after them; a w_full that it skips (the other block's) comes before
//   the next one that it waits for, as the converting warps go in order.
//   Sums: lse_full is not waited for where scores are, which come after it.  part: arrived at in every unit;
//   who waits for it in a unit of several tiles has seen scores for which the others had to be done with more
//   tiles than lie behind the slot's last unit.
//   Conversions: at their waits.
//
// Measured, 32 / 8 heads, d = 128.  A prompt of 8192 tokens in bf16 230 us, 0.64 of the measured product
// rate: a step of 256 keys x 128 columns takes some 2000 cycles, and shared memory feeds its products (18
// of 128 x 128 x 16, both operands from there) for some 1800 of them.  64 e4m3 contexts of 900 to 16384
// tokens, a token each, 108 to 114 us where the keys alone take 69 at a copy's rate: no unit is busy, but 28 warps
// of eight roles share the instruction caches (one of a scheduler's seven waits for instructions, another
// issues every second cycle; two waits more in the code of the widening warps, which do not run here, 122),
// so that each instruction of a role's step counts: a key's place worked out three times a unit instead of
// once was 134 us, all else alike.  One context of 517 tokens 6.1 us: a launch, the units' list, three loads
// that wait for each other, a product.  (A thread a key with scalar products: 23.6 ms, 1502 us and 10; one
// MMA warp and the LSE from shared memory: 312 and 213.)
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_tree_tile_kernel.cuh"

namespace attn {

constexpr int kWeighStep = 256;     // keys of a step: two blocks of 128
constexpr int kWeighSteps = 4;      // steps of a unit with one tile, at most
constexpr int kWeighCols = 128;     // query rows of a tile, at most
constexpr int kWeighStacked = 64;   // e4m3, columns up to which a query's two terms are rows of one operand
constexpr int kWeighGroups = 64;    // prefix-sum entries (each over ceil(B / 64) sequences)
constexpr int kWeighJobs = 6;       // units announced in shared memory
constexpr int kWeighFinders = 2;
// e4m3: factors of query rows, unit u % 8, and scale codes of keys, block x % 16.  K is at most kRingK
// <= 8 blocks ahead of the products and these two steps, four blocks, ahead of the sums.
constexpr int kWeighFactors = 8;
constexpr int kWeighCodes = 16;
constexpr int kWeighParts = 4;      // sums on their way from one pair of groups to the other (three units apart at most)
constexpr int kWeighSumWarp = 8, kWeighConvWarp = 24;

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
  int ring_k, ring_q;        // stages of K's ring and of Q's
  float c;                   // scale * log2(e)
  float rscale;              // 1 / scale
  float decay;
  uint32_t* status;
  uint32_t* page_word;
  unsigned long long timeout_ns;
};

// A sequence, every field clamped to what the buffers hold.
struct WeighSeq {
  int q0, T, ctx, n;
};
__device__ __forceinline__ WeighSeq weigh_seq(const WeighParams& p, int b) {
  WeighSeq s;
  s.q0 = min(max(__ldg(p.cu + b), 0), p.total_q);
  s.T = min(max(__ldg(p.cu + b + 1), s.q0), p.total_q) - s.q0;
  s.ctx = p.ctx ? min(max(__ldg(p.ctx + b), 0), p.cap) : 0;
  s.n = static_cast<int>(min(static_cast<long long>(s.ctx) + s.T, static_cast<long long>(p.cap)));
  return s;
}
// Keys of a sequence's units, when those with one tile have `steps` steps, and their number for a head.
__device__ __forceinline__ int weigh_unit_keys(const WeighParams& p, const WeighSeq& s, int steps) {
  return p.heads == p.G && s.T <= p.tokens ? steps * kWeighStep : kWeighStep;
}
__device__ __forceinline__ int weigh_units(const WeighParams& p, const WeighSeq& s, int steps) {
  const int keys = weigh_unit_keys(p, s, steps);
  return s.T > 0 ? s.n / keys + (s.n % keys != 0) : 0;
}

// A unit as its finder announces it.
struct WeighUnit {
  int q0, T, ctx, n;
  int h, key0;             // its first key
  int nq;                  // tiles of query rows; < 0: the end
  int steps;               // steps of its one tile (1 with several)
  __device__ __forceinline__ int first() const { return max(0, key0 - ctx); }  // the first token that sees any of its keys
};
struct WeighJob {
  WeighUnit unit;
  long long rows[16 * kWeighSteps];  // of the unit's slices of 16 keys in the pool, -1 without a page
  int pages[16 * kWeighSteps];
};

// A place in a ring of stages and the parity of its turn.
struct WeighRing {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++st == n) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// Columns of tile j of a unit: tokens [tok, tok + n) with heads [head, head + p.heads) of the group.
struct WeighCols {
  int tok, head, n;
};
__device__ __forceinline__ WeighCols weigh_cols(const WeighParams& p, int first, int T, int j) {
  WeighCols c;
  if (p.heads == p.G) {
    c.tok = first + j * p.tokens;
    c.head = 0;
    c.n = min(p.tokens, T - c.tok) * p.heads;
  } else {  // more than 128 heads a group: a token, 128 heads at a time
    const int per = (p.G + p.heads - 1) / p.heads;
    c.tok = first + j / per;
    c.head = (j % per) * p.heads;
    c.n = min(p.heads, p.G - c.head);
  }
  return c;
}

__device__ __forceinline__ void prefetch_l2(const float* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// mma_ss_f8 by one elected lane of a warp that agrees on everything.
__device__ __forceinline__ void mma_ss_f8_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 4 columns of 32-bit.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}

// A step of 16 in the product beside K and Q: 128 rows without swizzle, 8 x 16-byte blocks, the two of
// a row's 32 bytes 128 apart, the next eight rows 256 further.
constexpr int kWeighStepBytes = 128 * 32;
__device__ __forceinline__ uint32_t weigh_step_row(int r) { return (r >> 3) * 256 + (r & 7) * 16; }
__device__ __forceinline__ uint64_t weigh_step_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(128 >> 4) << 16) |
         (static_cast<uint64_t>(256 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

template <int D, bool kF8>
struct WeighCfg {
  static constexpr int kThreads = 32 * (kWeighConvWarp + (kF8 ? 4 : 0));
  static constexpr int kSub = D / 64;
  static constexpr int kSubBytes = 128 * 128;            // 128 rows x 64 bf16
  static constexpr int kTileBytes = kSub * kSubBytes;    // 128 rows in bf16
  static constexpr int kStageK = kF8 ? 128 * D : kTileBytes;  // a block of keys
  static constexpr int kWide = kF8 ? 2 : 0;              // operands in another form than they came
  // What the rings of K and Q share: (one tile a unit, as in decoding) stages of K for the bytes in
  // flight, or (several) of Q, whose way from L2 is 2000 to 3000 cycles with all SMs at it.
  static constexpr int kFewK = D == 128 ? 4 : 8;
  static constexpr int kFewQ = 2;  // (not 1: the LSE's warps see every other turn of a single stage, and could not tell them apart)
  static constexpr int kManyK = kF8 ? (D == 128 ? 2 : 4) : 2;
  static constexpr int kManyQ = kF8 ? (D == 128 ? 3 : 4) : (D == 128 ? 4 : 8);
  static constexpr int kLse = kF8 ? 3 : 4;               // tiles whose LSE is at hand
  static constexpr int kMaxK = kFewK > kManyK ? kFewK : kManyK, kMaxQ = kManyQ;
  static constexpr int kPool = kFewK * kStageK + kFewQ * kTileBytes;
  static_assert(kFewK % 2 == 0 && kManyK % 2 == 0, "a step's two blocks have neighbouring stages");
  static_assert(kManyK * kStageK + kManyQ * kTileBytes <= kPool, "both divisions of the stages");
  static constexpr int kOffWide = kPool;                                    // Q's stages, then K's, before it
  static constexpr int kOffOnes = kOffWide + kWide * kTileBytes;            // the step of 16: K's side,
  static constexpr int kOffStep = kOffOnes + kWeighStepBytes;               // Q's, tile by tile
  static constexpr int kOffCode = kOffStep + kLse * kWeighStepBytes;        // scale codes, 128 a block
  static constexpr int kOffLse = kOffCode + (kF8 ? kWeighCodes * 128 : 0);  // 128 floats a tile
  static constexpr int kOffFactor = kOffLse + kLse * 512;                   // 128 floats, unit u % 8
  static constexpr int kOffPart = kOffFactor + (kF8 ? kWeighFactors * 512 : 0);     // 256 floats, unit u % 4
  static constexpr int kOffJobs = kOffPart + kWeighParts * 1024;
  static constexpr int kOffPre = kOffJobs + kWeighJobs * static_cast<int>(sizeof(WeighJob));
  static constexpr int kOffBar = kOffPre + 8 * (2 * (kWeighGroups + 1) + 2);
  // {job, job_free}[J], {k_full, k_free}[K], {w_full, w_free}[W], {q_full, q_free}[Q], {s_full, s_free}[4],
  // part[P][2], lse_free[L][4], lse_full[L], drain[2]
  static constexpr int kNumBars = 2 * kWeighJobs + 2 * kMaxK + 2 * kWide + 2 * kMaxQ + 8 + 2 * kWeighParts + 5 * kLse + 2;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;                   // tmem base, abort, odd[4]
  static constexpr int kSmem = kOffMisc + 24 + 1024;
  // warps that read a unit: K, Q, products (2), LSE (2), sums (16), conversions (4)
  static constexpr int kReaders = 22 + (kF8 ? 4 : 0);
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <int D, bool kF8>
__global__ void __launch_bounds__(WeighCfg<D, kF8>::kThreads, 1)
    attn_weigh_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQs,
                      const __grid_constant__ CUtensorMap tmK, const WeighParams p) {
  using C = WeighCfg<D, kF8>;
  constexpr int MK = C::kMaxK, MQ = C::kMaxQ, NW = C::kWide, NWm = NW > 0 ? NW : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // (an offset: it stays a shared address)
  const uint32_t sbase = smem_u32(smem), sQ = sbase, sK = sbase + p.ring_q * C::kTileBytes, bar0 = sbase + C::kOffBar;
  auto bar_job = [&](int i) { return bar0 + 8u * i; };
  auto bar_job_free = [&](int i) { return bar0 + 8u * (kWeighJobs + i); };
  constexpr int kB0 = 2 * kWeighJobs;
  auto bar_k_full = [&](int s) { return bar0 + 8u * (kB0 + s); };
  auto bar_k_free = [&](int s) { return bar0 + 8u * (kB0 + MK + s); };
  constexpr int kB1 = kB0 + 2 * MK;
  auto bar_w_full = [&](int s) { return bar0 + 8u * (kB1 + s); };
  auto bar_w_free = [&](int s) { return bar0 + 8u * (kB1 + NW + s); };
  constexpr int kB2 = kB1 + 2 * NW;
  auto bar_q_full = [&](int s) { return bar0 + 8u * (kB2 + s); };
  auto bar_q_free = [&](int s) { return bar0 + 8u * (kB2 + MQ + s); };
  constexpr int kB3 = kB2 + 2 * MQ;
  // score buffers: block h of step g in buffer 2 (g % 2) + h
  auto bar_s_full = [&](int b) { return bar0 + 8u * (kB3 + b); };
  auto bar_s_free = [&](int b) { return bar0 + 8u * (kB3 + 4 + b); };
  // A barrier for each group of four warps, not one for several: a group's warps are never two of its
  // steps apart, as they share a score buffer, while the blocks' groups may be a ring's length apart.
  auto bar_part = [&](int i, int blk) { return bar0 + 8u * (kB3 + 8 + 2 * i + blk); };
  auto bar_lse_free = [&](int i, int grp) { return bar0 + 8u * (kB3 + 8 + 2 * kWeighParts + 4 * i + grp); };
  auto bar_lse_full = [&](int i) { return bar0 + 8u * (kB3 + 8 + 2 * kWeighParts + 4 * C::kLse + i); };
  auto bar_drain = [&](int h) { return bar0 + 8u * (kB3 + 8 + 2 * kWeighParts + 5 * C::kLse + h); };
  long long* pre = reinterpret_cast<long long*>(smem + C::kOffPre);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 4);
  // odd[i]: a column of the tile at place i adds nothing whatever its scores are
  volatile uint32_t* odd = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWeighJobs; ++i) {
      mbar_init(bar_job(i), 1);
      mbar_init(bar_job_free(i), C::kReaders);
    }
    for (int s = 0; s < MK; ++s) {
      mbar_init(bar_k_full(s), 1);
      mbar_init(bar_k_free(s), 1);
    }
    for (int s = 0; s < NW; ++s) {
      mbar_init(bar_w_full(s), 4);
      mbar_init(bar_w_free(s), 2);
    }
    for (int s = 0; s < MQ; ++s) {
      mbar_init(bar_q_full(s), 2);  // its rows and their LSE
      mbar_init(bar_q_free(s), 2);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(bar_s_full(b), 1);
      mbar_init(bar_s_free(b), 4);
    }
    for (int i = 0; i < 2 * kWeighParts; ++i) mbar_init(bar_part(0, i), 4);
    for (int i = 0; i < 4 * C::kLse; ++i) mbar_init(bar_lse_free(0, i), 4);
    for (int i = 0; i < C::kLse; ++i) mbar_init(bar_lse_full(i), 1);
    mbar_init(bar_drain(0), 1);
    mbar_init(bar_drain(1), 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  // the step of 16: K's side 1, 1, 1, 0 ..., Q's second half zeros (the first comes with the LSE)
  for (int r = threadIdx.x; r < (1 + C::kLse) * 128; r += C::kThreads) {
    uint4* row = reinterpret_cast<uint4*>(smem + C::kOffOnes + (r >> 7) * kWeighStepBytes + weigh_step_row(r & 127));
    row[0] = r < 128 ? make_uint4(0x3f803f80u, 0x00003f80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    row[8] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 2) tmem_alloc<512>(smem_u32(tmem_slot));
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmQs);
    if (p.num_pages > 0) tma_prefetch_desc(&tmK);  // without pages there is no map
  }
  griddep_wait();
  // pre[0 / 1][i]: units of the sequences before group i (groups of gs sequences) with 1 or kWeighSteps
  // steps where there is one tile.  The longer ones cost less a key and are taken when they still go
  // round the CTAs four times.
  const int gs = (p.B + kWeighGroups - 1) / kWeighGroups;
  {
    long long* warp_sums = pre + 2 * (kWeighGroups + 1);
    long long sum[2] = {0, 0};
    if (threadIdx.x < kWeighGroups) {
      const long long first = static_cast<long long>(threadIdx.x) * gs;
      for (long long b = first; b < min(first + gs, static_cast<long long>(p.B)); ++b) {
        const WeighSeq s = weigh_seq(p, static_cast<int>(b));
        sum[0] += static_cast<long long>(weigh_units(p, s, 1)) * p.Hkv;
        sum[1] += static_cast<long long>(weigh_units(p, s, kWeighSteps)) * p.Hkv;
        if (blockIdx.x == 0 && s.T > 0 && p.page_word && static_cast<long long>(s.ctx) + s.T > p.cap) atomicOr(p.page_word, 1u);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const long long v = __shfl_up_sync(0xffffffffu, sum[i], o);
          if (lane >= o) sum[i] += v;
        }
      if (threadIdx.x == 31) {
        warp_sums[0] = sum[0];
        warp_sums[1] = sum[1];
      }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < kWeighGroups) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pre[i * (kWeighGroups + 1) + threadIdx.x + 1] = sum[i] + (warp == 1 ? warp_sums[i] : 0);
        if (threadIdx.x == 0) pre[i * (kWeighGroups + 1)] = 0;
      }
    }
    __syncthreads();
    tc_fence_after();
  }
  const bool longer = pre[2 * kWeighGroups + 1] >= 4ll * gridDim.x;
  if (longer) pre += kWeighGroups + 1;
  // not before this CTA has its tensor memory: a later launch that got there first would hold it
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  WeighJob* jobs = reinterpret_cast<WeighJob*>(smem + C::kOffJobs);
  // The next unit, for a whole warp (one that gives up gives up with all its lanes); false at the end of
  // the list, or (ok = false too) when the wait ran out.  rows: what of the slot the warp reads besides.
  WeighRing jr;
  auto job_more = [&](WeighUnit& t, bool& ok, uint32_t site, auto rows) {
    ok = __all_sync(0xffffffffu, tile_wait(bar_job(jr.st), jr.ph, wc, site));
    if (!ok) return false;
    const int4* at = reinterpret_cast<const int4*>(jobs + jr.st);
    const int4 a = at[0], b = at[1];
    t = WeighUnit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    rows(jobs[jr.st], t);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_job_free(jr.st));
    jr.next(kWeighJobs);
    return t.nq >= 0;
  };
  auto job = [&](WeighUnit& t, bool& ok, uint32_t site) { return job_more(t, ok, site, [](const WeighJob&, const WeighUnit&) {}); };

  if (warp == 3 || warp == 6) {
    // ================================================================ units
    const long long U = pre[kWeighGroups];
    const int steps = longer ? kWeighSteps : 1;
    auto unit_of = [&](long long r) { return r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
    WeighRing slot;
    if (warp == 6) slot.next(kWeighJobs);
    bool ok = true;
    for (long long r = warp == 3 ? 0 : 1; r == 0 || unit_of(r - 1) < U; r += kWeighFinders) {  // the end is announced once
      const long long unit = unit_of(r);
      WeighUnit t = {};
      t.nq = -1;
      long long rows[2] = {-1, -1};
      int pages[2] = {-1, -1};
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
        for (;;) {
          const long long n = static_cast<long long>(weigh_units(p, s, steps)) * p.Hkv;
          if (y < n || b + 1 >= p.B) break;
          y -= n;
          s = weigh_seq(p, ++b);
        }
        const int keys = weigh_unit_keys(p, s, steps), run = static_cast<int>(tree_div(y, p.Hkv));
        t.q0 = s.q0;
        t.T = s.T;
        t.ctx = s.ctx;
        t.n = s.n;
        t.h = static_cast<int>(y - static_cast<long long>(run) * p.Hkv);
        t.key0 = run * keys;
        const int first = t.first();
        t.nq = p.heads == p.G ? (s.T - first + p.tokens - 1) / p.tokens : (s.T - first) * ((p.G + p.heads - 1) / p.heads);
        t.steps = (min(keys, s.n - t.key0) + kWeighStep - 1) / kWeighStep;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // lane i: slices i and i + 32
          const int pos = min(t.key0 + 16 * (lane + 32 * i), s.n - 1);
          const int in = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page);
          pages[i] = __ldg(p.table + static_cast<long long>(b) * p.max_pages + in);
          rows[i] = pos - in * p.page;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool need = 16 * (lane + 32 * i) < min(keys, s.n - t.key0);
          const bool have = need && static_cast<unsigned>(pages[i]) < static_cast<unsigned>(p.num_pages);
          if (need && !have && p.page_word) atomicOr(p.page_word, 1u);
          rows[i] = have ? (static_cast<long long>(pages[i]) * p.Hkv + t.h) * p.page + rows[i] : -1;
          if (have && p.decay != 0.f) prefetch_l2(p.w + rows[i]);
        }
      }
      ok = __all_sync(0xffffffffu, tile_wait(bar_job_free(slot.st), slot.ph ^ 1u, wc, 60));
      if (!ok) break;
      WeighJob& at = jobs[slot.st];
      if (lane == 0) {
        reinterpret_cast<int4*>(&at)[0] = make_int4(t.q0, t.T, t.ctx, t.n);
        reinterpret_cast<int4*>(&at)[1] = make_int4(t.h, t.key0, t.nq, t.steps);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        at.rows[lane + 32 * i] = rows[i];
        at.pages[lane + 32 * i] = pages[i];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_job(slot.st));
      for (int i = 0; i < kWeighFinders; ++i) slot.next(kWeighJobs);
    }
  } else if (warp == 0) {
    // ================================================================ K
    const uint64_t pol = policy_evict_first();
    const int box16 = p.box_rows / 16;
    WeighRing k;
    uint32_t live = 0, par = 0, x = 0;  // x: blocks
    bool ok = true;
    WeighUnit t;
    long long row[2] = {-1, -1};
    int page[2] = {-1, -1};
    while (job_more(t, ok, 61, [&](const WeighJob& at, const WeighUnit&) {  // lane i: slices i and i + 32
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        row[i] = at.rows[lane + 32 * i];
        page[i] = at.pages[lane + 32 * i];
      }
    })) {
      // A step's two blocks at a time, 16 lanes with a slice each (a warp beside busy ones gets an instruction
      // every ten cycles: block by block this was as slow as the products).  The ring's stages are even.
      // A row lies in its page's at row - (page * Hkv + h) * page_size.
#pragma unroll 1
      for (int st = 0; st < t.steps; ++st, x += 2, k.next(p.ring_k), k.next(p.ring_k)) {  // a block without keys is a block of anything
        const long long rw = st < 2 ? row[0] : row[1];
        const int pg = st < 2 ? page[0] : page[1];
        const bool mine = lane / 16 == (st & 1) && rw >= 0 && (lane & 7) % box16 == 0;
        const uint32_t who = __ballot_sync(0xffffffffu, mine) >> (16 * (st & 1));
        ok = __all_sync(0xffffffffu, tile_wait(bar_k_free(k.st), k.ph ^ 1u, wc, 62) && tile_wait(bar_k_free(k.st + 1), k.ph ^ 1u, wc, 62));
        if (!ok) break;
        constexpr int kRowB = kF8 ? D : 128;
        constexpr int kSubs = kF8 ? 1 : C::kSub;
        if (lane < 2)
          mbar_arrive_expect_tx(bar_k_full(k.st + lane), __popc((who >> (8 * lane)) & 0xffu) * p.box_rows * (kSubs * kRowB + (kF8 ? 1 : 0)));
        __syncwarp();
        if (mine) {
          const int h = (lane >> 3) & 1;
          const uint32_t dst = sK + (k.st + h) * C::kStageK + 16 * (lane & 7) * kRowB, bar = bar_k_full(k.st + h);
          const int in_page = static_cast<int>(rw - (static_cast<long long>(pg) * p.Hkv + t.h) * p.page);
#pragma unroll
          for (int s = 0; s < kSubs; ++s) tma_load_4d(dst + s * C::kSubBytes, &tmK, bar, s * 64, in_page, t.h, pg, pol);
          if constexpr (kF8)
            bulk_load(sbase + C::kOffCode + ((x + h) % kWeighCodes) * 128 + 16 * (lane & 7), p.ks + rw, p.box_rows, bar);
        }
        live |= 3u << k.st;
        par = (par & ~(3u << k.st)) | (k.ph ? 3u << k.st : 0u);
      }
      if (!ok) break;
    }
    // let the copies in flight land before this warp leaves
    if (lane == 0)
      for (int s = 0; s < p.ring_k; ++s)
        if ((live >> s) & 1u) mbar_wait_drain(bar_k_full(s), (par >> s) & 1u, p.timeout_ns);
  } else if (warp == 1) {
    // ================================================================ Q
    const uint64_t pol = policy_evict_normal();
    WeighRing q;
    uint32_t live = 0, par = 0;
    bool ok = true;
    WeighUnit t;
    while (job(t, ok, 63)) {
      const int first = t.first();
      for (int j = 0; j < t.nq; ++j, q.next(p.ring_q)) {
        ok = __all_sync(0xffffffffu, tile_wait(bar_q_free(q.st), q.ph ^ 1u, wc, 64));
        if (!ok) break;
        const WeighCols c = weigh_cols(p, first, t.T, j);
        // few tokens: only as many small copies as hold them
        const int toks = (c.n + p.heads - 1) / p.heads;
        const int small = (toks + p.small_tokens - 1) / p.small_tokens;
        const bool full = 4 * toks > p.tokens || small > 32;
        const int rows = full ? p.tokens * p.heads : p.small_tokens * p.heads;
        if (lane == 0) mbar_arrive_expect_tx(bar_q_full(q.st), (full ? 1 : small) * rows * C::kSub * 128);
        __syncwarp();
        if (lane < (full ? 1 : small)) {
#pragma unroll
          for (int s = 0; s < C::kSub; ++s)
            tma_load_4d(sQ + q.st * C::kTileBytes + s * C::kSubBytes + lane * rows * 128, full ? &tmQ : &tmQs, bar_q_full(q.st), s * 64,
                        t.h * p.G + c.head, t.q0 + c.tok + lane * p.small_tokens, 0, pol);
        }
        live |= 1u << q.st;
        par = (par & ~(1u << q.st)) | (q.ph << q.st);
      }
      if (!ok) break;
    }
    if (lane == 0)
      for (int s = 0; s < p.ring_q; ++s)
        if ((live >> s) & 1u) mbar_wait_drain(bar_q_full(s), (par >> s) & 1u, p.timeout_ns);
  } else if (warp == 2 || warp == 7) {
    // ================================================================ products
    // (all lanes go the same way and one elected issues, as in attn_fwd_pair_kernel; what a unit is comes through
    // a shuffle, so that the compiler knows it for the warp's.  Under a branch to one lane the batch of e4m3
    // contexts below took 152 us instead of 139, the prompt 243 instead of 233; units shuffled for every role 143)
    const int h = warp == 7 ? 1 : 0;  // the block
    auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) { return __all_sync(0xffffffffu, tile_wait(bar, parity, wc, site)) != 0; };
    const uint32_t dhi = (1024u >> 4) | (1u << 14) | (2u << 29);
    const uint32_t dhi8 = D == 128 ? dhi : (512u >> 4) | (1u << 14) | (4u << 29);  // e4m3 rows of 64 bytes: 64-byte swizzle
    const uint32_t klo = (sK >> 4) | (1u << 16), wlo = ((sbase + C::kOffWide) >> 4) | (1u << 16);
    const uint32_t qlo = (sQ >> 4) | (1u << 16);
    auto desc = [](uint32_t hi, uint32_t lo) { return (static_cast<uint64_t>(hi) << 32) | lo; };
    WeighRing k, q, w;
    if (h) k.next(p.ring_k);
    WeighRing l;     // places of the tiles' LSE
    uint32_t g = 0;  // steps
    bool ok = true;
    WeighUnit t;
    while (job(t, ok, 65)) {
      t.nq = __shfl_sync(0xffffffffu, t.nq, 0);
      t.steps = __shfl_sync(0xffffffffu, t.steps, 0);
      const bool single = t.nq == 1, narrow = kF8 && single;
      const uint32_t cols = __shfl_sync(0xffffffffu, (weigh_cols(p, t.first(), t.T, 0).n + 15) / 16 * 16, 0);
      {
        uint32_t a = 0, wst = 0;
        if (kF8 && !narrow) {  // widened keys: two stages, one for each issuer
          if (h) w.next(NWm);
          wst = w.st;
          ok = wait(bar_w_full(w.st), w.ph, 66);
          if (ok && lane == 0) mbar_arrive(bar_k_free(k.st));  // its codes have been read
          a = wlo + w.st * (C::kTileBytes >> 4);
          if (!h) w.next(NWm);
          w.next(NWm);
        }
        auto product = [&](uint32_t dst, uint32_t b, uint32_t idesc) {  // bf16
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (ks / 4) * (C::kSubBytes >> 4) + (ks % 4) * 2;
            mma_ss_elect(dst, desc(dhi, a + off), desc(dhi, b + off), idesc, ks > 0 ? 1u : 0u);
          }
          // the LSE last: everything before it is a sum of small terms
          mma_ss_elect(dst, weigh_step_desc(sbase + C::kOffOnes), weigh_step_desc(sbase + C::kOffStep + l.st * kWeighStepBytes), idesc, 1u);
        };
        if (single) {
          ok = narrow ? wait(bar_w_full(w.st), w.ph, 68) : wait(bar_q_full(q.st), q.ph, 69);
          if (narrow && ok && lane == 0) mbar_arrive(bar_q_free(q.st));  // its rows have been read: their two terms are there
          const bool stacked = narrow && cols <= kWeighStacked;
          const uint32_t idesc = narrow ? (1u << 4) | (((stacked ? 2 * cols : cols) >> 3) << 17) | (8u << 24)  // e4m3 x e4m3 -> fp32
                                        : idesc_bf16_f32(128, cols, 0);
          const uint32_t b = narrow ? wlo + w.st * (C::kTileBytes >> 4) : qlo + q.st * (C::kTileBytes >> 4);
          for (int j = 0; ok && j < t.steps; ++j, ++g) {
            const uint32_t bf = 2 * (g & 1) + h, dst = tmem + 128u * bf;
            ok = wait(bar_k_full(k.st), k.ph, 66) && wait(bar_s_free(bf), ((g >> 1) & 1) ^ 1, 70);
            if (!ok) break;
            tc_fence_after();
            a = klo + k.st * (C::kStageK >> 4);
            if constexpr (kF8) {
#pragma unroll
              for (int ks = 0; ks < D / 32; ++ks) mma_ss_f8_elect(dst, desc(dhi8, a + ks * 2), desc(dhi8, b + ks * 2), idesc, ks > 0 ? 1u : 0u);
              if (!stacked) {
#pragma unroll
                for (int ks = 0; ks < D / 32; ++ks) mma_ss_f8_elect(dst, desc(dhi8, a + ks * 2), desc(dhi8, b + (128 * D >> 4) + ks * 2), idesc, 1u);
              }
            } else {
              product(dst, b, idesc);
            }
            mma_commit_elect(bar_s_full(bf));
            mma_commit_elect(bar_k_free(k.st));
            k.next(p.ring_k);
            k.next(p.ring_k);
          }
          if (narrow) {
            mma_commit_elect(bar_w_free(w.st));
            w.next(NWm);
          } else {
            mma_commit_elect(bar_q_free(q.st));
          }
          q.next(p.ring_q);
          l.next(C::kLse);
        } else {
          if constexpr (!kF8) {
            ok = wait(bar_k_full(k.st), k.ph, 66);
            a = klo + k.st * (C::kStageK >> 4);
          }
          const uint32_t idesc = idesc_bf16_f32(128, cols, 0);
          for (int j = 0; ok && j < t.nq; ++j, ++g) {
            const uint32_t bf = 2 * (g & 1) + h;
            ok = wait(bar_q_full(q.st), q.ph, 69) && wait(bar_s_free(bf), ((g >> 1) & 1) ^ 1, 70);
            if (!ok) break;
            tc_fence_after();
            // with the first tile's columns, which are never fewer (what lies past a tile's own is not looked at)
            product(tmem + 128u * bf, qlo + q.st * (C::kTileBytes >> 4), idesc);
            mma_commit_elect(bar_s_full(bf));
            mma_commit_elect(bar_q_free(q.st));
            q.next(p.ring_q);
            l.next(C::kLse);
          }
          if constexpr (kF8) {  // nobody but this issuer had the stage
            mma_commit_elect(bar_w_free(wst));
            mma_commit_elect(bar_w_free(wst));
          } else {
            mma_commit_elect(bar_k_free(k.st));
          }
          k.next(p.ring_k);
          k.next(p.ring_k);
        }
      }
      if (!ok) break;
    }
    // every product issued must finish before tensor memory is released
    if (lane == 0) {
      mma_commit(bar_drain(h));
      mbar_wait_drain(bar_drain(h), 0, p.timeout_ns);
    }
  } else if (warp == 4 || warp == 5) {
    // ================================================================ LSE of the columns
    const int par = warp - 4;  // of the tiles
    int g = 0;                 // tiles
    bool ok = true;
    WeighUnit t;
    WeighRing q, l;
    if (par) {
      q.next(p.ring_q);
      l.next(C::kLse);
    }
    // this lane's columns, four of them: token of the tile and the way to their head's LSE from the first's
    int tok[4];
    long long off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tok[i] = (32 * i + lane) / p.heads;
      off[i] = static_cast<long long>(32 * i + lane - tok[i] * p.heads) * p.total_q + tok[i];
    }
    float next[4];
    while (job(t, ok, 71)) {
      const int first = t.first();
      auto load = [&](int j) {
        const WeighCols c = weigh_cols(p, first, t.T, j);
        const float* from = p.lse + static_cast<long long>(t.h * p.G + c.head) * p.total_q + t.q0 + c.tok;
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = 32 * i + lane < c.n ? __ldg(from + off[i]) : -INFINITY;
      };
      const int j0 = (par ^ g) & 1;
      if (j0 < t.nq) load(j0);
      for (int j = j0; j < t.nq; j += 2) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = next[i];
        if (j + 2 < t.nq) load(j + 2);
        // every group is done with the tile that had this place (a lane looks after one), and the stage of
        // its rows has been freed: what arrives there sooner would count for the tile before it
        ok = __all_sync(0xffffffffu, tile_wait(bar_lse_free(l.st, lane & 3), l.ph ^ 1u, wc, 72) &&
                                         tile_wait(bar_q_free(q.st), q.ph ^ 1u, wc, 72));
        if (!ok) break;
        bool none = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool out = fabsf(v[i]) == INFINITY;  // a row that saw nothing, or none: exp2(-inf)
          none |= out && (v[i] > 0.f || 32 * i + lane < p.tokens * p.heads);
          reinterpret_cast<float*>(smem + C::kOffLse)[l.st * 128 + 32 * i + lane] = out ? -INFINITY : -1.4426950408889634f * v[i];
          // -LSE / scale as three bf16 terms, exact: eight of its bits each
          const float x = out ? 0.f : -p.rscale * v[i];
          const float t1 = __uint_as_float(__float_as_uint(x) & 0xffff0000u), t23 = x - t1;
          const float t2 = __uint_as_float(__float_as_uint(t23) & 0xffff0000u);
          *reinterpret_cast<uint4*>(smem + C::kOffStep + l.st * kWeighStepBytes + weigh_step_row(32 * i + lane)) =
              make_uint4(__byte_perm(__float_as_uint(t1), __float_as_uint(t2), 0x7632), __float_as_uint(t23 - t2) >> 16, 0u, 0u);
        }
        none = __any_sync(0xffffffffu, none);
        if (lane == 0) odd[l.st] = none;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_lse_full(l.st));  // before q_full: a group that looks at the tile does not wait for this
          mbar_arrive(bar_q_full(q.st));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          q.next(p.ring_q);
          l.next(C::kLse);
        }
      }
      if (!ok) break;
      g += t.nq;
    }
  } else if (warp >= kWeighSumWarp && warp < kWeighConvWarp) {
    // ================================================================ exponentials and sums
    const int pair = (warp - kWeighSumWarp) >> 3, blk = ((warp - kWeighSumWarp) >> 2) & 1, r = (warp & 3) * 32 + lane;
    const int bf = 2 * pair + blk;
    const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128u * bf;
    float* parts = reinterpret_cast<float*>(smem + C::kOffPart) + 128 * blk + r;
    uint32_t g = 0, u = 0, x = 0;  // steps, units, blocks
    bool ok = true;
    WeighRing l;
    WeighUnit t;
    // Where this thread's keys are: in a unit of one tile its steps are every other one, two at most.
    long long at[2] = {-1, -1};
    auto rows = [&](const WeighJob& job, const WeighUnit& un) {
      const int s0 = un.nq == 1 ? (g ^ pair) & 1 : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) at[i] = job.rows[16 * (s0 + 2 * i) + 8 * blk + r / 16];
    };
    static_assert(kWeighSteps <= 4, "two steps a group");
    for (; job_more(t, ok, 73, rows); ++u) {
      const bool single = t.nq == 1, narrow = kF8 && single;
      const int first = t.first(), n = single ? t.steps : t.nq;
      const int j0 = (g ^ pair) & 1;                    // this pair's first step
      const bool last = single || ((n - 1) & 1) == j0;  // whether the result is this pair's to write
      float old[2] = {0.f, 0.f}, sum = 0.f, before = 0.f;  // before: the first step's sum
      const int pos = t.key0 + (single ? kWeighStep * j0 : 0) + 128 * blk + r;  // of the first
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int here = pos + 2 * kWeighStep * i;
        const bool is = at[i] >= 0 && here < t.n && (single ? j0 + 2 * i < n : i == 0 && last);
        at[i] = is ? at[i] + (r & 15) : -1;
        if (is && here < t.ctx && p.decay != 0.f) old[i] = p.w[at[i]];
      }
      int sees = max(pos - t.ctx - first, 0);  // tokens from first + sees on see this thread's key
      WeighCols c = weigh_cols(p, first, t.T, 0);
      // A tile that this group does not look at, handed back once its LSE has come: earlier it would be
      // handed back for the tile before it at its place.
      auto pass = [&]() {
        if (!__all_sync(0xffffffffu, tile_wait(bar_lse_full(l.st), l.ph, wc, 80))) return false;
        if (lane == 0) mbar_arrive(bar_lse_free(l.st, bf));
        l.next(C::kLse);
        return true;
      };
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        if ((j ^ j0) & 1) {  // the other pair's
          if (single) continue;
          ok = pass();
          if (!ok) break;
          continue;
        }
        if (!single) c = weigh_cols(p, first, t.T, j);
        if (single) sees = max(pos + kWeighStep * (j - j0) - t.ctx - first, 0);
        int c0 = 0;     // the key's first column of the tile
        int plain = narrow ? 0 : c.n & ~31;  // columns that every key of the warp sees, 32 at a time
        if (c.tok - first < kWeighStep) {
          c0 = max(sees - (c.tok - first), 0) * p.heads;
          if (__any_sync(0xffffffffu, c0 > 0)) plain = 0;
        }
        ok = __all_sync(0xffffffffu, tile_wait(bar_s_full(bf), ((g + j) >> 1) & 1, wc, 74));
        if (!ok) break;
        tc_fence_after();
        if (plain > 0 && odd[l.st]) plain = 0;
        float2 a0 = make_float2(0.f, 0.f), a1 = make_float2(0.f, 0.f);
        {
          const float2 cc = make_float2(p.c, p.c);
#pragma unroll 1
          for (int q = 0; q < plain; q += 32) {
            uint32_t s[32];
            tmem_ld32(ts + q, s);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 e = __fmul2_rn(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), cc);
              e.x = ex2_approx(e.x);
              e.y = ex2_approx(e.y);
              if (k & 1)
                a1 = __fadd2_rn(a1, e);
              else
                a0 = __fadd2_rn(a0, e);
            }
          }
        }
        if (plain < c.n) {
          const float4* nl = reinterpret_cast<const float4*>(smem + C::kOffLse) + l.st * 32;
          const float4* fac = reinterpret_cast<const float4*>(smem + C::kOffFactor) + (u % kWeighFactors) * 32;
          const int lo = narrow && c.n <= kWeighStacked ? (c.n + 15) / 16 * 16 : 0;  // where the second terms' products are
          float key_scale = 1.f;
          if (narrow) key_scale = scale_of(max(static_cast<uint32_t>(smem[C::kOffCode + ((x + 2 * j + blk) % kWeighCodes) * 128 + r]), 1u));
#pragma unroll 1
          for (int q = plain; q < c.n; q += 4) {
            uint32_t s[4], s2[4];
            tmem_ld4(ts + q, s);
            if (lo) tmem_ld4(ts + lo + q, s2);
            tmem_wait_ld();
            const float4 n4 = nl[q >> 2];  // (-infinity past the tile's columns)
            float4 f4 = make_float4(p.c, p.c, p.c, p.c);
            if (narrow) f4 = fac[q >> 2];
            const float n1[4] = {n4.x, n4.y, n4.z, n4.w}, f1[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float y = __uint_as_float(s[i]);
              if (lo) y += __uint_as_float(s2[i]);
              // (key_scale is 1 and the LSE in the product already where the operands are bf16)
              const float e = ex2_approx(fmaf(y * key_scale, f1[i], narrow ? n1[i] : 0.f));
              if (q + i >= c0 && n1[i] != -INFINITY) (i & 1 ? a0.y : a0.x) += e;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_s_free(bf));
        sum += (a0.x + a0.y) + (a1.x + a1.y);
        if (single) {
          if (j == j0) {
            before = sum;
            sum = 0.f;
          }
        } else {
          if (lane == 0) mbar_arrive(bar_lse_free(l.st, bf));
          l.next(C::kLse);
        }
      }
      if (!ok) break;
      if (single) {
        __syncwarp();
        ok = pass();
        if (!ok) break;
        // (the old weights have had both steps' time to come)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (at[i] >= 0) p.out[at[i]] = fmaf(p.decay, old[i], i ? sum : before);
      } else {
        // the sum of the even tiles and of the odd ones: the same two whichever pair has which
        const int slot = u % kWeighParts;
        if (!last) {
          parts[slot * 256] = sum;
        } else {
          ok = __all_sync(0xffffffffu, tile_wait(bar_part(slot, blk), (u / kWeighParts) & 1, wc, 79));
          if (!ok) break;
          sum += parts[slot * 256];
          if (at[0] >= 0) p.out[at[0]] = fmaf(p.decay, old[0], sum);
        }
      }
      // (every unit, so that a slot's turns follow from u; in a unit of one tile by the pair that has its second step)
      if (single ? j0 == 1 : !last) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_part(u % kWeighParts, blk));
      }
      g += n;
      x += 2 * (single ? n : 1);
    }
  } else if (kF8 && warp >= kWeighConvWarp) {
    // ================================================================ operands in another form (e4m3)
    if constexpr (kF8) {
      const int r = threadIdx.x - 32 * kWeighConvWarp;
      WeighRing k, q, w;
      uint32_t u = 0, x = 0;  // units, blocks
      bool ok = true;
      WeighUnit t;
      for (; job(t, ok, 75); ++u) {
        const int first = t.first();
        if (t.nq == 1) {
          // ---- the queries as two e4m3 terms, a lane 8 columns
          constexpr int kL = D / 8;  // lanes of a row
          // (w_free first: after several tiles, which this role does not wait for, it says that the last of them
          // have come, and so that q_full is at this tile's turn)
          ok = tile_wait(bar_w_free(w.st), w.ph ^ 1u, wc, 77) && tile_wait(bar_q_full(q.st), q.ph, wc, 76);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const int rows = weigh_cols(p, first, t.T, 0).n, ch = lane % kL;
          const bool stacked = rows <= kWeighStacked;  // the second terms are rows after the first ones, or a tile
          const uint8_t* src = smem + q.st * C::kTileBytes;
          uint8_t* dst = smem + C::kOffWide + w.st * C::kTileBytes;
          float* fac = reinterpret_cast<float*>(smem + C::kOffFactor) + (u % kWeighFactors) * 128;
#pragma unroll 1
          for (int r0 = (warp - kWeighConvWarp) * (32 / kL); r0 < rows; r0 += 4 * (32 / kL)) {
            const int qr = r0 + lane / kL;
            const uint4 x = *reinterpret_cast<const uint4*>(src + (ch / 8) * C::kSubBytes + qr * 128 + (((ch & 7) ^ (qr & 7)) << 4));
            uint32_t mx = finite_max(x);  // largest finite magnitude; bit 31: one is not
            if (any_nonfinite(x.x) || any_nonfinite(x.y) || any_nonfinite(x.z) || any_nonfinite(x.w)) mx |= 0x80000000u;
#pragma unroll
            for (int o = kL / 2; o > 0; o >>= 1) mx = max(mx & 0x7fffffffu, __shfl_xor_sync(0xffffffffu, mx, o) & 0x7fffffffu) |
                                                    ((mx | __shfl_xor_sync(0xffffffffu, mx, o)) & 0x80000000u);
            const uint32_t ef = min(max((mx & 0x7fffffffu) >> 7, 8u), 253u);  // exponent field of the row's largest value
            const float up = __uint_as_float((261u - ef) << 23);              // brings it into [128, 256)
            // a row that is not finite makes its keys' weights NaN
            if (ch == 0) fac[qr] = (mx >> 31) == 0u ? p.c * __uint_as_float((ef - 7u) << 23) : NAN;
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // four values each
              const float f0 = bf16_lo(v[2 * i]) * up, f1 = bf16_hi(v[2 * i]) * up;
              const float f2 = bf16_lo(v[2 * i + 1]) * up, f3 = bf16_hi(v[2 * i + 1]) * up;
              const uint32_t h0 = pack_e4m3x2(f0, f1), h1 = pack_e4m3x2(f2, f3);
              const float2 b0 = e4m3x2_to_f32(h0), b1 = e4m3x2_to_f32(h1);
              hi[i] = h0 | (h1 << 16);
              lo[i] = pack_e4m3x2(f0 - b0.x, f1 - b0.y) | (pack_e4m3x2(f2 - b1.x, f3 - b1.y) << 16);
            }
            const int sx = D == 128 ? (ch >> 1) ^ (qr & 7) : (ch >> 1) ^ ((qr >> 1) & 3);  // (rows 16 apart alike)
            uint8_t* to = dst + qr * D + (sx << 4) + (ch & 1) * 8;
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to + (stacked ? (rows + 15) / 16 * 16 : 128) * D) = make_uint2(lo[0], lo[1]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_w_full(w.st));
          w.next(NWm);
          for (int i = 0; i < 2 * t.steps; ++i) k.next(p.ring_k);
          x += 2 * t.steps;
        } else {
          // ---- both blocks of keys: codes times scale as bf16, a thread a key
          // This role does not wait for the keys of a unit with one tile.  Both stages free: its products are
          // done, its keys have come, and k_full is at this unit's turn (a turn too early, the stage would be
          // handed back before its copy has landed).
          {
            WeighRing both = w;
#pragma unroll 1
            for (int h = 0; ok && h < 2; ++h, both.next(NWm)) ok = __all_sync(0xffffffffu, tile_wait(bar_w_free(both.st), both.ph ^ 1u, wc, 77));
            if (!ok) break;
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h, ++x, w.next(NWm), k.next(p.ring_k)) {
            ok = __all_sync(0xffffffffu, tile_wait(bar_k_full(k.st), k.ph, wc, 78));
            if (!ok) break;
            const uint8_t* src = smem + p.ring_q * C::kTileBytes + k.st * C::kStageK + r * D;
            uint8_t* dst = smem + C::kOffWide + w.st * C::kTileBytes + r * 128;
            const uint32_t code = smem[C::kOffCode + (x % kWeighCodes) * 128 + r];
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
            if (lane == 0) mbar_arrive(bar_w_full(w.st));
          }
          if (!ok) break;
        }
        for (int j = 0; j < t.nq; ++j) q.next(p.ring_q);
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

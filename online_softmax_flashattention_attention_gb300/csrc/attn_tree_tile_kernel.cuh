// Attention of drafted tokens over a paged cache, units of up to 128 rows, sm_103a.
//
// The operation, units and work split of attn_tree_kernel.cuh, for calls whose drafted tokens
// and grouped heads make more rows than one 16-row tile: there every further tile reads the
// keys again and its warp-level products become the limit.  Here a tile holds the G heads of
// 128 / G tokens as the 128 lanes of tensor memory, and the products are tcgen05.mma: per
// block of 128 keys S = Q K^T (128 x 128 x d, into one of three score buffers) and
// o~ += P V, with P written back over S as bf16.  One CTA an SM, persistent over its range of
// the list of chunks (128 keys each).
//
// Warps: 0-3 softmax, thread r owns row r (tensor-memory lane r); 4 producer (TMA); 5 issues
// P V; 6 issues S; 7 (bf16) repairs V blocks at a sequence's end, see below; 8-11 (e4m3)
// convert blocks to bf16 with their scales, 128 keys x d values a block, exact.
//
// K and V blocks are up to eight boxes of 16 keys, each from the page it lies in (larger boxes
// when the page size allows: fewer copies).  A block that holds drafted keys, or keys past the
// end, or a page that does not exist, is "ragged": its V rows that must not count are zeroed
// (0 * NaN is NaN), and infinities and NaN in V of drafted keys are zeroed too and remembered:
// rows that see them get them added in the epilogue, rows that do not never meet them.
#pragma once

#include "attn_tree_kernel.cuh"

namespace attn {

constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kTileWarpTma = 4;
constexpr int kTileWarpPv = 5;
constexpr int kTileWarpS = 6;
constexpr int kTileWarpFix = 7;
constexpr uint32_t kTileRegsSoftmax = 232;  // of 3 x 168 (e4m3: 384 threads): 232 + 104 + 168 = 504
constexpr uint32_t kTileRegsOther = 104;
constexpr int kTileTags = 16;

template <int D, bool kF8>
struct TileCfg {
  static constexpr int kThreads = kF8 ? 384 : 256;
  static constexpr int kSub = D / 64;                    // 64-column sub-tiles of a bf16 row
  static constexpr int kSubBytes = 128 * 128;            // 128 rows x 64 bf16
  static constexpr int kTileBytes = kSub * kSubBytes;    // a block of K, V or Q in bf16
  static constexpr int kRawBytes = 128 * D;              // a block of K or V in e4m3
  static constexpr int kStages = kF8 ? (D == 64 ? 3 : 2) : (D == 64 ? 4 : 3);
  static constexpr int kRaw = kF8 ? 2 : 0;               // e4m3 stages
  static constexpr int kSBufs = 3;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffRaw = kOffV + kStages * kTileBytes;          // K then V of each raw stage
  static constexpr int kOffScale = kOffRaw + kRaw * 2 * kRawBytes;      // 128 codes of K, 128 of V a stage
  static constexpr int kOffBar = kOffScale + kRaw * 256;
  // q_full, q_free, {k_full, v_full, k_free, v_free, v_fixed}[S], {s_full, pv_done, p_full}[B],
  // drain[2], {rk_full, rv_full, rk_free, rv_free}[R]
  static constexpr int kNumBars = 2 + 5 * kStages + 3 * kSBufs + 2 + 4 * kRaw;
  static constexpr int kOffPre = kOffBar + 8 * kNumBars;
  static constexpr int kOffMisc = kOffPre + 8 * (kPlanGroups + 1 + 4);  // tmem base, abort, valid[8], tags[16]
  static constexpr int kSmem = kOffMisc + 8 + 32 + 4 * kTileTags + 1024;
  static_assert(kSmem <= 232448, "shared memory per CTA");
  __host__ __device__ static constexpr uint32_t col_s(int b) { return 128u * b; }
  static constexpr uint32_t kColO = 128u * kSBufs;
  static constexpr uint32_t kIdescS = idesc_bf16_f32(kTileRows, kTileKeys, 0);
  static constexpr uint32_t kIdescO = idesc_bf16_f32(kTileRows, D, 1);
  static_assert(kColO + D <= 512, "tensor memory");
};

// A bf16 pair with its infinite and NaN halves zeroed.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
  return w;
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

template <int D, bool kF8>
__global__ void __launch_bounds__(TileCfg<D, kF8>::kThreads, 1)
    attn_tree_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const TreeParams p) {
  using C = TileCfg<D, kF8>;
  constexpr int S = C::kStages, NB = C::kSBufs, R = C::kRaw > 0 ? C::kRaw : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + C::kOffQ, sK = sbase + C::kOffK, sV = sbase + C::kOffV;
  const uint32_t bar0 = sbase + C::kOffBar;
  const uint32_t bar_q_full = bar0, bar_q_free = bar0 + 8u;
  auto bar_k_full = [&](int s) { return bar0 + 8u * (2 + s); };
  auto bar_v_full = [&](int s) { return bar0 + 8u * (2 + S + s); };
  auto bar_k_free = [&](int s) { return bar0 + 8u * (2 + 2 * S + s); };
  auto bar_v_free = [&](int s) { return bar0 + 8u * (2 + 3 * S + s); };
  auto bar_v_fixed = [&](int s) { return bar0 + 8u * (2 + 4 * S + s); };
  auto bar_s_full = [&](int b) { return bar0 + 8u * (2 + 5 * S + b); };
  auto bar_pv_done = [&](int b) { return bar0 + 8u * (2 + 5 * S + NB + b); };
  auto bar_p_full = [&](int b) { return bar0 + 8u * (2 + 5 * S + 2 * NB + b); };
  auto bar_drain = [&](int i) { return bar0 + 8u * (2 + 5 * S + 3 * NB + i); };
  auto bar_raw = [&](int kind, int s) { return bar0 + 8u * (4 + 5 * S + 3 * NB + kind * C::kRaw + s); };
  long long* pre = reinterpret_cast<long long*>(smem + C::kOffPre);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 4);
  // valid[g % 8]: which 16-key slices of block g exist (written before the block's copies are
  // announced; a ring is at most four blocks deep)
  volatile uint32_t* valid = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 8);
  // tag[u % 16] = u + 1 once unit u (of this CTA) has met an infinite or NaN drafted value
  volatile uint32_t* tag = reinterpret_cast<volatile uint32_t*>(smem + C::kOffMisc + 40);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx wc{abort_flag, p.status, p.timeout_ns};

  if (threadIdx.x == 0) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_free, 1);
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_k_full(s), kF8 ? 4 : 1);
      mbar_init(bar_v_full(s), kF8 ? 4 : 1);
      mbar_init(bar_k_free(s), 1);
      mbar_init(bar_v_free(s), 1);
      mbar_init(bar_v_fixed(s), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(bar_s_full(b), 1);
      mbar_init(bar_pv_done(b), 1);
      mbar_init(bar_p_full(b), 4);
    }
    mbar_init(bar_drain(0), 1);
    mbar_init(bar_drain(1), 1);
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(bar_raw(0, s), 1);
      mbar_init(bar_raw(1, s), 1);
      mbar_init(bar_raw(2, s), 4);
      mbar_init(bar_raw(3, s), 4);
    }
    *abort_flag = 0u;
    for (int i = 0; i < kTileTags; ++i) tag[i] = 0u;
    fence_mbar_init();
  }
  if (warp == kTileWarpPv) tmem_alloc<512>(smem_u32(tmem_slot));
  if (warp == kTileWarpTma && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  griddep_wait();
  griddep_launch_dependents();
  const int gs = (p.B + kPlanGroups - 1) / kPlanGroups;
  tc_fence_before();
  tree_plan<kTileRows, kTileKeys>(p, gs, pre, pre + kPlanGroups + 1);  // ends with a barrier of the CTA
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long W = pre[kPlanGroups];
  const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  const long long per = W / grid, extra = W % grid;
  const long long x0 = per * cta + min(static_cast<long long>(cta), extra);
  const long long x1 = x0 + per + (cta < extra ? 1 : 0);

  // Every role walks the same pieces; g counts their blocks, u the pieces themselves.
  if (warp == kTileWarpTma) {
    // ================================================================ producer
    if constexpr (kF8) setmaxnreg_dec<kTileRegsOther>();
    const uint64_t pol = policy_evict_first();
    constexpr int kRing = kF8 ? R : S;
    const int box16 = p.box_rows / 16;  // slices a box holds
    int g = 0, u = 0;
    uint32_t k_live = 0, k_par = 0, v_live = 0, v_par = 0;
    bool ok = true;
    for (long long x = x0; ok && x < x1;) {
      const TreePiece pc = tree_piece<kTileRows, kTileKeys>(p, gs, pre, x, x1);
      x += pc.adv;
      if (pc.ch1 <= pc.ch0) continue;
      if (u > 0) ok = mbar_wait(bar_q_free, (u - 1) & 1, wc, 33);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar_q_full, C::kSub * p.tok_tile * p.G * 128);
        for (int s = 0; s < C::kSub; ++s)
          tma_load_4d(sQ + s * C::kSubBytes, &tmQ, bar_q_full, s * 64, 0, pc.h, pc.s.q0 + pc.tile * p.tok_tile, pol);
      }
      ++u;
      // lane i < 8 looks after slice i of a block; its page is fetched a block ahead
      auto page_of = [&](int j) {
        const long long pos = static_cast<long long>(j) * kTileKeys + 16 * lane;
        const bool need = lane < 8 && j < pc.ch1 && pos < pc.s.n;
        return need ? __ldg(p.table + static_cast<long long>(pc.b) * p.max_pages + static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page)) : -1;
      };
      int next = page_of(pc.ch0);
      for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
        const int pg = next;
        next = page_of(j + 1);
        const bool have = static_cast<unsigned>(pg) < static_cast<unsigned>(p.num_pages);
        if (!have && lane < 8 && static_cast<long long>(j) * kTileKeys + 16 * lane < pc.s.n && p.page_word)
          atomicOr(p.page_word, 1u);
        const uint32_t vm = __ballot_sync(0xffffffffu, have && lane < 8);
        const int row = static_cast<int>((static_cast<uint32_t>(j) * kTileKeys + 16u * lane) % static_cast<uint32_t>(p.page));
        const bool mine = have && lane < 8 && lane % box16 == 0;
        const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
        const int st = g % kRing;
        const uint32_t ph = (g / kRing) & 1, bit = 1u << st;
        const uint32_t kfree = kF8 ? bar_raw(2, st) : bar_k_free(st), vfree = kF8 ? bar_raw(3, st) : bar_v_free(st);
        const uint32_t kfull = kF8 ? bar_raw(0, st) : bar_k_full(st), vfull = kF8 ? bar_raw(1, st) : bar_v_full(st);
        constexpr int kRowB = kF8 ? D : 128;                 // bytes of a row of a (sub-)tile
        constexpr int kSubs = kF8 ? 1 : C::kSub;
        const uint32_t kdst = kF8 ? sbase + C::kOffRaw + st * 2 * C::kRawBytes : sK + st * C::kTileBytes;
        const uint32_t vdst = kF8 ? kdst + C::kRawBytes : sV + st * C::kTileBytes;
        const uint32_t bytes = boxes * p.box_rows * (kSubs * kRowB + (kF8 ? 1 : 0));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          ok = __all_sync(0xffffffffu, mbar_wait(kv ? vfree : kfree, ph ^ 1, wc, 34 + kv));
          if (!ok) break;
          const uint32_t full = kv ? vfull : kfull;
          if (lane == 0) {
            if (kv == 0) valid[g & 7] = vm;
            mbar_arrive_expect_tx(full, bytes);
          }
          __syncwarp();
          if (mine) {
            const uint32_t dst = (kv ? vdst : kdst) + 16 * lane * kRowB;
#pragma unroll
            for (int s = 0; s < kSubs; ++s)
              tma_load_4d(dst + s * C::kSubBytes, kv ? &tmV : &tmK, full, s * 64, row, pc.h, pg, pol);
            if constexpr (kF8) {
              const long long r = (static_cast<long long>(pg) * p.Hkv + pc.h) * p.page + row;
              bulk_load(sbase + C::kOffScale + st * 256 + kv * 128 + 16 * lane, (kv ? p.vs : p.ks) + r, p.box_rows, full);
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
        if (!ok) break;
      }
    }
    // let the copies in flight land before this warp leaves
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < kRing; ++s) {
        if ((k_live >> s) & 1u) mbar_wait_drain(kF8 ? bar_raw(0, s) : bar_k_full(s), (k_par >> s) & 1u, p.timeout_ns);
        if ((v_live >> s) & 1u) mbar_wait_drain(kF8 ? bar_raw(1, s) : bar_v_full(s), (v_par >> s) & 1u, p.timeout_ns);
      }
      if (u > 0) mbar_wait_drain(bar_q_full, (u - 1) & 1, p.timeout_ns);
    }
  } else if (warp == kTileWarpPv || warp == kTileWarpS) {
    // ================================================================ products
    if constexpr (kF8) setmaxnreg_dec<kTileRegsOther>();
    if (lane == 0) {
      const uint32_t dhi = (1024u >> 4) | (1u << 14) | (2u << 29);
      int g = 0, u = 0;
      bool ok = true;
      uint32_t fixed_par = 0;  // parity each v_fixed completes next
      for (long long x = x0; ok && x < x1;) {
        const TreePiece pc = tree_piece<kTileRows, kTileKeys>(p, gs, pre, x, x1);
        x += pc.adv;
        if (pc.ch1 <= pc.ch0) continue;
        if (warp == kTileWarpS) {
          const uint32_t qlo = (sQ >> 4) | (1u << 16);
          const uint32_t klo = (sK >> 4) | (1u << 16);
          ok = mbar_wait(bar_q_full, u & 1, wc, 36);
          for (int j = pc.ch0; ok && j < pc.ch1; ++j, ++g) {
            const int st = g % S, bf = g % NB;
            if (g >= NB) ok = mbar_wait(bar_pv_done(bf), ((g - NB) / NB) & 1, wc, 37);
            ok = ok && mbar_wait(bar_k_full(st), (g / S) & 1, wc, 38);
            if (!ok) break;
            tc_fence_after();
            const uint32_t blo = klo + st * (C::kTileBytes >> 4);
            const uint32_t dst = tmem + C::col_s(bf);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks / 4) * (C::kSubBytes >> 4) + (ks % 4) * 2;
              mma_ss(dst, (static_cast<uint64_t>(dhi) << 32) | (qlo + off),
                     (static_cast<uint64_t>(dhi) << 32) | (blo + off), C::kIdescS, ks > 0 ? 1u : 0u);
            }
            mma_commit(bar_s_full(bf));
            mma_commit(bar_k_free(st));
          }
          if (!ok) break;
          mma_commit(bar_q_free);
        } else {
          const uint32_t vlo = (sV >> 4) | (static_cast<uint32_t>(C::kSubBytes >> 4) << 16);
          for (int j = pc.ch0; ok && j < pc.ch1; ++j, ++g) {
            const int st = g % S;
            ok = mbar_wait(bar_v_full(st), (g / S) & 1, wc, 39);
            if (!kF8 && ok && (static_cast<long long>(j + 1) * kTileKeys > pc.s.ctx || valid[g & 7] != 0xffu)) {
              ok = mbar_wait(bar_v_fixed(st), (fixed_par >> st) & 1u, wc, 40);
              fixed_par ^= 1u << st;
            }
            ok = ok && mbar_wait_poll(bar_p_full(g % NB), (g / NB) & 1, wc, 41);
            if (!ok) break;
            tc_fence_after();
            const uint32_t blo = vlo + st * (C::kTileBytes >> 4);
            const uint32_t a = tmem + C::col_s(g % NB);
#pragma unroll
            for (int ks = 0; ks < kTileKeys / 16; ++ks)
              mma_ts(tmem + C::kColO, a + ks * 8, (static_cast<uint64_t>(dhi) << 32) | (blo + ks * (16 * 128 >> 4)),
                     C::kIdescO, (j > pc.ch0 || ks > 0) ? 1u : 0u);
            mma_commit(bar_pv_done(g % NB));
            mma_commit(bar_v_free(st));
          }
        }
        ++u;
      }
      mma_commit(bar_drain(warp == kTileWarpS));
      mbar_wait_drain(bar_drain(warp == kTileWarpS), 0, p.timeout_ns);
    }
  } else if (warp == kTileWarpFix) {
    // ================================================================ ragged blocks of V (bf16)
    if constexpr (kF8) {
      setmaxnreg_dec<kTileRegsOther>();  // the warp without a role completes its warpgroup
    } else {
      int g = 0, u = 0;
      bool ok = true;
      for (long long x = x0; ok && x < x1;) {
        const TreePiece pc = tree_piece<kTileRows, kTileKeys>(p, gs, pre, x, x1);
        x += pc.adv;
        if (pc.ch1 <= pc.ch0) continue;
        for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
          const int st = g % S, kb = j * kTileKeys;
          ok = __all_sync(0xffffffffu, mbar_wait(bar_v_full(st), (g / S) & 1, wc, 42));
          if (!ok) break;
          const uint32_t vm = valid[g & 7];
          if (static_cast<long long>(kb) + kTileKeys <= pc.s.ctx && vm == 0xffu) continue;
          bool odd = false;
          for (int i = lane; i < kTileKeys * (D / 8); i += 32) {
            const int r = i / (D / 8), ch = i % (D / 8);
            const bool here = ((vm >> (r / 16)) & 1u) && kb + r < pc.s.n;
            if (here && kb + r < pc.s.ctx) continue;
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
          if (lane == 0) mbar_arrive(bar_v_fixed(st));
        }
        ++u;
      }
    }
  } else if (kF8 && warp >= 8) {
    // ================================================================ e4m3 -> bf16
    if constexpr (kF8) {
      const int r = threadIdx.x - 256;  // key of the block
      int g = 0, u = 0;
      bool ok = true;
      for (long long x = x0; ok && x < x1;) {
        const TreePiece pc = tree_piece<kTileRows, kTileKeys>(p, gs, pre, x, x1);
        x += pc.adv;
        if (pc.ch1 <= pc.ch0) continue;
        for (int j = pc.ch0; ok && j < pc.ch1; ++j, ++g) {
          const int st = g % S, rs = g % R, kb = j * kTileKeys;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            ok = mbar_wait(bar_raw(kv, rs), (g / R) & 1, wc, 43 + kv) &&
                 mbar_wait(kv ? bar_v_free(st) : bar_k_free(st), ((g / S) & 1) ^ 1, wc, 45 + kv);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t vm = valid[g & 7];
            const bool here = ((vm >> (r / 16)) & 1u) && kb + r < pc.s.n;
            const bool scan = kv && kb + r >= pc.s.ctx;
            const uint8_t* src = smem + C::kOffRaw + rs * 2 * C::kRawBytes + kv * C::kRawBytes + r * D;
            uint8_t* dst = smem + (kv ? C::kOffV : C::kOffK) + st * C::kTileBytes + r * 128;
            const uint32_t code = smem[C::kOffScale + rs * 256 + kv * 128 + r];
            const uint32_t two = (code << 7) | (code << 23);  // 2^(code - 127) twice, as bf16
            const __nv_bfloat162 scale = *reinterpret_cast<const __nv_bfloat162*>(&two);
            bool odd = false;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const int sw = D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
              const uint4 raw = *reinterpret_cast<const uint4*>(src + (sw << 4));
              uint4 a = widen8(raw.x, raw.y, scale), b = widen8(raw.z, raw.w, scale);
              if (!here) {
                a = make_uint4(0, 0, 0, 0);
                b = make_uint4(0, 0, 0, 0);
              } else if (scan) {
                if (any_nonfinite(a.x) || any_nonfinite(a.y) || any_nonfinite(a.z) || any_nonfinite(a.w) ||
                    any_nonfinite(b.x) || any_nonfinite(b.y) || any_nonfinite(b.z) || any_nonfinite(b.w)) {
                  odd = true;
                  a = make_uint4(finite_only(a.x), finite_only(a.y), finite_only(a.z), finite_only(a.w));
                  b = make_uint4(finite_only(b.x), finite_only(b.y), finite_only(b.z), finite_only(b.w));
                }
              }
              // 16 columns = chunks 2 c, 2 c + 1 of the bf16 row, in sub-tile c / 4
              uint8_t* to = dst + (c / 4) * C::kSubBytes;
              const int ch = (2 * c) & 7;
              *reinterpret_cast<uint4*>(to + ((ch ^ (r & 7)) << 4)) = a;
              *reinterpret_cast<uint4*>(to + (((ch + 1) ^ (r & 7)) << 4)) = b;
            }
            if (odd) tag[u % kTileTags] = u + 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(kv ? bar_v_full(st) : bar_k_full(st));
              mbar_arrive(bar_raw(2 + kv, rs));
            }
          }
        }
        ++u;
      }
    }
  } else {
    // ================================================================ softmax
    if constexpr (kF8) setmaxnreg_inc<kTileRegsSoftmax>();
    const int r = threadIdx.x;
    const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float c = p.c;
    constexpr float kTau = 8.f;  // o~ is rescaled when the max rises by more (log2 units)
    int g = 0, u = 0;
    bool ok = true, has_tail = false;
    for (long long x = x0; ok && x < x1;) {
      const TreePiece pc = tree_piece<kTileRows, kTileKeys>(p, gs, pre, x, x1);
      x += pc.adv;
      if (pc.ch1 <= pc.ch0) continue;
      int tok, head;
      const bool row_here = tree_row<kTileRows>(p, pc.s, pc.tile, r, &tok, &head);
      const unsigned long long sees = row_here ? tree_sees(p, pc.s, tok) : 0ull;
      const bool idle = !__any_sync(0xffffffffu, row_here);  // no row of this warp exists
      float m = -INFINITY, l = 0.f;
      for (int j = pc.ch0; j < pc.ch1; ++j, ++g) {
        const uint32_t colS = C::col_s(g % NB);
        ok = __all_sync(0xffffffffu, mbar_wait(bar_s_full(g % NB), (g / NB) & 1, wc, 47));
        if (!ok) break;
        if (idle) {  // its lanes of P hold scores: rows nobody reads
          if (lane == 0) mbar_arrive(bar_p_full(g % NB));
          continue;
        }
        tc_fence_after();
        float s[kTileKeys];
        {
          uint32_t sr[kTileKeys];
#pragma unroll
          for (int q = 0; q < kTileKeys / 32; ++q) tmem_ld32(tl + colS + q * 32, sr + q * 32);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < kTileKeys; ++k) s[k] = __uint_as_float(sr[k]);
        }
        const int kb = j * kTileKeys;
        const uint32_t vm = valid[g & 7];
        if (static_cast<long long>(kb) + kTileKeys > pc.s.ctx || vm != 0xffu) {
          const int off = pc.s.ctx - kb;  // context keys of the block; the drafted ones follow
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int o = off - 32 * w;
            uint32_t see = o >= 32 ? 0xffffffffu : o <= 0 ? 0u : (1u << o) - 1u;
            if (o < 32 && o > -64) see |= static_cast<uint32_t>(o >= 0 ? sees << o : sees >> -o);
            if (!((vm >> (2 * w)) & 1u)) see &= 0xffff0000u;
            if (!((vm >> (2 * w + 1)) & 1u)) see &= 0x0000ffffu;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((see >> k) & 1u)) s[32 * w + k] = -INFINITY;
          }
        }
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = fmaxf(s[2 * i], s[2 * i + 1]);
#pragma unroll
        for (int k = 16; k < kTileKeys; k += 16)
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = fmax3(a[i], s[k + 2 * i], s[k + 2 * i + 1]);
        const float mx = fmaxf(fmaxf(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5])), fmaxf(a[6], a[7])) * c;
        const float m_new = mx > m + kTau ? mx : m;
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = ex2_approx(m - ref);
        const float2 c2 = make_float2(c, c), nm2 = make_float2(-ref, -ref);
        float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < kTileKeys / 32; ++q) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 e = __ffma2_rn(make_float2(s[q * 32 + 2 * k], s[q * 32 + 2 * k + 1]), c2, nm2);
            e.x = ex2_approx(e.x);
            e.y = ex2_approx(e.y);
            if (k & 1)
              acc1 = __fadd2_rn(acc1, e);
            else
              acc0 = __fadd2_rn(acc0, e);
            // P to bf16 (relative 2^-8 at most), as in attn_tree_kernel
            pk[k] = pack_bf16x2(e.x, e.y);
          }
          tmem_st16(tl + colS + q * 16, pk);
        }
        const float2 acc = __fadd2_rn(acc0, acc1);
        l = l * alpha + (acc.x + acc.y);
        const bool moved = m_new != m;
        m = m_new;
        if (j > pc.ch0 && __any_sync(0xffffffffu, moved)) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar_pv_done((g - 1) % NB), ((g - 1) / NB) & 1, wc, 48));
          if (!ok) break;
          tc_fence_after();
          const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tl + C::kColO + q * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), al2);
              o[2 * k] = __float_as_uint(v.x);
              o[2 * k + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tl + C::kColO + q * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full(g % NB));
      }
      if (!ok) break;
      // ---- o~ out: the piece's last P V (and so all of them) has landed
      ok = __all_sync(0xffffffffu, mbar_wait(bar_pv_done((g - 1) % NB), ((g - 1) / NB) & 1, wc, 49));
      if (!ok) break;
      tc_fence_after();
      const bool whole = pc.ch0 == 0 && pc.ch1 == pc.s.nch;
      if (!idle) {
        uint32_t o[D];
#pragma unroll
        for (int q = 0; q < D / 32; ++q) tmem_ld32(tl + C::kColO + q * 32, o + q * 32);
        tmem_wait_ld();
        if (tag[u % kTileTags] == static_cast<uint32_t>(u + 1)) {
          // infinities and NaN among the drafted values of this piece, zero in the product: to
          // the rows that see them (a positive weight leaves them what they are)
          for (unsigned long long left = sees; left; left &= left - 1) {
            const int pos = pc.s.ctx + __ffsll(static_cast<long long>(left)) - 1;
            if (pos >= pc.s.n || pos < pc.ch0 * kTileKeys || pos - kTileKeys >= (pc.ch1 - 1) * kTileKeys) continue;
            const int pg = __ldg(p.table + static_cast<long long>(pc.b) * p.max_pages + pos / p.page);
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) continue;
            const long long at = (static_cast<long long>(pg) * p.Hkv + pc.h) * p.page + pos % p.page;
#pragma unroll
            for (int k = 0; k < D / 2; ++k) {
              uint32_t w;
              if constexpr (kF8) {
                const uint32_t two = (static_cast<uint32_t>(__ldg(p.vs + at)) << 7) | (static_cast<uint32_t>(__ldg(p.vs + at)) << 23);
                const uint32_t cw = e4m3x2_to_bf16x2(__ldg(reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.v) + at * D) + k));
                const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&cw), *reinterpret_cast<const __nv_bfloat162*>(&two));
                w = *reinterpret_cast<const uint32_t*>(&v);
              } else {
                w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.v) + at * D) + k);
              }
              if (!isfinite(bf16_lo(w))) o[2 * k] = __float_as_uint(__uint_as_float(o[2 * k]) + bf16_lo(w));
              if (!isfinite(bf16_hi(w))) o[2 * k + 1] = __float_as_uint(__uint_as_float(o[2 * k + 1]) + bf16_hi(w));
            }
          }
        }
        if (row_here) {
          if (whole) {
            const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
            const int hq = pc.h * p.G + head;
            uint4* dst = reinterpret_cast<uint4*>(p.o + (static_cast<long long>(pc.s.q0 + tok) * p.Hq + hq) * D);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__uint_as_float(o[8 * k + 2 * i]) * inv, __uint_as_float(o[8 * k + 2 * i + 1]) * inv);
              dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            p.lse[static_cast<long long>(hq) * p.total_q + pc.s.q0 + tok] =
                l > 0.f || l != l ? m * 0.69314718055994531f + logf(l) : -INFINITY;
          } else {
            const long long at = static_cast<long long>(2 * cta + (pc.ch0 == 0 ? 1 : 0)) * kTileRows + r;
            float4* dst = reinterpret_cast<float4*>(p.st_o + at * D);
#pragma unroll
            for (int k = 0; k < D / 4; ++k)
              dst[k] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                   __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
            p.st_m[at] = m;
            p.st_l[at] = l;
          }
        }
      }
      // o~ has been read out: the next piece's first P V comes after this thread's next arrival
      tc_fence_before();
      if (pc.ch0 == 0 && pc.ch1 < pc.s.nch) {
        has_tail = true;
        if (r == 0)
          p.meta[cta] = make_int4(pc.b, pc.h, pc.tile, tree_owner(x + (pc.s.nch - pc.ch1) - 1, per, extra));
      }
      ++u;
    }
    if (!has_tail && r == 0) p.meta[cta] = make_int4(0, 0, 0, -1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kTileWarpPv) {
    tc_fence_after();
    tmem_dealloc<512>(*reinterpret_cast<volatile uint32_t*>(tmem_slot));
  }
}

}  // namespace attn

// The paged key/value cache: writing packed new tokens into it and reading cached positions
// back, sm_103a.
//
// Cache: k, v [num_pages, Hkv, page, d], bf16 or e4m3; e4m3 rows carry one scale code each,
// uint8 [num_pages, Hkv, page], value = code * 2^(s - 127).  Position p of sequence b is row
// p % page of page block_table[b, p / page].
//
// Quantisation of a row x: a = max |x_i| over its finite values, e the least integer >= -126
// with a <= 448 * 2^e (448: the largest e4m3 value), s = e + 127, code_i = x_i * 2^-e to the
// nearest e4m3 value, ties to even; infinities become +-448, NaN stays NaN.  With a power of
// two for a scale both x * 2^-e and code * 2^e are exact, so the one rounding to e4m3 (half a
// step: relative 2^-4, or 2^-10 * 2^e where the code is subnormal) is all that is lost, and a
// value read back is exactly a bf16.  (At e = 120, the largest there is, magnitudes past
// 240 * 2^120 are brought back to it: the next value up, 2^128, is no bf16.)  One byte a row is
// 1/128 of the codes at d = 128.
//
// Both kernels only move bytes.  d / 8 lanes own one (token, head) row of K and of V: one
// 16-byte bf16 access a lane, and for the row maximum a few shuffles.  A thread has the loads
// of kCacheUnroll rows of K and V in flight; in the write they do not depend on where the
// rows go, so they are issued before the sequence of a token is searched for.
//
// Bound: DRAM; the e4m3 write also by instructions (two thirds of the issue slots: the row
// maximum, eight products and four conversions a lane).  Measured on GB300, 8 heads, d = 128:
// 9 prompts of 900 to 16384 tokens into an e4m3 cache, 262 MB in 48.4 us, 5.4 TB/s; 6 prefixes of
// 3000 to 32768 tokens out of one, 772 MB in 126 us, 6.1 TB/s; one token 2.8 us, a launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace attn {

constexpr int kCacheThreads = 256;
constexpr int kCacheUnroll = 4;  // rows of K and of V a lane group has in flight

// What the entry points say about a cache and its block table.
struct CacheParams {
  void* k;                  // [num_pages, Hkv, page, d]
  void* v;
  uint8_t* ks;              // [num_pages, Hkv, page], e4m3 only
  uint8_t* vs;
  const int32_t* table;     // [B, max_pages]
  const int32_t* cu;        // [B + 1] packed rows of the sequences
  const int32_t* start;     // [B] first position of each sequence's rows, or null (0)
  int B, Hkv, num_pages, page, max_pages;
  int total;                // packed rows
  int step_t, step_h;       // write: a block's row groups, in tokens and heads
  const __nv_bfloat16* src_k;  // write: packed K and V, element (t, h, x) at t * st + h * sh + x
  const __nv_bfloat16* src_v;
  long long k_st, k_sh, v_st, v_sh;
  __nv_bfloat16* dst_k;     // read: [total, Hkv, d]
  __nv_bfloat16* dst_v;
  uint32_t* page_word;      // bit 0: a position without a page, or a page outside the cache
};

// Row (of head 0) of packed token `tok` in the cache, in units of rows: page * Hkv * page_size
// + row in the page; -1 when the token is in no sequence, -2 when its position has no page.
// The sequence is the last one that starts at or before the token; a block table or a
// cu_seqlens that holds anything at all leads to a row inside the cache or to none.
__device__ __forceinline__ long long cache_row_of(const CacheParams& p, int tok) {
  int lo = 0, hi = p.B;  // the sequence is in [lo, hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (__ldg(p.cu + mid) <= tok)
      lo = mid;
    else
      hi = mid;
  }
  const int first = max(__ldg(p.cu + lo), 0);
  if (tok < first || tok >= __ldg(p.cu + lo + 1)) return -1;
  const int start = p.start ? max(__ldg(p.start + lo), 0) : 0;
  const long long pos = static_cast<long long>(start) + (tok - first);
  if (pos >= static_cast<long long>(p.max_pages) * p.page) return -2;
  const int slot = static_cast<int>(static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page));  // pos < 2^31
  const int pg = __ldg(p.table + static_cast<long long>(lo) * p.max_pages + slot);
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) return -2;
  return static_cast<long long>(pg) * p.Hkv * p.page + (pos - static_cast<long long>(slot) * p.page);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats to two e4m3 codes (low byte: the first), nearest even, +-448 past the range.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes to f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// 2^(s - 127) for scale codes 1 .. 254.
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// Largest finite |x| of eight bf16 as its bits (they order as the values do).
__device__ __forceinline__ uint32_t finite_max(const uint4& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = (&x.x)[i] & 0x7fff7fffu;
    const uint32_t a = w & 0xffffu, b = w >> 16;
    m = max(m, a < 0x7f80u ? a : 0u);
    m = max(m, b < 0x7f80u ? b : 0u);
  }
  return m;
}

// Elementwise maximum of two bf16 pairs; a NaN yields to the other operand.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Largest |x| of eight bf16 that is no NaN, as its bits; 0 if all are.
__device__ __forceinline__ uint32_t number_max(const uint4& x) {
  uint32_t m = max_bf16x2(max_bf16x2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), max_bf16x2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  m = max_bf16x2(m, 0u);
  return max(m & 0xffffu, m >> 16);
}

// Scale code of a row whose largest finite |x| has these bf16 bits: with a = (1 + mm / 128) *
// 2^(ef - 127) and 448 = 1.75 * 2^8, e is ef - 135 while 1 + mm / 128 <= 1.75, else one more.
__device__ __forceinline__ uint32_t scale_code(uint32_t bits) {
  const int ef = static_cast<int>(bits >> 7), mm = static_cast<int>(bits & 127u);
  const int s = ef - 8 + (mm > 96 ? 1 : 0);
  return static_cast<uint32_t>(max(s, 1));  // zero and subnormal rows: 2^-126
}

constexpr uint32_t kTopScale = 247;  // e = 120

// Magnitudes of two bf16 to at most 240 * 2^120 (bits 0x7f70), infinities too, NaN as it is.
__device__ __forceinline__ uint32_t under_top(uint32_t w) {
  const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
  if (a > 0x7f70u && a <= 0x7f80u) w = (w & 0xffff8000u) | 0x7f70u;
  if (b > 0x7f70u && b <= 0x7f80u) w = (w & 0x8000ffffu) | 0x7f700000u;
  return w;
}

__device__ __forceinline__ uint2 quantise8(uint4 x, uint32_t s) {
  if (s == kTopScale) x = make_uint4(under_top(x.x), under_top(x.y), under_top(x.z), under_top(x.w));
  const float2 inv = make_float2(scale_of(254u - s), scale_of(254u - s));
  auto two = [&](uint32_t w) {
    const float2 v = __fmul2_rn(make_float2(bf16_lo(w), bf16_hi(w)), inv);
    return pack_e4m3x2(v.x, v.y);
  };
  return make_uint2(two(x.x) | (two(x.y) << 16), two(x.z) | (two(x.w) << 16));
}

__device__ __forceinline__ uint4 dequantise8(const uint2& c, float scale) {
  uint4 r;
  const float2 a = e4m3x2_to_f32(c.x & 0xffffu), b = e4m3x2_to_f32(c.x >> 16);
  const float2 d = e4m3x2_to_f32(c.y & 0xffffu), e = e4m3x2_to_f32(c.y >> 16);
  r.x = pack_bf16x2(a.x * scale, a.y * scale);
  r.y = pack_bf16x2(b.x * scale, b.y * scale);
  r.z = pack_bf16x2(d.x * scale, d.y * scale);
  r.w = pack_bf16x2(e.x * scale, e.y * scale);
  return r;
}

// 16 bytes that are read once: past L1, which keeps cu_seqlens and the block table.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// A block owns (token, head) rows [blockIdx * kPerBlock, ...) in packed order.
template <int D>
struct CacheTile {
  static constexpr int kLanes = D / 8;                                    // lanes of a row
  static constexpr int kGroups = kCacheThreads / kLanes;                  // rows a block does at once
  static constexpr int kPerBlock = kGroups * kCacheUnroll;
};

// Token of a (token, head) row; the 64-bit division only where it is needed.
__device__ __forceinline__ int cache_token(long long item, int heads) {
  if ((item >> 32) == 0) return static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(heads));
  return static_cast<int>(item / heads);
}

// Cache rows of the tokens of the kPerBlock rows from item0 on, into shared memory.
template <int D>
__device__ __forceinline__ void cache_rows(const CacheParams& p, long long item0, long long items, long long* rows) {
  const int tok0 = cache_token(item0, p.Hkv);
  const long long last = min(item0 + CacheTile<D>::kPerBlock, items) - 1;
  const int ntok = cache_token(last, p.Hkv) - tok0 + 1;
  for (int i = threadIdx.x; i < ntok; i += kCacheThreads) {
    const long long r = cache_row_of(p, tok0 + i);
    if (r == -2 && p.page_word) atomicOr(p.page_word, 1u);
    rows[i] = r;
  }
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kCacheThreads, 4) attn_cache_write_kernel(const CacheParams p) {
  using C = CacheTile<D>;
  __shared__ long long rows[C::kPerBlock];
  griddep_wait();
  griddep_launch_dependents();
  const long long items = static_cast<long long>(p.total) * p.Hkv;
  const long long item0 = static_cast<long long>(blockIdx.x) * C::kPerBlock;
  const int group = threadIdx.x / C::kLanes, lane = threadIdx.x % C::kLanes;
  const int tok0 = cache_token(item0, p.Hkv);
  uint4 xk[kCacheUnroll], xv[kCacheUnroll];
  int tok[kCacheUnroll], head[kCacheUnroll];
  int t = cache_token(min(item0 + group, items - 1), p.Hkv);
  int h = static_cast<int>(min(item0 + group, items - 1) - static_cast<long long>(t) * p.Hkv);
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    tok[u] = item0 + u * C::kGroups + group < items ? t : -1;
    head[u] = h;
    xk[u] = xv[u] = make_uint4(0, 0, 0, 0);
    if (tok[u] >= 0) {
      xk[u] = ld_stream(reinterpret_cast<const uint4*>(p.src_k + t * p.k_st + h * p.k_sh) + lane);
      xv[u] = ld_stream(reinterpret_cast<const uint4*>(p.src_v + t * p.v_st + h * p.v_sh) + lane);
    }
    // kGroups rows further: p.step_t tokens and p.step_h heads
    t += p.step_t;
    h += p.step_h;
    if (h >= p.Hkv) {
      h -= p.Hkv;
      ++t;
    }
  }
  cache_rows<D>(p, item0, items, rows);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    const long long r0 = tok[u] >= 0 ? rows[tok[u] - tok0] : -1;
    const long long r = r0 + static_cast<long long>(head[u]) * p.page;
    if constexpr (kF8) {
      // both maxima in one word for the shuffles; an infinity (the maximum of finite values is
      // wanted) sends the row the long way
      uint32_t m = number_max(xk[u]) | (number_max(xv[u]) << 16);
#pragma unroll
      for (int o = C::kLanes / 2; o > 0; o >>= 1)  // every lane of the warp, rows written or not
        m = max_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
      uint32_t mk = m & 0xffffu, mv = m >> 16;
      if (__any_sync(0xffffffffu, mk >= 0x7f80u || mv >= 0x7f80u)) {
        mk = finite_max(xk[u]);
        mv = finite_max(xv[u]);
#pragma unroll 1
        for (int o = C::kLanes / 2; o > 0; o >>= 1) {
          mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
          mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        }
      }
      const uint32_t sk = scale_code(mk), sv = scale_code(mv);
      if (r0 >= 0) {
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k) + r * D)[lane] = quantise8(xk[u], sk);
        reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v) + r * D)[lane] = quantise8(xv[u], sv);
        if (lane == 0) {
          p.ks[r] = static_cast<uint8_t>(sk);
          p.vs[r] = static_cast<uint8_t>(sv);
        }
      }
    } else if (r0 >= 0) {
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k) + r * D)[lane] = xk[u];
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v) + r * D)[lane] = xv[u];
    }
  }
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kCacheThreads) attn_cache_read_kernel(const CacheParams p) {
  using C = CacheTile<D>;
  __shared__ long long rows[C::kPerBlock];
  griddep_wait();
  griddep_launch_dependents();
  const long long items = static_cast<long long>(p.total) * p.Hkv;
  const long long item0 = static_cast<long long>(blockIdx.x) * C::kPerBlock;
  const int group = threadIdx.x / C::kLanes, lane = threadIdx.x % C::kLanes;
  const int tok0 = cache_token(item0, p.Hkv);
  cache_rows<D>(p, item0, items, rows);
  __syncthreads();
  uint4 xk[kCacheUnroll], xv[kCacheUnroll];
  long long src[kCacheUnroll];
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    const long long it = item0 + u * C::kGroups + group;
    src[u] = -1;  // a row in no sequence: left as it was
    xk[u] = xv[u] = make_uint4(0, 0, 0, 0);
    if (it < items) {
      const int t = cache_token(it, p.Hkv);
      const long long r0 = rows[t - tok0];
      src[u] = r0;
      if (r0 >= 0) {
        const long long r = r0 + (it - static_cast<long long>(t) * p.Hkv) * p.page;
        if constexpr (kF8) {
          const uint2 ck = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.k) + r * D) + lane);
          const uint2 cv = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.v) + r * D) + lane);
          xk[u] = make_uint4(ck.x, ck.y, __ldg(p.ks + r), 0);
          xv[u] = make_uint4(cv.x, cv.y, __ldg(p.vs + r), 0);
        } else {
          xk[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.k) + r * D) + lane);
          xv[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.v) + r * D) + lane);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kCacheUnroll; ++u) {
    if (src[u] == -1) continue;  // -2 (no page): zeros
    const long long it = item0 + u * C::kGroups + group;
    if constexpr (kF8) {
      xk[u] = dequantise8(make_uint2(xk[u].x, xk[u].y), scale_of(xk[u].z));
      xv[u] = dequantise8(make_uint2(xv[u].x, xv[u].y), scale_of(xv[u].z));
    }
    reinterpret_cast<uint4*>(p.dst_k + it * D)[lane] = xk[u];
    reinterpret_cast<uint4*>(p.dst_v + it * D)[lane] = xv[u];
  }
}

}  // namespace attn

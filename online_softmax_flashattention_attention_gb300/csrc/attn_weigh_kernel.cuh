// Attention weight that cached keys receive from a call's queries, sm_103a.
//
// Sequence b has ctx_b cached tokens and T_b new ones at positions ctx_b .. ctx_b + T_b - 1, whose
// queries have been through the attention already: LSE is theirs.  Row (t, g) of K/V head h, query
// head h G + g of token t, sees position p <= ctx_b + t, and
//   out[p] = decay * weights[p] + sum over the rows that see p of exp(scale q . k_p - LSE),
// where positions from ctx_b on start from 0.  A row that saw nothing (LSE = -infinity) adds nothing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_cache_kernel.cuh"
#include "ptx.cuh"

namespace attn {

constexpr int kWeighKeys = 128;     // of a unit
constexpr int kWeighGroups = 64;    // prefix-sum entries (each over ceil(B / 64) sequences)
constexpr int kWeighThreads = 128;

struct WeighParams {
  const __nv_bfloat16* q;    // [total_q, Hq, d]
  const float* lse;          // [Hq, total_q]
  const void* k;             // the cache's keys
  const uint8_t* ks;         // their scale codes, e4m3 only
  const float* w;            // [num_pages, Hkv, page]; not read when decay == 0
  float* out;                // the same
  const int32_t* table;      // [B, max_pages]
  const int32_t* cu;         // [B + 1]
  const int32_t* ctx;        // [B] or null
  int B, Hq, Hkv, G, total_q;
  int num_pages, page, max_pages, cap;
  float c;                   // scale * log2(e)
  float decay;
  uint32_t* page_word;
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

template <int D, bool kF8>
__global__ void __launch_bounds__(kWeighThreads) attn_weigh_kernel(const WeighParams p) {
  __shared__ long long pre[kWeighGroups + 1];
  __shared__ float qs[16][D];
  __shared__ float nl[16];
  griddep_wait();
  griddep_launch_dependents();
  const int gs = (p.B + kWeighGroups - 1) / kWeighGroups;
  if (threadIdx.x < kWeighGroups) {
    long long sum = 0;
    for (long long b = static_cast<long long>(threadIdx.x) * gs; b < min(static_cast<long long>(threadIdx.x + 1) * gs, static_cast<long long>(p.B)); ++b) {
      const WeighSeq s = weigh_seq(p, static_cast<int>(b));
      sum += static_cast<long long>(s.tiles) * p.Hkv;
      if (blockIdx.x == 0 && s.T > 0 && p.page_word && static_cast<long long>(s.ctx) + s.T > p.cap) atomicOr(p.page_word, 1u);
    }
    pre[threadIdx.x + 1] = sum;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    pre[0] = 0;
    for (int i = 0; i < kWeighGroups; ++i) pre[i + 1] += pre[i];
  }
  __syncthreads();
  for (long long u = blockIdx.x; u < pre[kWeighGroups]; u += gridDim.x) {
    int grp = 0;
    while (pre[grp + 1] <= u) ++grp;
    long long y = u - pre[grp];
    int b = grp * gs;
    WeighSeq s = weigh_seq(p, b);
    while (y >= static_cast<long long>(s.tiles) * p.Hkv) {
      y -= static_cast<long long>(s.tiles) * p.Hkv;
      s = weigh_seq(p, ++b);
    }
    const int tile = static_cast<int>(y / p.Hkv), h = static_cast<int>(y - static_cast<long long>(tile) * p.Hkv);
    const int pos = tile * kWeighKeys + threadIdx.x;
    int pg = -1;
    if (pos < s.n) {
      pg = __ldg(p.table + static_cast<long long>(b) * p.max_pages + static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page));
      if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) {
        pg = -1;
        if (p.page_word) atomicOr(p.page_word, 1u);
      }
    }
    const long long row = (static_cast<long long>(pg) * p.Hkv + h) * p.page + pos % p.page;
    float key[D];
    if (pg >= 0) {
      const float sc = kF8 ? scale_of(p.ks[row]) : 1.f;
#pragma unroll
      for (int i = 0; i < D / 2; ++i) {
        if constexpr (kF8) {
          const float2 f = e4m3x2_to_f32(reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(p.k) + row * D)[i]);
          key[2 * i] = f.x * sc;
          key[2 * i + 1] = f.y * sc;
        } else {
          const uint32_t w = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.k) + row * D)[i];
          key[2 * i] = bf16_lo(w);
          key[2 * i + 1] = bf16_hi(w);
        }
      }
    }
    float sum = 0.f;
    const int rows = s.T * p.G;
    const int first = max(0, tile * kWeighKeys - s.ctx) * p.G;  // rows before it see no key of the tile
    for (int r0 = first; r0 < rows; r0 += 16) {
      __syncthreads();
      for (int i = threadIdx.x; i < 16 * D; i += kWeighThreads) {
        const int r = r0 + i / D;
        if (r < rows)
          qs[i / D][i % D] = __bfloat162float(p.q[(static_cast<long long>(s.q0 + r / p.G) * p.Hq + h * p.G + r % p.G) * D + i % D]);
      }
      if (threadIdx.x < 16 && r0 + threadIdx.x < rows) {
        const int r = r0 + threadIdx.x;
        nl[threadIdx.x] = p.lse[static_cast<long long>(h * p.G + r % p.G) * p.total_q + s.q0 + r / p.G] * 1.4426950408889634f;
      }
      __syncthreads();
      float part = 0.f;
      for (int j = 0; j < min(16, rows - r0); ++j) {
        if (pos > s.ctx + (r0 + j) / p.G || nl[j] == -INFINITY || pg < 0) continue;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < D; ++i) dot = fmaf(qs[j][i], key[i], dot);
        part += ex2_approx(fmaf(dot, p.c, -nl[j]));
      }
      sum += part;
    }
    if (pg >= 0) p.out[row] = (p.decay != 0.f && pos < s.ctx ? p.decay * p.w[row] : 0.f) + sum;
  }
}

}  // namespace attn

// Eviction from the paged cache by accumulated attention weight, sm_103a.
//
// Each (sequence, K/V head) with n > keep tokens keeps its first `sink` positions, its last
// `recent` ones and, of those between, the keep - sink - recent with the largest weights (equal
// ones: the first).  attn_evict_select_kernel writes the kept positions in increasing order;
// attn_evict_move_kernel packs their rows (K, V, scale codes, weights) to positions 0, 1, ... of
// the sequence's own pages, or of other ones.
//
// Choice.  A weight becomes an integer key of the same order (NaN as -infinity, -0 as 0).  A cluster
// of 1 to 8 CTAs shares a unit: each holds its stretch of the keys in shared memory, read once.  The
// threshold, the key of the last one kept, is found by cutting the interval that holds it into at
// most 2048 equal parts: one histogram, summed over the cluster through distributed shared memory,
// says in which part it lies.  The first interval is [least key, largest key], so three rounds at
// most (32 bits, 11 a round) and mostly two.  Then every warp counts what its stretch keeps, and
// knows from the counts before it where its positions go: no order is left to atomics.
//
// Packing in place: place i receives the row of position kept[i] >= i.  A block walks the places in
// order, some at a time, and reads all rows of a step before it writes any; what it writes lies
// before everything it has yet to read.  Blocks share a head by columns, which do not depend on each
// other.  Into other pages there is no order to keep, and blocks share a head by rows.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_cache_kernel.cuh"
#include "ptx.cuh"

namespace attn {

// Bound: 48 e4m3 sequences of 900 to 16384 tokens, 8 heads, d = 128, to 4096 each: 152 us, of which the
// choice is 38 (its rounds wait for shared memory and each other) and the rows' way 113, 5.8 TB/s and so
// DRAM; K's and V's rows by blocks of their own 173, addresses looked up by every lane 213.  One sequence
// of 1733 to 1024 is two launches and a chain of loads and cluster barriers, 14 us.  One long sequence waits
// for latencies: bf16, 100000 tokens to 65536, 8 heads, 435 us of which 366 are one block's way through a
// head's weights, 256 rows at a time; in place, where the rows' blocks go like that too, 625.
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictBinBits = 11;
constexpr int kEvictMaxKeys = 49152;  // keys a CTA holds in shared memory; further ones are read again
constexpr int kEvictLoads = 8;        // weights a thread has in flight
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

struct EvictParams {
  uint8_t* k;                // the pool, rows of row_bytes
  uint8_t* v;
  uint8_t* ks;               // scale codes or null
  uint8_t* vs;
  float* w;                  // [num_pages, Hkv, page]
  const int32_t* table;      // [B, max_pages]
  const int32_t* to;         // [B, to_pages]: where the kept rows go
  const int32_t* lens;       // [B]
  int32_t* kept;             // [B, Hkv, keep]
  int32_t* out_lens;         // [B]
  int B, Hkv, num_pages, page, max_pages, to_pages;
  int keep, sink, recent;
  int row_bytes;
  int key_cap;               // keys in shared memory
  int in_place;              // to == table
  int slice;                 // bytes of a row a block moves
  int rows_per_block;        // places a block moves (all of them in place)
  uint32_t* page_word;
};

__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  return static_cast<int>(min(static_cast<long long>(max(__ldg(p.lens + b), 0)), static_cast<long long>(p.max_pages) * p.page));
}

// Row of head h at a position (or place) through a block table, in rows of the pool; -1 without a page.
__device__ __forceinline__ long long evict_row(const EvictParams& p, const int32_t* table, int pages, int b, int h, int pos) {
  const int slot = static_cast<uint32_t>(pos) / static_cast<uint32_t>(p.page);
  if (slot >= pages) return -1;
  const int pg = __ldg(table + static_cast<long long>(b) * pages + slot);
  if (static_cast<unsigned>(pg) >= static_cast<unsigned>(p.num_pages)) return -1;
  return (static_cast<long long>(pg) * p.Hkv + h) * p.page + (pos - slot * p.page);
}

// A key that orders as the weight does; NaN as -infinity.
__device__ __forceinline__ uint32_t evict_key(float w) {
  if (!(w == w)) w = -INFINITY;
  w += 0.f;  // -0 as 0
  const uint32_t u = __float_as_uint(w);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) attn_evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[2][kEvictBins];
  __shared__ uint32_t warp_sum[kEvictWarps];
  __shared__ uint32_t range[2];        // least and largest key of this CTA
  __shared__ uint32_t found[3];        // part, keys above it, keys in it
  __shared__ uint32_t counts[2][kEvictWarps];
  __shared__ uint32_t cta_counts[2];   // keys above the threshold, equal to it
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / C, b = unit / p.Hkv, h = unit - b * p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int n = evict_len(p, b);
  int32_t* kept = p.kept + static_cast<long long>(unit) * p.keep;
  if (h == 0 && rank == 0 && tid == 0) p.out_lens[b] = min(n, p.keep);
  if (n <= p.keep) {  // the whole cluster: nothing to choose
    for (int i = rank * kEvictThreads + tid; i < p.keep; i += C * kEvictThreads) kept[i] = i < n ? i : -1;
    return;
  }
  for (int i = rank * kEvictThreads + tid; i < p.sink + p.recent; i += C * kEvictThreads) {
    const int place = i < p.sink ? i : p.keep - p.recent + (i - p.sink);
    kept[place] = i < p.sink ? i : n - p.recent + (i - p.sink);
  }
  uint32_t need = p.keep - p.sink - p.recent;
  if (need == 0) return;

  // ---- this CTA's stretch of the candidates: [c0, c1) of the positions from sink on
  const int m = n - p.recent - p.sink;
  const int seg = (m + C - 1) / C;
  const int c0 = min(rank * seg, m), c1 = min(c0 + seg, m);
  auto read = [&](int c) {
    const long long r = evict_row(p, p.table, p.max_pages, b, h, p.sink + c);
    return evict_key(r < 0 ? -INFINITY : p.w[r]);
  };
  auto key_at = [&](int c) { return c - c0 < p.key_cap ? keys[c - c0] : read(c); };
  if (tid == 0) {
    range[0] = 0xffffffffu;
    range[1] = 0u;
  }
  for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[0][i] = hist[1][i] = 0;
  __syncthreads();
  uint32_t lo = 0xffffffffu, hi = 0u;
  // several at a time: a page is one load away, its weight another, some 2000 cycles together
  for (int b0 = c0 + tid; b0 < c1; b0 += kEvictThreads * kEvictLoads) {
    long long at[kEvictLoads];
    uint32_t key[kEvictLoads];
#pragma unroll
    for (int i = 0; i < kEvictLoads; ++i) {
      const int c = b0 + i * kEvictThreads;
      at[i] = c < c1 ? evict_row(p, p.table, p.max_pages, b, h, p.sink + c) : -1;
    }
#pragma unroll
    for (int i = 0; i < kEvictLoads; ++i) key[i] = evict_key(at[i] < 0 ? -INFINITY : p.w[at[i]]);
#pragma unroll
    for (int i = 0; i < kEvictLoads; ++i) {
      const int c = b0 + i * kEvictThreads;
      if (c >= c1) break;
      if (at[i] < 0 && p.page_word) atomicOr(p.page_word, 1u);
      if (c - c0 < p.key_cap) keys[c - c0] = key[i];
      lo = min(lo, key[i]);
      hi = max(hi, key[i]);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    atomicMin(&range[0], lo);
    atomicMax(&range[1], hi);
  }
  cluster.sync();
  lo = 0xffffffffu;
  hi = 0u;
  for (int q = 0; q < C; ++q) {
    const uint32_t* other = cluster.map_shared_rank(range, q);
    lo = min(lo, other[0]);
    hi = max(hi, other[1]);
  }

  // ---- the threshold: the interval [lo, lo + 2^bits) holds it
  uint32_t span = hi - lo, above, shift;
  for (int round = 0;; ++round) {
    shift = 32 - __clz(span) > kEvictBinBits ? 32 - __clz(span) - kEvictBinBits : 0;
    uint32_t* mine = hist[round & 1];
    for (int c = c0 + tid; c < c1; c += kEvictThreads) {
      const uint32_t off = key_at(c) - lo;  // keys below lo wrap past the span
      if (off <= span) atomicAdd(&mine[off >> shift], 1u);
    }
    cluster.sync();  // also: everybody is done with the other histogram
    // sums over the cluster, each thread four neighbouring parts from the top down
    constexpr int kPer = kEvictBins / kEvictThreads;
    uint32_t part[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) part[i] = 0;
    const int first = kEvictBins - (tid + 1) * kPer;
    for (int q = 0; q < C; ++q) {
      const uint32_t* other = cluster.map_shared_rank(mine, q);
#pragma unroll
      for (int i = 0; i < kPer; ++i) part[i] += other[first + i];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += part[i];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[(round + 1) & 1][i] = 0;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int q = 0; q < warp; ++q) before += warp_sum[q];
    if (before < need && before + sum >= need) {  // one thread: the part is among its four
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i) {
        if (before < need && before + part[i] >= need) {
          found[0] = first + i;
          found[1] = before;
          found[2] = part[i];
          before = need;  // none of the others
        } else {
          before += part[i];
        }
      }
    }
    __syncthreads();
    lo += found[0] << shift;
    need -= found[1];
    above = found[2];
    if (above == need || shift == 0) break;
    span = (1u << shift) - 1u;
  }
  // kept: keys above `limit`, and the first `equal` of those equal to it
  const bool whole = above == need;
  const uint32_t limit = whole ? lo - 1 : lo;  // no key is 0
  const uint32_t equal = whole ? 0 : need;

  // ---- where every warp's kept positions go
  const int sub = ((c1 - c0 + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int w0 = min(c0 + warp * sub, c1), w1 = min(w0 + sub, c1);
  uint32_t gt = 0, eq = 0;
  for (int c = w0 + lane; c < w1; c += 32) {
    const uint32_t key = key_at(c);
    gt += key > limit;
    eq += key == limit;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    counts[0][warp] = gt;
    counts[1][warp] = eq;
  }
  __syncthreads();
  if (tid < 2) {
    uint32_t s = 0;
    for (int q = 0; q < kEvictWarps; ++q) s += counts[tid][q];
    cta_counts[tid] = s;
  }
  cluster.sync();
  gt = eq = 0;
  for (int q = 0; q < rank; ++q) {
    const uint32_t* other = cluster.map_shared_rank(cta_counts, q);
    gt += other[0];
    eq += other[1];
  }
  for (int q = 0; q < warp; ++q) {
    gt += counts[0][q];
    eq += counts[1][q];
  }
  for (int c = w0 + lane; c - lane < w1; c += 32) {
    const uint32_t key = c < w1 ? key_at(c) : 0u;  // 0: neither above nor equal
    const uint32_t g = __ballot_sync(0xffffffffu, key > limit && c < w1);
    const uint32_t e = __ballot_sync(0xffffffffu, key == limit && c < w1);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t eb = eq + __popc(e & below);
    if (((g >> lane) & 1u) || (((e >> lane) & 1u) && eb < equal))
      kept[p.sink + gt + __popc(g & below) + min(eb, equal)] = p.sink + c;
    gt += __popc(g);
    eq += __popc(e);
  }
  cluster.sync();  // nobody leaves while its counts may be read
}

// blocks + 1 blocks a unit: `blocks` for K's and V's rows, one for scale codes and weights.
__global__ void __launch_bounds__(kMoveThreads) attn_evict_move_kernel(const EvictParams p, int blocks) {
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x / (blocks + 1), block = blockIdx.x - unit * (blocks + 1);
  const int b = unit / p.Hkv, h = unit - b * p.Hkv;
  const int n = evict_len(p, b), rows = min(n, p.keep);
  const int32_t* kept = p.kept + static_cast<long long>(unit) * p.keep;
  const bool here = p.in_place && n <= p.keep;  // every row is where it belongs
  if (here) return;
  if (block == blocks) {
    // scale codes and weights: a thread a row
    for (int i0 = 0; i0 < rows; i0 += kMoveThreads) {
      const int i = i0 + threadIdx.x;
      const int pos = i < rows ? kept[i] : 0;
      const long long from = i < rows ? evict_row(p, p.table, p.max_pages, b, h, pos) : -1;
      const long long to = i < rows ? evict_row(p, p.to, p.to_pages, b, h, i) : -1;
      if (i < rows && (from < 0 || to < 0) && p.page_word) atomicOr(p.page_word, 1u);
      const float w = from >= 0 ? p.w[from] : 0.f;
      const uint8_t a = p.ks && from >= 0 ? p.ks[from] : 1, c = p.vs && from >= 0 ? p.vs[from] : 1;
      __syncthreads();
      if (to >= 0) {
        p.w[to] = w;
        if (p.ks) {
          p.ks[to] = a;
          p.vs[to] = c;
        }
      }
    }
    return;
  }
  const int slices = p.row_bytes / p.slice;
  const int lanes = p.slice / 16, col = (block % slices) * p.slice + (threadIdx.x % lanes) * 16;  // lanes: a power of two
  const int r0 = block / slices * p.rows_per_block, r1 = min(rows, r0 + p.rows_per_block);
  const int step = kMoveThreads / lanes;  // rows a block moves at once
  // The way of 256 rows, a thread each (two divisions and two loads), then the rows.
  __shared__ long long from[kMoveThreads], to[kMoveThreads];
  for (int i0 = r0; i0 < r1; i0 += kMoveThreads) {
    const int i = i0 + threadIdx.x;
    long long f = -1, t = -1;
    if (i < r1) {
      const int pos = kept[i];
      if (!p.in_place || pos != i) {
        f = evict_row(p, p.table, p.max_pages, b, h, pos);
        t = evict_row(p, p.to, p.to_pages, b, h, i);
      }
    }
    from[threadIdx.x] = f;
    to[threadIdx.x] = t;
    __syncthreads();
    for (int k0 = threadIdx.x / lanes; k0 < kMoveThreads; k0 += step * kMoveUnroll) {
      uint4 x[2][kMoveUnroll];
      long long dst[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const int k = k0 + u * step;
        const long long src = k < kMoveThreads ? from[k] : -1;
        dst[u] = k < kMoveThreads ? to[k] : -1;
        x[0][u] = x[1][u] = make_uint4(0, 0, 0, 0);
        if (dst[u] >= 0 && src >= 0) {
          x[0][u] = *reinterpret_cast<const uint4*>(p.k + src * p.row_bytes + col);
          x[1][u] = *reinterpret_cast<const uint4*>(p.v + src * p.row_bytes + col);
        }
      }
      if (p.in_place) __syncthreads();  // a step's rows are read before any is written
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u)
        if (dst[u] >= 0) {
          *reinterpret_cast<uint4*>(p.k + dst[u] * p.row_bytes + col) = x[0][u];
          *reinterpret_cast<uint4*>(p.v + dst[u] * p.row_bytes + col) = x[1][u];
        }
    }
    __syncthreads();
  }
}

}  // namespace attn

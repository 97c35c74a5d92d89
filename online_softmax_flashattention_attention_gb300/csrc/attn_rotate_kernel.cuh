// Norms of query and key heads and their rotation by position in one pass, sm_103a.
//
// A row x is one head of one token, d = 64 or 128 values.  With a weight w it becomes
// y_i = x_i w_i / sqrt(mean(x^2) + eps); without one y = x.  Then column i < r of the first 2 r
// columns (r = num_freq) turns with its partner, i + r or (interleaved) 2 i with 2 i + 1, by
// t = position * inv_freq[i]: (a, b) -> (a cos t - b sin t, b cos t + a sin t).  All of it in fp32,
// rounded to bf16 once.
//
// The angle.  Only its fraction of a turn counts, so it is kept as a fixed-point number: with
// F = frac(|inv_freq| / 2 pi) * 2^64 (one product in 64-bit floats; negated where inv_freq is negative),
// position * F modulo 2^64 is that fraction without another rounding, at any position: the error is
// position * inv_freq * 2^-52 rad at most, as a product of 64-bit floats has, and 2^-23 rad for what
// follows in fp32 (of a half turn, 24 bits).
//
// A row is d / 8 lanes, each with two pieces of four columns: half-split, a piece of the first half and
// the one it turns with; so no value changes lanes, and a norm's sum is all that crosses them.  Rows
// share their factors: with A_i = w_i cos t and B_i = +-w_partner sin t a row costs two products a
// value and one for its norm.  A block owns kRotTokens tokens at a time: its threads look up the
// positions and compute each of the tokens' angles once, in shared memory, while the first rows are on
// their way; then each group of lanes keeps A and B of one token in registers and walks the token's
// heads, Q's, then K's.  Blocks are persistent, so that the frequencies (64-bit floats, slow here) and
// weights are made once a block.
//
// Bound: DRAM.  58327 tokens of 9 prompts, 32 / 8 heads, d = 128: 220 us, 5.4 TB/s, 0.80 of a plain
// copy's rate; with partners a lane's exchange away 340, without the next rows ahead 230.  One token,
// 3.4 us, is a launch and three loads that wait for each other.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_cache_kernel.cuh"
#include "ptx.cuh"

namespace attn {

constexpr int kRotThreads = 256;
constexpr int kRotTokens = 4;   // of a block
constexpr int kRotUnroll = 4;   // rows a group of lanes has in flight

struct RotateParams {
  const __nv_bfloat16* src[2];   // Q, K: element (t, h, x) at t * st + h * sh + x
  __nv_bfloat16* dst[2];
  long long src_t[2], src_h[2], dst_t[2], dst_h[2];
  const void* weight[2];         // [d] or null
  const int32_t* cu;             // [B + 1] or null: all rows are one sequence
  const int32_t* start;          // [B] or null (0)
  const int32_t* positions;      // [total] or null (start + place in the sequence)
  const float* freq;             // [num_freq]
  int num_freq, weight_f32;
  float eps;
  int B, Hq, H, total;           // H: heads of Q and K together
  int heads_per_block;
};

// Whether row `tok` belongs to a sequence, and its position.
__device__ __forceinline__ bool rotate_position(const RotateParams& p, int tok, long long* pos) {
  int lo = 0, first = 0;
  if (p.cu) {
    int hi = p.B;  // the sequence is in [lo, hi): the last one that starts at or before the row
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (__ldg(p.cu + mid) <= tok)
        lo = mid;
      else
        hi = mid;
    }
    first = max(__ldg(p.cu + lo), 0);
    if (tok < first || tok >= __ldg(p.cu + lo + 1)) return false;
  }
  *pos = p.positions ? __ldg(p.positions + tok)
                     : static_cast<long long>(p.start ? max(__ldg(p.start + lo), 0) : 0) + (tok - first);
  return true;
}

// Column i's turn a position, as a fraction of 2^64.  A negative one is the other's modulo 2^64: the
// fraction of a small negative number itself, 1 less that number, would have 53 bits of 1.
__device__ __forceinline__ unsigned long long rotate_step(float freq) {
  const double turns = static_cast<double>(fabsf(freq)) * 0.15915494309189533577;  // 1 / 2 pi
  const unsigned long long step = __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
  return freq < 0.f ? 0ull - step : step;
}

struct RotRow {
  uint2 a, b;  // the lane's two pieces of four columns
};

// kPairs: interleaved.  kAll: every column turns.
template <int D, bool kPairs, bool kAll>
__global__ void __launch_bounds__(kRotThreads, 3) attn_qk_rotate_kernel(const RotateParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kRotThreads / kLanes;
  constexpr int kPerTok = kGroups / kRotTokens;  // groups that share a token
  constexpr int kU = kRotUnroll;
  __shared__ float2 turn[kRotTokens][D / 2];     // cos, sin
  __shared__ unsigned long long step[D / 2];
  __shared__ float weight[2][D];
  __shared__ long long at[kRotTokens];
  __shared__ int in[kRotTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int tk = group / kPerTok, sub = group % kPerTok;
  const int r = p.num_freq;
  // the lane's pieces: columns ca .. + 3 and cb .. + 3; which frequency the first of ca has, if it turns
  int ca = 8 * lane, cb = 8 * lane + 4, fa = 4 * lane;
  bool turned = kAll || 8 * lane < 2 * r;
  if (!kPairs) {
    turned = kAll || 4 * lane < r;
    ca = turned ? 4 * lane : 2 * r + 8 * (lane - r / 4);
    cb = turned ? ca + r : ca + 4;
    fa = ca;
  }
  const int head0 = blockIdx.y * p.heads_per_block, head1 = min(p.H, head0 + p.heads_per_block);
  for (int i = threadIdx.x; i < 2 * D; i += kRotThreads) {
    const void* w = p.weight[i / D];
    weight[i / D][i % D] = !w ? 1.f : p.weight_f32 ? static_cast<const float*>(w)[i % D]
                                                   : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i % D]);
  }
  if (threadIdx.x < r) step[threadIdx.x] = rotate_step(__ldg(p.freq + threadIdx.x));
  // (unsigned: the last step may pass 2^31)
  for (unsigned t0 = blockIdx.x * kRotTokens; t0 < static_cast<unsigned>(p.total); t0 += gridDim.x * kRotTokens) {
    const unsigned tok = t0 + tk;
    __syncthreads();  // the last tokens' angles have been used
    if (threadIdx.x < kRotTokens) {
      const unsigned t = t0 + threadIdx.x;
      long long pos = 0;
      in[threadIdx.x] = t < static_cast<unsigned>(p.total) && rotate_position(p, static_cast<int>(t), &pos);
      at[threadIdx.x] = pos;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRotTokens * r; i += kRotThreads) {
      const int t = i / r, f = i - t * r;
      const unsigned long long frac = static_cast<unsigned long long>(at[t]) * step[f];
      // half turns in [-1, 1)
      const float half = static_cast<float>(static_cast<int>(frac >> 32)) * 4.656612873077393e-10f;  // 2^-31
      float s, c;
      sincospif(half, &s, &c);
      if (!(fabsf(__ldg(p.freq + f)) < INFINITY)) s = c = NAN;
      turn[t][f] = make_float2(c, s);
    }
    __syncthreads();
    if (tok >= static_cast<unsigned>(p.total) || !in[tk]) continue;  // whole warps: a token's groups are
    static_assert(kPerTok * kLanes % 32 == 0, "a warp has one token");

#pragma unroll
    for (int k = 0; k < 2; ++k) {  // Q's heads, then K's
      const int h0 = max(head0 - (k ? p.Hq : 0), 0), h1 = min(head1 - (k ? p.Hq : 0), k ? p.H - p.Hq : p.Hq);
      if (h0 >= h1) continue;
      const __nv_bfloat16* src = p.src[k] + tok * p.src_t[k] + (h0 + sub) * p.src_h[k];
      __nv_bfloat16* dst = p.dst[k] + tok * p.dst_t[k] + (h0 + sub) * p.dst_h[k];
      const long long sstep = kPerTok * p.src_h[k], dstep = kPerTok * p.dst_h[k];
      RotRow x[kU];
      auto load = [&](int h) {
#pragma unroll
        for (int u = 0; u < kU; ++u, src += sstep)
          if (h + u * kPerTok < h1) {
            x[u].a = *reinterpret_cast<const uint2*>(src + ca);
            x[u].b = *reinterpret_cast<const uint2*>(src + cb);
          }
      };
      load(h0 + sub);
      // out_a = A va + Ba other, out_b = B vb + Bb other (other: the column it turns with)
      float wa[4], wb[4], Ac[4], Bc[4], As[4], Bs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wa[i] = weight[k][ca + i];
        wb[i] = weight[k][cb + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Ac[i] = wa[i];
        Bc[i] = wb[i];
        As[i] = Bs[i] = 0.f;
        if (turned) {
          const float2 x = turn[tk][kPairs ? fa + i / 2 : fa + i], y = kPairs ? turn[tk][fa + 2 + i / 2] : x;
          Ac[i] *= x.x;
          Bc[i] *= y.x;
          As[i] = kPairs ? ((i & 1) ? x.y : -x.y) * wa[i ^ 1] : -x.y * wb[i];
          Bs[i] = kPairs ? ((i & 1) ? y.y : -y.y) * wb[i ^ 1] : x.y * wa[i];
        }
      }
      const bool norm = p.weight[k] != nullptr;
#pragma unroll 1
      for (int hb = h0; hb < h1; hb += kU * kPerTok) {  // (the same rounds for every lane of a warp)
        const int h = hb + sub;
        RotRow row[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) row[u] = x[u];
        load(h + kU * kPerTok);  // the next rows, while these are in hand
#pragma unroll
        for (int u = 0; u < kU; ++u, dst += dstep) {
          float2 va[2] = {make_float2(bf16_lo(row[u].a.x), bf16_hi(row[u].a.x)), make_float2(bf16_lo(row[u].a.y), bf16_hi(row[u].a.y))};
          float2 vb[2] = {make_float2(bf16_lo(row[u].b.x), bf16_hi(row[u].b.x)), make_float2(bf16_lo(row[u].b.y), bf16_hi(row[u].b.y))};
          float inv = 1.f;
          if (norm) {
            float2 ss = __fmul2_rn(va[0], va[0]);
            ss = __ffma2_rn(va[1], va[1], ss);
            ss = __ffma2_rn(vb[0], vb[0], ss);
            ss = __ffma2_rn(vb[1], vb[1], ss);
            float sum = ss.x + ss.y;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            inv = rsqrtf(sum * (1.f / D) + p.eps);
          }
          float2 oa[2], ob[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            oa[i] = __fmul2_rn(va[i], make_float2(Ac[2 * i], Ac[2 * i + 1]));
            ob[i] = __fmul2_rn(vb[i], make_float2(Bc[2 * i], Bc[2 * i + 1]));
            if (kAll || turned) {
              const float2 other_a = kPairs ? make_float2(va[i].y, va[i].x) : vb[i];
              const float2 other_b = kPairs ? make_float2(vb[i].y, vb[i].x) : va[i];
              oa[i] = __ffma2_rn(other_a, make_float2(As[2 * i], As[2 * i + 1]), oa[i]);
              ob[i] = __ffma2_rn(other_b, make_float2(Bs[2 * i], Bs[2 * i + 1]), ob[i]);
            }
            oa[i] = __fmul2_rn(oa[i], make_float2(inv, inv));
            ob[i] = __fmul2_rn(ob[i], make_float2(inv, inv));
          }
          if (h + u * kPerTok < h1) {
            *reinterpret_cast<uint2*>(dst + ca) = make_uint2(pack_bf16x2(oa[0].x, oa[0].y), pack_bf16x2(oa[1].x, oa[1].y));
            *reinterpret_cast<uint2*>(dst + cb) = make_uint2(pack_bf16x2(ob[0].x, ob[0].y), pack_bf16x2(ob[1].x, ob[1].y));
          }
        }
      }
    }
  }
}

}  // namespace attn

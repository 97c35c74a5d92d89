// Norms of query and key heads and their rotation by position in one pass, sm_103a.
//
// A row x is one head of one token, d = 64 or 128 values.  With a weight w it becomes
// y_i = x_i w_i / sqrt(mean(x^2) + eps); without one y = x.  Then column i < r of the first 2 r
// columns (r = num_freq) turns with its partner, i + r or (interleaved) 2 i with 2 i + 1, by
// t = position * inv_freq[i]: (a, b) -> (a cos t - b sin t, b cos t + a sin t).  All of it in fp32,
// rounded to bf16 once.
//
// The angle.  Only its fraction of a turn counts, so it is kept as a fixed-point number: with
// F = frac(inv_freq / 2 pi) * 2^64 (one product in 64-bit floats), position * F modulo 2^64 is that
// fraction without another rounding, at any position: the error is position * inv_freq * 2^-52 rad
// at most, as a product of 64-bit floats has, and 2^-24 of it for what follows in fp32.
//
// A row is d / 8 lanes of 16 bytes: both halves of a half-split pair lie at the same place in two
// lanes, so a partner's eight values are four shuffles away.  Rows share their factors: with
// A_i = w_i cos t and B_i = +-w_partner sin t a row costs two products a value and one for its
// norm.  A block owns kRotTokens tokens: its threads look up the positions and compute each of the
// tokens' angles once, in shared memory, while the first rows are on their way; then each group of
// lanes keeps A and B of one token in registers and walks the token's heads.
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
  int num_freq, interleaved, weight_f32;
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

// Column i's turn a position, as a fraction of 2^64.
__device__ __forceinline__ unsigned long long rotate_step(float freq) {
  const double turns = static_cast<double>(freq) * 0.15915494309189533577;  // 1 / 2 pi
  return __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
}

// Eight weights from column c on, 1 without any.
__device__ __forceinline__ void rotate_weights(const void* w, int f32, int c, float* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = 1.f;
  if (!w) return;
  if (f32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = __ldg(static_cast<const float*>(w) + c + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c + i]);
  }
}

template <int D>
__global__ void __launch_bounds__(kRotThreads, 4) attn_qk_rotate_kernel(const RotateParams p) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kRotThreads / kLanes;
  constexpr int kPerTok = kGroups / kRotTokens;  // groups that share a token
  __shared__ float2 turn[kRotTokens][D / 2];     // cos, sin
  __shared__ long long at[kRotTokens];
  __shared__ int in[kRotTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  const int tk = group / kPerTok, tok = blockIdx.x * kRotTokens + tk;
  const int h0 = blockIdx.y * p.heads_per_block + group % kPerTok;
  const int h1 = min(p.H, static_cast<int>(blockIdx.y + 1) * p.heads_per_block);
  const bool row_here = tok < p.total;
  uint4 x[kRotUnroll];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const int hh = h + u * kPerTok, k = hh >= p.Hq;
      if (row_here && hh < h1)
        x[u] = *(reinterpret_cast<const uint4*>(p.src[k] + tok * p.src_t[k] + (hh - (k ? p.Hq : 0)) * p.src_h[k]) + lane);
    }
  };
  load(h0);
  if (threadIdx.x < kRotTokens) {
    const int t = blockIdx.x * kRotTokens + threadIdx.x;
    long long pos = 0;
    in[threadIdx.x] = t < p.total && rotate_position(p, t, &pos);
    at[threadIdx.x] = pos;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRotTokens * p.num_freq; i += kRotThreads) {
    const int t = i / p.num_freq, f = i - t * p.num_freq;
    const unsigned long long frac = static_cast<unsigned long long>(at[t]) * rotate_step(__ldg(p.freq + f));
    // half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int>(frac >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half, &s, &c);
    if (!(fabsf(__ldg(p.freq + f)) < INFINITY)) s = c = NAN;
    turn[t][f] = make_float2(c, s);
  }
  __syncthreads();
  if (!row_here || !in[tk]) return;  // a whole group of lanes: shuffles below are among a group's lanes

  const uint32_t mask = kLanes == 32 ? 0xffffffffu : ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const int r8 = p.num_freq / 8;  // lanes of a half
  const bool turned = lane < 2 * r8;
  const bool second = !p.interleaved && lane >= r8;
  const int partner = !turned || p.interleaved ? lane : second ? lane - r8 : lane + r8;
  float A[8], Bf[8];
  int have = -1;  // whose factors A and B are
  for (int h = h0; h < h1; h += kRotUnroll * kPerTok) {
    if (h != h0) load(h);
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const int hh = h + u * kPerTok, k = hh >= p.Hq;
      if (hh >= h1) break;
      if (k != have) {
        have = k;
        float wo[8], wp[8];
        rotate_weights(p.weight[k], p.weight_f32, 8 * lane, wo);
        rotate_weights(p.weight[k], p.weight_f32, 8 * partner, wp);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          A[i] = wo[i];
          Bf[i] = 0.f;
          if (turned) {
            const float2 cs = turn[tk][p.interleaved ? 4 * lane + i / 2 : 8 * lane + i - (second ? p.num_freq : 0)];
            const bool plus = p.interleaved ? (i & 1) : second;
            A[i] = wo[i] * cs.x;
            Bf[i] = (plus ? cs.y : -cs.y) * (p.interleaved ? wo[i ^ 1] : wp[i]);
          }
        }
      }
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      float v[8], o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
      float inv = 1.f;
      if (p.weight[k]) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
        for (int s = kLanes / 2; s > 0; s >>= 1) ss += __shfl_xor_sync(mask, ss, s);
        inv = rsqrtf(ss * (1.f / D) + p.eps);
      }
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = turned ? fmaf(v[i ^ 1], Bf[i], v[i] * A[i]) : v[i] * A[i];
      } else {
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __shfl_sync(mask, w[i], partner, kLanes);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = (i & 1) ? bf16_hi(q[i / 2]) : bf16_lo(q[i / 2]);
          o[i] = turned ? fmaf(other, Bf[i], v[i] * A[i]) : v[i] * A[i];
        }
      }
      uint4 r;
      r.x = pack_bf16x2(o[0] * inv, o[1] * inv);
      r.y = pack_bf16x2(o[2] * inv, o[3] * inv);
      r.z = pack_bf16x2(o[4] * inv, o[5] * inv);
      r.w = pack_bf16x2(o[6] * inv, o[7] * inv);
      *(reinterpret_cast<uint4*>(p.dst[k] + tok * p.dst_t[k] + (hh - (k ? p.Hq : 0)) * p.dst_h[k]) + lane) = r;
    }
  }
}

}  // namespace attn

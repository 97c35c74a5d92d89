// Join of the states that prompts with split keys leave (PromptPlan), sm_103a.
//
// A row's parts have states (m, l, o~) over disjoint keys; moved to the largest m they add up, as
// attn_merge_kernel.cuh has it, and O = o~ / l, LSE = (m + log2 l) ln 2 (m in log2 units here).  An infinity or NaN that a row sees stays
// what it is even where its part's weight underflows to zero, as it does without parts.
//
// A warp owns a row: lane t has columns [t d / 32, (t + 1) d / 32), so a part's row is one read of 256 or
// 512 bytes.  Eight parts are read before any is used.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_fwd_kernel.cuh"

namespace attn {

constexpr int kPromptMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPromptMergeThreads) attn_prompt_merge_kernel(const FwdParams p) {
  constexpr int kPer = D / 32;
  constexpr int kChunk = 8;
  __shared__ PromptPlan plan;
  __shared__ int tiles[kLevelSeqs + 1];  // (tile, head) pairs of the ranks before
  const int lane = threadIdx.x & 31;
  griddep_wait();  // the states are written
  griddep_launch_dependents();
  for (int i = threadIdx.x; i < static_cast<int>(sizeof(PromptPlan) / 4); i += blockDim.x)
    reinterpret_cast<int*>(&plan)[i] = __ldcg(reinterpret_cast<const int*>(p.plan) + i);
  __syncthreads();
  for (int r = threadIdx.x; r <= plan.split; r += blockDim.x) {
    int n = 0;
    for (int o = 0; o < r; ++o) n += (plan.first[o + 1] - plan.first[o]) / plan.parts[o];
    tiles[r] = n;
  }
  __syncthreads();
  const int rows = tiles[plan.split] * kBM;
  int r = 0;
  for (int at = blockIdx.x * (kPromptMergeThreads / 32) + (threadIdx.x >> 5); at < rows; at += gridDim.x * (kPromptMergeThreads / 32)) {
    while (tiles[r + 1] <= at / kBM) ++r;
    const int th = at / kBM - tiles[r], parts = plan.parts[r], b = plan.seq[r];
    const int tile = th / p.H, head = th - tile * p.H;
    const int qs = min(max(__ldg(p.cu_q + b), 0), p.total_q), qe = min(max(__ldg(p.cu_q + b + 1), qs), p.total_q);
    const int row = tile * kBM + at % kBM;
    if (row >= qe - qs) continue;
    const size_t first = (static_cast<size_t>(plan.first[r]) + static_cast<size_t>(th) * parts) * kBM + at % kBM;
    float M = -INFINITY, L = 0.f, acc[kPer] = {};
    for (int s0 = 0; s0 < parts; s0 += kChunk) {
      float ms[kChunk], ls[kChunk], os[kChunk][kPer];
#pragma unroll
      for (int c = 0; c < kChunk; ++c) {
        ms[c] = -INFINITY;
        ls[c] = 0.f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) os[c][k] = 0.f;
        if (s0 + c < parts) {
          const size_t i = first + static_cast<size_t>(s0 + c) * kBM;
          ms[c] = __ldg(p.st_m + i);
          ls[c] = __ldg(p.st_l + i);
          const float* src = p.st_o + i * D + lane * kPer;
          if constexpr (kPer == 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(src));
            os[c][0] = v.x;
            os[c][1] = v.y;
            os[c][2] = v.z;
            os[c][3] = v.w;
          } else {
            const float2 v = __ldg(reinterpret_cast<const float2*>(src));
            os[c][0] = v.x;
            os[c][1] = v.y;
          }
        }
      }
      auto weighed = [](float w, float x) { return fabsf(x) < INFINITY ? w * x : x; };
      float mc = M;
#pragma unroll
      for (int c = 0; c < kChunk; ++c) mc = fmaxf(mc, ms[c]);
      const float ref = mc == -INFINITY ? 0.f : mc;
      const float a = ex2_approx(M - ref);  // 0 while nothing was seen
      L *= a;
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = weighed(a, acc[k]);
#pragma unroll
      for (int c = 0; c < kChunk; ++c) {
        const float w = ex2_approx(ms[c] - ref);  // 0 for an empty part
        L = fmaf(w, ls[c], L);
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] += weighed(w, os[c][k]);
      }
      M = mc;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    __nv_bfloat16* dst = p.o + head * p.os_h + (static_cast<long long>(qs) + row) * p.os_r + lane * kPer;
    if constexpr (kPer == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0) p.lse[static_cast<size_t>(head) * p.total_q + qs + row] = L > 0.f || L != L ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace attn

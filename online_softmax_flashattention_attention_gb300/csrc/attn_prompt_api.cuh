// Host side of the entry points of include/attn.h that serve prompts and caches of bounded length
// (attn_qk_rotate, attn_fwd_prompt, attn_cache_weigh, attn_cache_evict).  Included by attn_lib.cu
// after attn_api.cu and attn_cache_api.cuh, whose checks, device set-up and launches it shares.
#pragma once

#include "attn_evict_kernel.cuh"
#include "attn_prompt_merge_kernel.cuh"
#include "attn_rotate_kernel.cuh"
#include "attn_weigh_kernel.cuh"

namespace {

// Positions of a sequence that weights are added to or evicted by, at most: the kernels count them in 32
// bits, by steps of up to 4096.
constexpr long long kMostPositions = INT32_MAX - 0x1ffffll;

// Strides (token, head) in elements of packed [total, heads, d] tensors; may_repeat: an input whose
// elements may be seen more than once.
attn_status check_strides(const int64_t* s, const char* name, bool may_repeat) {
  for (int i = 0; i < 2; ++i)
    if (s[i] < (may_repeat ? 0 : 8) || (s[i] & 7) != 0 || s[i] >= (1ll << 38))
      return fail(ATTN_ERR_BAD_ARG, "stride %lld of %s: must be a multiple of 8 elements (16 bytes) in [%d, 2^38)",
                  static_cast<long long>(s[i]), name, may_repeat ? 0 : 8);
  return ATTN_OK;
}

template <typename... Params, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(Params...), unsigned grid, unsigned cluster, unsigned block, size_t smem,
                               cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Strides as the kernels take them: those of an axis of one element may be anything, and are not used.
void fix_strides(const int64_t* s, int rows, int heads, int d, long long* row, long long* head) {
  *head = heads > 1 ? s[1] : d;
  *row = rows > 1 ? s[0] : static_cast<long long>(heads) * d;
}

// Whether a prompt's tiles go by cost (PromptWalk): 0 no, then head by head, as the packed forward has
// them; 1 yes; 2 where the sequences' lengths differ.  By cost, all K and V are read side by side, so beside
// sequences of eight tiles and more it takes that they stay in L2, or that a block read from DRAM serves
// enough scores (four heads' tiles at d = 128, where sequences of 2048 tokens on average are wanted too, one
// CTA's two tiles at d = 64).  Measured on GB300, by heads and by cost, us.  In L2, 32 / 8 heads: 8192
// tokens 455 and 423, at d = 64 339 and 307.  Past it, 150 to 330 MB of K and V, d = 128: 9 prompts of 900 to
// 8192 1893 and 1720, 24 of 500 to 4000 854 and 826, but 40 of 1000 549 and 593, 20 of 2048 722 and 752 (by
// heads in the same kernel 716); the 9 with a K/V head for two query heads 1896 and 1917, for one 1910 and
// 2159.  d = 64: 18 of 900 to 8192 2900 and 2420, 80 of 1000 864 and 737.  Too short for the ranks that the
// order needs: 77 tokens 6.2 and 7.3; 7 of 61 to 517 over prefixes of up to 5000, 16 / 4 heads, 45 and 50.
int prompt_by_cost(int B, int Hq, int Hkv, const Geometry& geo, int d, int causal, bool pair) {
  if (!causal || B > attn::kLevelSeqs || geo.grid_q <= 7 * attn::kBM) return 0;
  if (kv_footprint(1, Hkv, static_cast<int>(geo.k_rows), d) <= kRankMajorMaxKvBytes) return 1;
  if (d == 128) return Hq / Hkv >= 4 && geo.k_rows >= 2048ll * B ? 2 : 0;
  return pair || Hq / Hkv >= 2 ? 1 : 0;
}

template <int D>
attn_status prompt_params(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int Hq, int Hkv, int max_q,
                          float scale, int causal, uint32_t* status, const Geometry& geo, CUtensorMap* mq, CUtensorMap* mk,
                          CUtensorMap* mv, CUtensorMap* mo, attn::FwdParams* p) {
  attn_status st;
  Geometry no_keys = geo;
  no_keys.k_rows = 0;
  if ((st = make_launch<D, false>(Q, K, V, O, LSE, B, Hq, max_q, 0, scale, causal, nullptr, status, StateOut{},
                                  Variant{}, no_keys, mq, mk, mv, mo, p)) != ATTN_OK)
    return st;
  if (geo.k_rows > 0) {  // K and V have heads of their own
    if ((st = make_map(mk, K, D, geo.k_rows, Hkv, 1, geo.ks)) != ATTN_OK) return st;
    if ((st = make_map(mv, V, D, geo.k_rows, Hkv, 1, geo.vs)) != ATTN_OK) return st;
  }
  p->total_k = static_cast<int>(geo.k_rows);
  p->v = static_cast<const __nv_bfloat16*>(V);
  p->vs_r = geo.vs[2];
  p->vs_h = geo.vs[1];
  p->plan = nullptr;
  p->slots = 0;
  divisor(Hq / Hkv, &p->dm_g, &p->ds_g);
  return ATTN_OK;
}

// kPair: d = 64, two query tiles a CTA (attn_fwd_pair_kernel).
template <int D, bool kPair, bool kByCost>
attn_status launch_prompt(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int Hq, int Hkv,
                          int max_q, float scale, int causal, cudaStream_t stream, int dev, uint32_t* status,
                          const Geometry& geo, int cost) {
  static bool attr_set[kMaxDevices] = {};
  using C = std::conditional_t<kPair, attn::PairCfg, attn::FwdCfg<D>>;
  attn_status st;
  if constexpr (kPair)
    st = set_smem_attr(attn::attn_fwd_pair_kernel<0, true, true, kByCost>, C::kSmemAlloc, dev, attr_set);
  else
    st = set_smem_attr(attn::attn_fwd_kernel<D, false, 0, true, attn::kBN, true, kByCost>, C::kSmemAlloc, dev, attr_set);
  if (st != ATTN_OK) return st;
  CUtensorMap mq, mk, mv, mo;
  attn::FwdParams p;
  if ((st = prompt_params<D>(Q, K, V, O, LSE, B, Hq, Hkv, max_q, scale, causal, status, geo, &mq, &mk, &mv, &mo, &p)) != ATTN_OK)
    return st;
  if (kPair) {
    p.num_items = static_cast<int>(static_cast<long long>((p.num_qtiles + 1) / 2) * p.BH);
    p.order_div = (p.num_qtiles + 1) / 2;
  }
  if (kByCost) p.seq_sort = cost;  // the ranks' place
  set_divisors(&p);
  const unsigned grid = static_cast<unsigned>(std::min(p.num_items, sm_count(dev)));
  const int smem = p.seq_sort ? C::kSmemAlloc : C::kSmemAllocNoPerm;
  cudaError_t e;
  if constexpr (kPair)
    e = launch_pdl(attn::attn_fwd_pair_kernel<0, true, true, kByCost>, grid, attn::kPairThreads, smem, stream, mq, mk, mv, p);
  else
    e = launch_pdl(attn::attn_fwd_kernel<D, false, 0, true, attn::kBN, true, kByCost>, grid, attn::kThreads, smem, stream, mq, mk,
                   mv, mo, p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "kernel launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

// Whether a prompt's keys may be split (PromptPlan), by what the host knows: few tiles, and a sequence
// with so many keys that its tiles would still run when the others are done.  With several sequences that
// one is taken to have half of the prefixes' tokens.  Measured on GB300, split and not: 128 tokens over
// 2048, 32 heads, d = 128 18.1 and 19.8 us, over 4096 22.1 and 32.7, over 16384 43.9 and 106.3; 512 over
// 4096, 16 heads, d = 64 27.0 and 32.5; 7 prompts of 69 to 517 over prefixes up to 5000 20.3 and 44.6.
// The other way round (two launches, the plan): 128 over 512, 32 heads, d = 128 14.2 and 9.9; 512 over
// 4096 41.3 and 36.1.  Sequences as long as each other lose what an uneven batch would win, as the host knows
// the sum of their keys alone: 8 of 100 over 3000, 32 / 8 heads, 62.5 and 56.5; 4 of them 33.7 and 28.8; 8
// over 6000 102 and 95; 4 of 100 over 2000, 16 / 4 heads, 26.0 and 21.6.
bool prompt_splits(int B, int Hq, int max_q, int total_q, int total_k, int sms) {
  if (B > attn::kLevelSeqs) return false;
  const long long tiles = std::min(static_cast<long long>(total_q) / attn::kBM + B,
                                   static_cast<long long>(B) * ((max_q + attn::kBM - 1) / attn::kBM)) * Hq;
  if (tiles > 2ll * sms) return false;
  const double before = std::max(total_k - total_q, 0) / (B > 1 ? 2.0 : 1.0);
  const double blocks = (before + std::min(total_k, total_q) / static_cast<double>(B)) / attn::kBN;
  return blocks * (1.0 - 1.5 * static_cast<double>(tiles) / B / sms) >= 11.0;
}

// Workspace of such a call: the plan, and 4 states an SM.
constexpr size_t kPlanBytes = 1024;
static_assert(sizeof(attn::PromptPlan) <= kPlanBytes, "room");
size_t split_bytes(int sms, int d) { return kPlanBytes + static_cast<size_t>(4 * sms) * attn::kBM * (d + 2) * 4; }

template <int D>
attn_status launch_prompt_split(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int Hq, int Hkv,
                                int max_q, float scale, int causal, cudaStream_t stream, int dev, uint32_t* status,
                                const Geometry& geo, void* workspace) {
  static bool attr_set[kMaxDevices] = {};
  using C = attn::FwdCfg<D>;
  auto kernel = attn::attn_fwd_kernel<D, true, 0, true, attn::kBN, true, false>;
  attn_status st;
  if ((st = set_smem_attr(kernel, C::kSmemAlloc, dev, attr_set)) != ATTN_OK) return st;
  CUtensorMap mq, mk, mv, mo;
  attn::FwdParams p;
  if ((st = prompt_params<D>(Q, K, V, O, LSE, B, Hq, Hkv, max_q, scale, causal, status, geo, &mq, &mk, &mv, &mo, &p)) != ATTN_OK)
    return st;
  const int sms = sm_count(dev);
  p.plan = static_cast<attn::PromptPlan*>(workspace);
  p.slots = 4 * sms;
  p.st_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPlanBytes);
  p.st_m = p.st_o + static_cast<size_t>(p.slots) * attn::kBM * D;
  p.st_l = p.st_m + static_cast<size_t>(p.slots) * attn::kBM;
  set_divisors(&p);
  cudaError_t e = launch_pdl(kernel, static_cast<unsigned>(sms), attn::kThreads, C::kSmemAlloc, stream, mq, mk, mv, mo, p);
  if (e == cudaSuccess)
    e = launch_pdl(attn::attn_prompt_merge_kernel<D>, 4 * static_cast<unsigned>(sms), attn::kPromptMergeThreads, 0, stream, p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "kernel launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

// Q as (d, heads, tokens): a box holds `tokens` tokens of `heads` heads.
attn_status weigh_q_map(CUtensorMap* map, const void* Q, int d, int Hq, int total, int heads, int tokens) {
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(total), 1};
  cuuint64_t strides[3] = {row, row * Hq, row * Hq * total};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(Q), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return ATTN_OK;
}

template <int D, bool kF8>
attn_status launch_weigh(const void* Q, int Hq, const attn_cache* c, attn::WeighParams p, int dev, cudaStream_t stream) {
  static bool attr_set[kMaxDevices] = {};
  using C = attn::WeighCfg<D, kF8>;
  auto kernel = attn::attn_weigh_kernel<D, kF8>;
  attn_status st;
  if ((st = set_smem_attr(kernel, C::kSmem, dev, attr_set)) != ATTN_OK) return st;
  p.heads = std::min(p.G, attn::kWeighCols);
  p.tokens = attn::kWeighCols / p.heads;
  // a small copy of Q: whole groups of 8 rows (of the swizzle), if two and more of them make a tile
  p.small_tokens = p.heads % 8 == 0 ? 1 : p.heads % 4 == 0 ? 2 : p.heads % 2 == 0 ? 4 : 8;
  if (2 * p.small_tokens > p.tokens) p.small_tokens = p.tokens;
  p.box_rows = 128;  // the most keys that no page border cuts
  while (p.page % p.box_rows != 0) p.box_rows /= 2;
  // The stages of shared memory go to K or to Q by the tiles of query rows that a sequence has on
  // average: see WeighCfg.
  const bool many = static_cast<long long>(p.total_q) * p.G > 4ll * attn::kWeighCols * p.B;
  p.ring_k = many ? C::kManyK : C::kFewK;
  p.ring_q = many ? C::kManyQ : C::kFewQ;
  CUtensorMap mq, ms, mk = {};
  if ((st = weigh_q_map(&mq, Q, D, Hq, p.total_q, p.heads, p.tokens)) != ATTN_OK) return st;
  if ((st = weigh_q_map(&ms, Q, D, Hq, p.total_q, p.heads, p.small_tokens)) != ATTN_OK) return st;
  if (c->num_pages > 0 && (st = cache_map(&mk, c->k, c, p.box_rows)) != ATTN_OK) return st;
  cudaError_t e = launch_pdl(kernel, static_cast<unsigned>(sm_count(dev)), C::kThreads, C::kSmem, stream, mq, ms, mk, p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "weigh kernel launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

}  // namespace

extern "C" {

attn_status attn_qk_rotate(const void* Q, const void* K, void* Q_out, void* K_out, const int64_t* q_strides,
                           const int64_t* k_strides, const int64_t* q_out_strides, const int64_t* k_out_strides,
                           const int32_t* cu_seqlens, const int32_t* start_lens, const int32_t* positions,
                           const float* inv_freq, int num_freq, int interleaved, const void* q_weight,
                           const void* k_weight, int weight_type, float eps, int B, int Hq, int Hkv, int d, int total,
                           void* stream) {
  g_err[0] = '\0';
  attn_status st;
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED_D, "d=%d; supported: 64, 128", d);
  if (B < 0 || total < 0 || Hq < 0 || Hkv < 0 || Hq > kMaxHeads || Hkv > kMaxHeads)
    return fail(ATTN_ERR_BAD_SHAPE, "B=%d total=%d Hq=%d Hkv=%d; sizes must not be negative, heads at most %d", B, total,
                Hq, Hkv, kMaxHeads);
  if (num_freq < 0 || num_freq % 8 != 0 || 2 * static_cast<long long>(num_freq) > d)
    return fail(ATTN_ERR_BAD_SHAPE, "num_freq=%d; must be a multiple of 8 in [0, d / 2]", num_freq);
  if (weight_type != ATTN_WEIGHT_BF16 && weight_type != ATTN_WEIGHT_FP32)
    return fail(ATTN_ERR_BAD_ARG, "weight type %d; ATTN_WEIGHT_BF16 or ATTN_WEIGHT_FP32", weight_type);
  if (!std::isfinite(eps) || eps < 0.f) return fail(ATTN_ERR_BAD_ARG, "eps must be finite and >= 0");
  if (!cu_seqlens && B != 1) return fail(ATTN_ERR_BAD_SHAPE, "B=%d; without cu_seqlens all rows are one sequence (B = 1)", B);
  if (B == 0 || total == 0 || Hq + Hkv == 0) return ATTN_OK;
  const void* src[2] = {Q, K};
  void* dst[2] = {Q_out, K_out};
  const void* weight[2] = {q_weight, k_weight};
  const int64_t* in[2] = {q_strides, k_strides};
  const int64_t* out[2] = {q_out_strides, k_out_strides};
  const int heads[2] = {Hq, Hkv};
  const char* names[2] = {"Q", "K"};
  const char* out_names[2] = {"Q_out", "K_out"};
  attn::RotateParams p = {};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (!src[i] || !dst[i]) return fail(ATTN_ERR_NULLPTR, "%s and %s must not be NULL", names[i], out_names[i]);
    if (odd16(src[i]) || odd16(dst[i]))
      return fail(ATTN_ERR_MISALIGNED, "%s and %s must be 16-byte aligned", names[i], out_names[i]);
    if (!in[i] || !out[i]) return fail(ATTN_ERR_NULLPTR, "the strides of %s and %s must not be NULL", names[i], out_names[i]);
    fix_strides(in[i], total, heads[i], d, &p.src_t[i], &p.src_h[i]);
    fix_strides(out[i], total, heads[i], d, &p.dst_t[i], &p.dst_h[i]);
    const int64_t used_in[2] = {p.src_t[i], p.src_h[i]}, used_out[2] = {p.dst_t[i], p.dst_h[i]};
    if ((st = check_strides(used_in, names[i], true)) != ATTN_OK) return st;
    if ((st = check_strides(used_out, out_names[i], false)) != ATTN_OK) return st;
    if (odd_to(weight[i], weight_type == ATTN_WEIGHT_FP32 ? 4 : 2))
      return fail(ATTN_ERR_MISALIGNED, "a weight must be aligned to its type");
    p.src[i] = static_cast<const __nv_bfloat16*>(src[i]);
    p.dst[i] = static_cast<__nv_bfloat16*>(dst[i]);
    p.weight[i] = weight[i];
  }
  if (num_freq > 0 && !inv_freq) return fail(ATTN_ERR_NULLPTR, "inv_freq must not be NULL when num_freq > 0");
  if (odd_to(inv_freq, 4) || odd_to(cu_seqlens, 4) || odd_to(start_lens, 4) || odd_to(positions, 4))
    return fail(ATTN_ERR_MISALIGNED, "inv_freq, cu_seqlens, start_lens and positions must be 4-byte aligned");
  p.cu = cu_seqlens;
  p.start = start_lens;
  p.positions = positions;
  p.freq = inv_freq;
  p.num_freq = num_freq;
  p.weight_f32 = weight_type == ATTN_WEIGHT_FP32;
  p.eps = eps;
  p.B = B;
  p.Hq = Hq;
  p.H = Hq + Hkv;
  p.total = total;
  int dev;
  uint32_t* status;
  if ((st = get_device(&dev)) != ATTN_OK || (st = setup(dev, &status)) != ATTN_OK) return st;
  // A block takes all heads of its tokens, so that their angles are computed once, unless that
  // leaves SMs idle; then as few as it has in flight.
  const unsigned blocks = (static_cast<unsigned>(total) + attn::kRotTokens - 1) / attn::kRotTokens;
  const unsigned full = 3u * static_cast<unsigned>(sm_count(dev));  // blocks that run at once
  const int least = attn::kRotThreads / (d / 8) / attn::kRotTokens * attn::kRotUnroll;
  p.heads_per_block = 2 * blocks >= full ? p.H : least;
  const unsigned parts = static_cast<unsigned>((p.H + p.heads_per_block - 1) / p.heads_per_block);
  const dim3 grid(parts == 1 ? std::min(blocks, full) : blocks, parts);
  using Kernel = void (*)(attn::RotateParams);
  const bool all = 2 * num_freq == d;
  auto pick = [&](Kernel pairs_all, Kernel pairs, Kernel halves_all, Kernel halves) {
    return interleaved ? (all ? pairs_all : pairs) : (all ? halves_all : halves);
  };
  const Kernel kernel = d == 128 ? pick(attn::attn_qk_rotate_kernel<128, true, true>, attn::attn_qk_rotate_kernel<128, true, false>,
                                        attn::attn_qk_rotate_kernel<128, false, true>, attn::attn_qk_rotate_kernel<128, false, false>)
                                 : pick(attn::attn_qk_rotate_kernel<64, true, true>, attn::attn_qk_rotate_kernel<64, true, false>,
                                        attn::attn_qk_rotate_kernel<64, false, true>, attn::attn_qk_rotate_kernel<64, false, false>);
  cudaError_t e = launch_pdl2(kernel, grid, attn::kRotThreads, 0, static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "rotate kernel launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

size_t attn_prompt_workspace_bytes(int B, int Hq, int max_seqlen_q, int total_q, int total_k, int d) {
  if (B < 1 || Hq < 1 || Hq > kMaxHeads || max_seqlen_q < 1 || total_q < 1 || total_k < 1 || (d != 64 && d != 128)) return 0;
  if (max_seqlen_q > INT32_MAX - 255) return 0;
  int dev;
  uint32_t* status = nullptr;
  if (get_device(&dev) != ATTN_OK || setup(dev, &status) != ATTN_OK) return 0;
  const int sms = sm_count(dev);
  return prompt_splits(B, Hq, max_seqlen_q, total_q, total_k, sms) ? split_bytes(sms, d) : 0;
}

attn_status attn_fwd_prompt(const void* Q, const void* K, const void* V, void* O, float* LSE, const int64_t* q_strides,
                            const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                            const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B, int Hq, int Hkv,
                            int max_seqlen_q, int total_q, int total_k, int d, float scale, int causal, void* workspace,
                            size_t workspace_bytes, void* stream) {
  g_err[0] = '\0';
  attn_status st;
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED_D, "d=%d; supported: 64, 128", d);
  if (B < 0 || Hq < 0 || max_seqlen_q < 0 || total_q < 0 || total_k < 0)
    return fail(ATTN_ERR_BAD_SHAPE, "negative size (B=%d Hq=%d max_seqlen_q=%d total_q=%d total_k=%d)", B, Hq,
                max_seqlen_q, total_q, total_k);
  if (Hkv < 1 || Hkv > kMaxHeads || Hq > kMaxHeads || Hq % Hkv != 0)
    return fail(ATTN_ERR_BAD_SHAPE, "Hq=%d must be a multiple of Hkv=%d, both at most %d", Hq, Hkv, kMaxHeads);
  // rows are counted in 32 bits, rounded up to a block of 128
  if (max_seqlen_q > INT32_MAX - 255 || total_q > INT32_MAX - 255 || total_k > INT32_MAX - 255)
    return fail(ATTN_ERR_BAD_SHAPE, "max_seqlen_q, total_q and total_k are at most 2^31 - 256");
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(ATTN_ERR_BAD_ARG, "scale must be finite and > 0");
  if (static_cast<long long>(B) * Hq == 0 || max_seqlen_q == 0 || total_q == 0) return ATTN_OK;
  const long long seq_heads = static_cast<long long>(B) * Hq, tiles = row_tiles(max_seqlen_q);
  if (seq_heads > kMostItems || seq_heads * tiles > kMostItems)
    return fail(ATTN_ERR_BAD_SHAPE, "problem too large (%lld tiles of 128 rows for each of %lld sequences' heads)", tiles, seq_heads);
  if (!Q || !O || !LSE || !cu_seqlens_q || !cu_seqlens_k)
    return fail(ATTN_ERR_NULLPTR, "Q, O, LSE and the cu_seqlens arrays must not be NULL");
  if (total_k > 0 && (!K || !V)) return fail(ATTN_ERR_NULLPTR, "K and V must not be NULL when total_k > 0");
  if (odd16(Q) || odd16(O) || (total_k > 0 && (odd16(K) || odd16(V))))
    return fail(ATTN_ERR_MISALIGNED, "Q, K, V and O must be 16-byte aligned");
  if (odd_to(LSE, 4) || odd_to(cu_seqlens_q, 4) || odd_to(cu_seqlens_k, 4))
    return fail(ATTN_ERR_MISALIGNED, "LSE and the cu_seqlens arrays must be 4-byte aligned");
  Geometry g;
  const int64_t* in[4] = {q_strides, k_strides, v_strides, o_strides};
  const char* names[4] = {"Q", "K", "V", "O"};
  long long* out[4] = {g.qs, g.ks, g.vs, g.os};
  for (int i = 0; i < 4; ++i) {
    const bool kv = i == 1 || i == 2;
    if (kv && total_k == 0) {
      out[i][0] = out[i][1] = out[i][2] = d;
      continue;
    }
    const int rows = kv ? total_k : total_q, heads = kv ? Hkv : Hq;
    if (!in[i]) return fail(ATTN_ERR_NULLPTR, "%s's strides must not be NULL", names[i]);
    fix_strides(in[i], rows, heads, d, &out[i][2], &out[i][1]);
    const int64_t used[2] = {out[i][2], out[i][1]};
    if ((st = check_strides(used, names[i], false)) != ATTN_OK) return st;
    out[i][0] = 8;  // one batch
  }
  g.q_rows = total_q;
  g.k_rows = total_k;
  g.map_b = 1;
  g.grid_q = max_seqlen_q;
  g.cu_q = cu_seqlens_q;
  g.cu_k = cu_seqlens_k;
  int dev;
  uint32_t* status = nullptr;
  if ((st = get_device(&dev)) != ATTN_OK || (st = setup(dev, &status)) != ATTN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = sm_count(dev);
  if (workspace && prompt_splits(B, Hq, max_seqlen_q, total_q, total_k, sms)) {
    if (odd16(workspace)) return fail(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    if (workspace_bytes < split_bytes(sms, d))
      return fail(ATTN_ERR_BAD_ARG, "workspace of %zu B is smaller than the %zu B needed", workspace_bytes, split_bytes(sms, d));
    return (d == 128 ? launch_prompt_split<128> : launch_prompt_split<64>)(Q, K, V, O, LSE, B, Hq, Hkv, max_seqlen_q, scale, causal,
                                                                           s, dev, status, g, workspace);
  }
  const bool pair = d == 64 && use_pair_kernel(dev, B, Hq, g, causal);
  const int cost = prompt_by_cost(B, Hq, Hkv, g, d, causal, pair);
  auto launch = d == 128 ? (cost ? launch_prompt<128, false, true> : launch_prompt<128, false, false>)
                : pair   ? (cost ? launch_prompt<64, true, true> : launch_prompt<64, true, false>)
                         : (cost ? launch_prompt<64, false, true> : launch_prompt<64, false, false>);
  return launch(Q, K, V, O, LSE, B, Hq, Hkv, max_seqlen_q, scale, causal, s, dev, status, g, cost);
}

attn_status attn_cache_weigh(const void* Q, const float* LSE, const attn_cache* cache, const float* weights, float* out,
                             const int32_t* block_table, int max_pages, const int32_t* cu_seqlens_q,
                             const int32_t* ctx_lens, int B, int Hq, int total_q, float scale, float decay,
                             void* stream) {
  g_err[0] = '\0';
  attn_status st = check_cache(cache, max_pages, false);
  if (st != ATTN_OK) return st;
  if (static_cast<long long>(max_pages) * cache->page_size > kMostPositions)
    return fail(ATTN_ERR_BAD_SHAPE, "max_pages=%d: a sequence has at most %lld positions", max_pages, kMostPositions);
  if (B < 0 || Hq < 0 || total_q < 0)
    return fail(ATTN_ERR_BAD_SHAPE, "negative size (B=%d Hq=%d total_q=%d)", B, Hq, total_q);
  if (Hq > kMaxHeads) return fail(ATTN_ERR_BAD_SHAPE, "Hq=%d; at most %d", Hq, kMaxHeads);
  if (Hq % cache->num_heads != 0)
    return fail(ATTN_ERR_BAD_SHAPE, "Hq=%d must be a multiple of the cache's %d heads", Hq, cache->num_heads);
  if (!std::isfinite(scale) || !(scale >= 0x1p-100f)) return fail(ATTN_ERR_BAD_ARG, "scale must be finite and at least 2^-100");
  if (!std::isfinite(decay)) return fail(ATTN_ERR_BAD_ARG, "decay must be finite");
  if (B == 0 || Hq == 0 || total_q == 0) return ATTN_OK;
  if (!Q || !LSE || !out) return fail(ATTN_ERR_NULLPTR, "Q, LSE and out must not be NULL");
  if (decay != 0.f && !weights) return fail(ATTN_ERR_NULLPTR, "weights must not be NULL unless decay is 0");
  if ((st = check_table(block_table, max_pages, cu_seqlens_q, ctx_lens)) != ATTN_OK) return st;
  if (odd16(Q)) return fail(ATTN_ERR_MISALIGNED, "Q must be 16-byte aligned");
  if (odd_to(LSE, 4) || odd_to(weights, 4) || odd_to(out, 4))
    return fail(ATTN_ERR_MISALIGNED, "LSE, weights and out must be 4-byte aligned");
  // tiles of query rows are counted in 32 bits
  const int G = Hq / cache->num_heads;
  if (static_cast<long long>(total_q) * ((G + attn::kWeighCols - 1) / attn::kWeighCols) > INT32_MAX - 255)
    return fail(ATTN_ERR_BAD_SHAPE, "total_q=%d is too large for %d heads a group", total_q, G);
  attn::WeighParams p = {};
  int dev;
  if ((st = cache_device(&dev, &p.status, &p.page_word)) != ATTN_OK) return st;
  p.lse = LSE;
  p.ks = cache->k_scale;
  p.w = weights;
  p.out = out;
  p.table = block_table;
  p.cu = cu_seqlens_q;
  p.ctx = ctx_lens;
  p.B = B;
  p.Hkv = cache->num_heads;
  p.G = G;
  p.total_q = total_q;
  p.num_pages = cache->num_pages;
  p.page = cache->page_size;
  p.max_pages = max_pages;
  p.cap = max_pages * cache->page_size;
  p.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.rscale = 1.f / scale;
  p.decay = decay;
  p.timeout_ns = wait_limit_ns();
  const bool f8 = cache->type == ATTN_CACHE_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 128)
    return f8 ? launch_weigh<128, true>(Q, Hq, cache, p, dev, s) : launch_weigh<128, false>(Q, Hq, cache, p, dev, s);
  return f8 ? launch_weigh<64, true>(Q, Hq, cache, p, dev, s) : launch_weigh<64, false>(Q, Hq, cache, p, dev, s);
}

attn_status attn_cache_evict(const attn_cache* cache, float* weights, const int32_t* block_table, int max_pages,
                             const int32_t* out_table, int out_max_pages, const int32_t* lens, int32_t* kept,
                             int32_t* out_lens, int B, int keep, int sink, int recent, void* stream) {
  g_err[0] = '\0';
  attn_status st = check_cache(cache, max_pages);
  if (st != ATTN_OK) return st;
  const bool in_place = !out_table || out_table == block_table;
  if (B < 0 || keep < 0 || sink < 0 || recent < 0 || static_cast<long long>(sink) + recent > keep)
    return fail(ATTN_ERR_BAD_SHAPE, "B=%d keep=%d sink=%d recent=%d; none negative, sink + recent at most keep", B, keep,
                sink, recent);
  const long long room = static_cast<long long>(max_pages) * cache->page_size;
  if (room > kMostPositions || keep > kMostPositions)
    return fail(ATTN_ERR_BAD_SHAPE, "a sequence of %lld positions, keep=%d; at most %lld", room, keep, kMostPositions);
  if (!in_place) {
    if (out_max_pages < 0 || static_cast<long long>(out_max_pages) * cache->page_size > INT32_MAX - 255)
      return fail(ATTN_ERR_BAD_SHAPE, "out_max_pages=%d: a sequence has at most 2^31 - 256 positions", out_max_pages);
    if (static_cast<long long>(out_max_pages) * cache->page_size < std::min<long long>(keep, room))
      return fail(ATTN_ERR_BAD_SHAPE, "out_table has room for %lld positions of %lld kept",
                  static_cast<long long>(out_max_pages) * cache->page_size, std::min<long long>(keep, room));
  } else if (out_table && out_max_pages != max_pages) {
    return fail(ATTN_ERR_BAD_SHAPE, "out_table is block_table: out_max_pages=%d must be max_pages=%d", out_max_pages, max_pages);
  }
  if (B == 0) return ATTN_OK;
  if (!lens || !out_lens || (keep > 0 && !kept)) return fail(ATTN_ERR_NULLPTR, "lens, kept and out_lens must not be NULL");
  // (every CTA reads its sequence's length, at a time of its own)
  const uintptr_t in0 = reinterpret_cast<uintptr_t>(lens), out0 = reinterpret_cast<uintptr_t>(out_lens);
  if ((in0 > out0 ? in0 - out0 : out0 - in0) < static_cast<uintptr_t>(B) * sizeof(int32_t))
    return fail(ATTN_ERR_BAD_ARG, "out_lens must not overlap lens");
  if (max_pages > 0 && !block_table) return fail(ATTN_ERR_NULLPTR, "block_table must not be NULL");
  if (cache->num_pages > 0 && !weights) return fail(ATTN_ERR_NULLPTR, "weights must not be NULL");
  if (odd_to(weights, 4) || odd_to(block_table, 4) || odd_to(out_table, 4) || odd_to(lens, 4) || odd_to(kept, 4) ||
      odd_to(out_lens, 4))
    return fail(ATTN_ERR_MISALIGNED, "weights, tables, lens, kept and out_lens must be 4-byte aligned");
  attn::EvictParams p = {};
  int dev;
  uint32_t* status;
  if ((st = cache_device(&dev, &status, &p.page_word)) != ATTN_OK) return st;
  p.k = static_cast<uint8_t*>(cache->k);
  p.v = static_cast<uint8_t*>(cache->v);
  p.ks = cache->type == ATTN_CACHE_E4M3 ? cache->k_scale : nullptr;
  p.vs = cache->type == ATTN_CACHE_E4M3 ? cache->v_scale : nullptr;
  p.w = weights;
  p.table = block_table;
  p.to = in_place ? block_table : out_table;
  p.lens = lens;
  p.kept = kept;
  p.out_lens = out_lens;
  p.B = B;
  p.Hkv = cache->num_heads;
  p.num_pages = cache->num_pages;
  p.page = cache->page_size;
  p.max_pages = max_pages;
  p.to_pages = in_place ? max_pages : out_max_pages;
  p.keep = keep;
  p.sink = sink;
  p.recent = recent;
  p.row_bytes = cache->d * (cache->type == ATTN_CACHE_E4M3 ? 1 : 2);
  p.in_place = in_place ? 1 : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // A unit's weights are shared by as many CTAs as hold 8192 of them each, 8 at most, while SMs are idle.  How
  // many keys a CTA has room for goes by the table, as the lengths are the device's: 48 sequences of up to 16384
  // tokens with tables of as many positions (64 KB a CTA, two an SM) 151 us, of 131072 (192 KB, one) 193.
  const long long units = static_cast<long long>(B) * p.Hkv;
  unsigned cluster = 1;
  while (cluster < 8 && room > 8192ll * cluster && units * cluster < sm_count(dev)) cluster *= 2;
  p.key_cap = static_cast<int>(std::min<long long>((room + cluster - 1) / cluster, attn::kEvictMaxKeys));
  static bool attr_set[kMaxDevices] = {};
  if ((st = set_smem_attr(attn::attn_evict_select_kernel, attn::kEvictMaxKeys * 4, dev, attr_set)) != ATTN_OK) return st;
  // Packing: in place a block walks all rows of some columns; else rows in runs of 256.
  int slices = 1;
  const long long most = std::min<long long>(keep, room);
  p.rows_per_block = 256;
  if (in_place) {
    while (slices * 32 < p.row_bytes && units * slices < 2 * sm_count(dev)) slices *= 2;
    p.rows_per_block = INT32_MAX;
  }
  p.slice = p.row_bytes / slices;
  const long long blocks = in_place ? slices : (most + p.rows_per_block - 1) / p.rows_per_block;
  if (units * cluster > INT32_MAX || units * (blocks + 1) > INT32_MAX)
    return fail(ATTN_ERR_BAD_SHAPE, "too many (sequence, head) units (%lld)", units);
  cudaError_t e = launch_pdl_cluster(attn::attn_evict_select_kernel, static_cast<unsigned>(units * cluster), cluster,
                                     attn::kEvictThreads, static_cast<size_t>(p.key_cap) * 4, s, p);
  if (e == cudaSuccess && keep > 0)
    e = launch_pdl(attn::attn_evict_move_kernel, static_cast<unsigned>(units * (blocks + 1)), attn::kMoveThreads, 0,
                   s, p, static_cast<int>(blocks));
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "evict kernel launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

}  // extern "C"

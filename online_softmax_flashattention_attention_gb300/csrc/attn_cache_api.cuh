// Host side of the paged-cache entry points of include/attn.h (attn_cache_write,
// attn_cache_read, attn_fwd_tree and what belongs to them).  Included by attn_lib.cu after
// attn_api.cu, whose argument checks, error text, device set-up and launch it shares.
#pragma once

#include "attn_cache_kernel.cuh"
#include "attn_tree_kernel.cuh"
#include "attn_tree_tile_kernel.cuh"

namespace {

// Bit 0: a position without a page, or a block-table entry outside the cache, was met since
// attn_cache_check last read the word (device array of the library: no allocation).
static __device__ uint32_t g_page_word[4];
uint32_t* g_page_addr[kMaxDevices] = {};

attn_status page_word(int dev, uint32_t** out) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_page_addr[dev]) {
    void* a = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&a, g_page_word);
    if (e != cudaSuccess || !a) return fail(ATTN_ERR_NO_DEVICE, "cudaGetSymbolAddress: %s", cudaGetErrorString(e));
    g_page_addr[dev] = static_cast<uint32_t*>(a);
  }
  *out = g_page_addr[dev];
  return ATTN_OK;
}

constexpr int kMaxPage = 65536, kMaxHeads = 65536;

bool odd16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool odd_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

attn_status check_cache(const attn_cache* c, int max_pages) {
  if (!c) return fail(ATTN_ERR_NULLPTR, "cache must not be NULL");
  if (c->size < sizeof(attn_cache))
    return fail(ATTN_ERR_BAD_ARG, "attn_cache.size=%zu; expected at least %zu", c->size, sizeof(attn_cache));
  if (c->d != 64 && c->d != 128) return fail(ATTN_ERR_UNSUPPORTED_D, "d=%d; supported: 64, 128", c->d);
  if (c->type != ATTN_CACHE_BF16 && c->type != ATTN_CACHE_E4M3)
    return fail(ATTN_ERR_BAD_ARG, "cache type %d; ATTN_CACHE_BF16 or ATTN_CACHE_E4M3", c->type);
  if (c->page_size < 16 || c->page_size % 16 != 0 || c->page_size > kMaxPage)
    return fail(ATTN_ERR_BAD_SHAPE, "page_size=%d; must be a multiple of 16 in [16, %d]", c->page_size, kMaxPage);
  if (c->num_pages < 0 || c->num_heads < 1 || c->num_heads > kMaxHeads)
    return fail(ATTN_ERR_BAD_SHAPE, "num_pages=%d num_heads=%d; num_pages >= 0, num_heads in [1, %d]", c->num_pages,
                c->num_heads, kMaxHeads);
  // the kernels round positions up to a block of keys in 32 bits
  if (max_pages < 0 || static_cast<long long>(max_pages) * c->page_size > INT32_MAX - 255)
    return fail(ATTN_ERR_BAD_SHAPE, "max_pages=%d: a sequence has at most 2^31 - 256 positions", max_pages);
  if (c->num_pages > 0) {
    if (!c->k || !c->v) return fail(ATTN_ERR_NULLPTR, "the cache's k and v must not be NULL");
    if (odd16(c->k) || odd16(c->v)) return fail(ATTN_ERR_MISALIGNED, "the cache's k and v must be 16-byte aligned");
    if (c->type == ATTN_CACHE_E4M3) {
      if (!c->k_scale || !c->v_scale) return fail(ATTN_ERR_NULLPTR, "an e4m3 cache needs k_scale and v_scale");
      if (odd16(c->k_scale) || odd16(c->v_scale))
        return fail(ATTN_ERR_MISALIGNED, "k_scale and v_scale must be 16-byte aligned");
    }
  }
  return ATTN_OK;
}

attn_status check_table(const int32_t* table, int max_pages, const int32_t* cu, const int32_t* lens) {
  if (!cu) return fail(ATTN_ERR_NULLPTR, "the cu_seqlens array must not be NULL");
  if (max_pages > 0 && !table) return fail(ATTN_ERR_NULLPTR, "block_table must not be NULL");
  if (odd_to(table, 4) || odd_to(cu, 4) || odd_to(lens, 4))
    return fail(ATTN_ERR_MISALIGNED, "block_table, cu_seqlens and the lengths must be 4-byte aligned");
  return ATTN_OK;
}

attn::CacheParams cache_params(const attn_cache* c, const int32_t* table, int max_pages, const int32_t* cu,
                               const int32_t* start, int B, int total) {
  attn::CacheParams p = {};
  p.k = c->k;
  p.v = c->v;
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.table = table;
  p.cu = cu;
  p.start = start;
  p.B = B;
  p.Hkv = c->num_heads;
  p.num_pages = c->num_pages;
  p.page = c->page_size;
  p.max_pages = max_pages;
  p.total = total;
  return p;
}

// Blocks of a cache kernel, or an error when there are too many.
attn_status cache_grid(const attn_cache* c, int total, unsigned* grid) {
  const long long items = static_cast<long long>(total) * c->num_heads;
  const int per = c->d == 128 ? attn::CacheTile<128>::kPerBlock : attn::CacheTile<64>::kPerBlock;
  const long long n = (items + per - 1) / per;
  if (n > INT32_MAX) return fail(ATTN_ERR_BAD_SHAPE, "too many (token, head) rows (%lld)", items);
  *grid = static_cast<unsigned>(n);
  return ATTN_OK;
}

using CacheKernel = void (*)(attn::CacheParams);

attn_status launch_cache(CacheKernel kernel, unsigned grid, const attn::CacheParams& p, void* stream) {
  cudaError_t e = launch_pdl(kernel, grid, attn::kCacheThreads, 0, static_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "cache kernel launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

// Device set-up shared by the entry points below: the current device and its two words.
attn_status cache_device(int* dev, uint32_t** status, uint32_t** pages) {
  attn_status st = get_device(dev);
  if (st == ATTN_OK) st = setup(*dev, status);
  if (st == ATTN_OK) st = page_word(*dev, pages);
  return st;
}

// 4-D map (d, page rows, heads, pages) of the cache's K or V, box (128 bytes at most, box_rows).
attn_status cache_map(CUtensorMap* map, const void* ptr, const attn_cache* c, int box_rows) {
  const bool f8 = c->type == ATTN_CACHE_E4M3;
  const cuuint64_t row = static_cast<cuuint64_t>(c->d) * (f8 ? 1 : 2);
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                        static_cast<cuuint64_t>(c->num_heads), static_cast<cuuint64_t>(c->num_pages)};
  cuuint64_t strides[3] = {row, row * c->page_size, row * c->page_size * c->num_heads};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(f8 ? c->d : 64), static_cast<cuuint32_t>(box_rows), 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = f8 && c->d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  CUresult r = g_encode(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                        const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return ATTN_OK;
}

// Workspace of attn_fwd_tree: room for this many CTAs (up to three an SM, or one), whatever the
// device has, so that its size follows from the arguments alone.
constexpr int kTreeMaxCtas = 480;
constexpr int kTileMaxCtas = 160;

// Whether a call takes the 128-row tiles: when a sequence may have more rows than one 16-row
// tile, whose second tile would read the keys again.  Measured on GB300, 32 query and 8 K/V heads,
// d = 128, page 64, 16 rows in the 16-row kernel and 20 in the other: one sequence of 131072 tokens
// bf16 94 and 88 us, e4m3 66 and 95; 64 sequences of 500 tokens bf16 36 and 38, e4m3 37 and 52.
// The other way round, 32 rows: 119 and 89, 106 and 96; 60 and 40, 59 and 52.
bool use_tile_kernel(int G, int max_seqlen_q) { return G <= attn::kTileRows && G * max_seqlen_q > attn::kTreeRows; }

struct TreeSpace {
  size_t o, m, l, meta, total;  // byte offsets
};
TreeSpace tree_space(int rows, int ctas, int d) {
  TreeSpace s;
  const size_t n = static_cast<size_t>(2) * ctas * rows;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  s.o = 0;
  s.m = up(n * d * 4);
  s.l = s.m + up(n * 4);
  s.meta = s.l + up(n * 4);
  s.total = s.meta + up(static_cast<size_t>(2 * ctas) * sizeof(int4));
  return s;
}

// Launches `kernel` with programmatic stream serialization on a 2-D grid.
template <typename... Params, typename... Args>
cudaError_t launch_pdl2(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                        Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <int D, bool kF8>
attn_status launch_tree(const attn_cache* c, attn::TreeParams p, void* ws, cudaStream_t stream, int dev) {
  static bool attr_set[kMaxDevices] = {};
  using C = attn::TreeCfg<D, kF8>;
  auto kernel = attn::attn_tree_kernel<D, kF8>;
  attn_status st;
  if ((st = set_smem_attr(kernel, C::kSmem, dev, attr_set)) != ATTN_OK) return st;
  CUtensorMap mk = {}, mv = {};
  if (c->num_pages > 0) {  // without pages nothing is loaded
    if ((st = cache_map(&mk, c->k, c, 16)) != ATTN_OK) return st;
    if ((st = cache_map(&mv, c->v, c, 16)) != ATTN_OK) return st;
  }
  const unsigned grid = static_cast<unsigned>(std::min(kTreeMaxCtas, C::kCtas * sm_count(dev)));
  const TreeSpace sp = tree_space(attn::kTreeRows, kTreeMaxCtas, D);
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.st_o = reinterpret_cast<float*>(w + sp.o);
  p.st_m = reinterpret_cast<float*>(w + sp.m);
  p.st_l = reinterpret_cast<float*>(w + sp.l);
  p.meta = reinterpret_cast<int4*>(w + sp.meta);
  // Measured on GB300 (0, 2, 4, 8, 14 tried): 7 chains over contexts of 0 to 5000 tokens at d = 64
  // 94, 36, 29, 28, 32 us; 64 sequences of 1000 to 16384 e4m3 tokens 227, 209, 198, 204, 215 us.
  p.fan = 1;
  p.unit_cost = D == 128 ? 4 : 6;
  cudaError_t e = launch_pdl(kernel, grid, attn::kTreeThreads, C::kSmem, stream, mk, mv, p);
  if (e == cudaSuccess)
    e = launch_pdl2(attn::attn_tree_merge_kernel<D, attn::kTreeRows>, dim3(grid, attn::kTreeRows / 4), 128, 0, stream,
                    p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "tree attention launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

// Q as (d, heads of a group, groups, tokens); a box is a tile's rows.
attn_status tile_q_map(CUtensorMap* map, const attn::TreeParams& p, int d) {
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.G), static_cast<cuuint64_t>(p.Hkv),
                        static_cast<cuuint64_t>(p.total_q)};
  cuuint64_t strides[3] = {row, row * p.G, row * p.Hq};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(p.G), 1, static_cast<cuuint32_t>(p.tok_tile)};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<__nv_bfloat16*>(p.q), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return ATTN_OK;
}

template <int D, bool kF8>
attn_status launch_tile(const attn_cache* c, attn::TreeParams p, void* ws, cudaStream_t stream, int dev) {
  static bool attr_set[kMaxDevices] = {};
  using C = attn::TileCfg<D, kF8>;
  auto kernel = attn::attn_tree_tile_kernel<D, kF8>;
  attn_status st;
  if ((st = set_smem_attr(kernel, C::kSmem, dev, attr_set)) != ATTN_OK) return st;
  p.tok_tile = attn::kTileRows / p.G;
  p.unit_cost = 4;  // measured (2, 3, 4, 6): within 5 % of the best of them in 18 batches, the others within 10 to 15
  p.box_rows = 128;  // the most keys that no page border cuts
  while (p.page % p.box_rows != 0) p.box_rows /= 2;
  CUtensorMap mq, mk = {}, mv = {};
  if ((st = tile_q_map(&mq, p, D)) != ATTN_OK) return st;
  if (c->num_pages > 0) {
    if ((st = cache_map(&mk, c->k, c, p.box_rows)) != ATTN_OK) return st;
    if ((st = cache_map(&mv, c->v, c, p.box_rows)) != ATTN_OK) return st;
  }
  // Two CTAs walk the same keys with a tile each, so that the second reads them from L2, where
  // the keys' bandwidth is the limit (256-byte rows) and sequences have more than a tile of
  // tokens on average.  Measured on GB300 against a unit a tile: 131072 tokens, 64 drafts, 4 heads
  // a group 166 -> 132 us; 32 sequences with 1 to 64 drafts, a tile or less on average, 79 -> 107.
  p.fan = !kF8 && D == 128 && p.total_q > static_cast<long long>(p.tok_tile) * p.B ? 2 : 1;
  const unsigned grid = static_cast<unsigned>(std::min(kTileMaxCtas, std::max(sm_count(dev), p.fan)) / p.fan * p.fan);
  const TreeSpace sp = tree_space(attn::kTileRows, kTileMaxCtas, D);
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.st_o = reinterpret_cast<float*>(w + sp.o);
  p.st_m = reinterpret_cast<float*>(w + sp.m);
  p.st_l = reinterpret_cast<float*>(w + sp.l);
  p.meta = reinterpret_cast<int4*>(w + sp.meta);
  cudaError_t e = launch_pdl(kernel, grid, C::kThreads, C::kSmem, stream, mq, mk, mv, p);
  if (e == cudaSuccess)
    e = launch_pdl2(attn::attn_tree_merge_kernel<D, attn::kTileRows>, dim3(grid, attn::kTileRows / 4), 128, 0, stream,
                    p);
  if (e != cudaSuccess) return fail(ATTN_ERR_LAUNCH, "tree attention launch: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

template <int D, bool kF8>
attn_status launch_tree_any(const attn_cache* c, const attn::TreeParams& p, void* ws, cudaStream_t stream, int dev) {
  return use_tile_kernel(p.G, p.max_q) ? launch_tile<D, kF8>(c, p, ws, stream, dev)
                                       : launch_tree<D, kF8>(c, p, ws, stream, dev);
}

}  // namespace

extern "C" {

attn_status attn_cache_write(const attn_cache* cache, const void* K, const void* V, const int64_t* k_strides,
                             const int64_t* v_strides, const int32_t* block_table, int max_pages,
                             const int32_t* cu_seqlens, const int32_t* start_lens, int B, int total, void* stream) {
  g_err[0] = '\0';
  attn_status st = check_cache(cache, max_pages);
  if (st != ATTN_OK) return st;
  if (B < 0 || total < 0) return fail(ATTN_ERR_BAD_SHAPE, "negative size (B=%d total=%d)", B, total);
  if (B == 0 || total == 0) return ATTN_OK;
  if (!K || !V || !k_strides || !v_strides) return fail(ATTN_ERR_NULLPTR, "K, V and their strides must not be NULL");
  if ((st = check_table(block_table, max_pages, cu_seqlens, start_lens)) != ATTN_OK) return st;
  if (odd16(K) || odd16(V)) return fail(ATTN_ERR_MISALIGNED, "K and V must be 16-byte aligned");
  for (const int64_t* s : {k_strides, v_strides})
    for (int i = 0; i < 2; ++i)
      if (s[i] < 0 || (s[i] & 7) != 0 || s[i] >= (1ll << 38))
        return fail(ATTN_ERR_BAD_ARG, "stride %lld: must be a multiple of 8 elements (16 bytes) in [0, 2^38)",
                    static_cast<long long>(s[i]));
  unsigned grid;
  if ((st = cache_grid(cache, total, &grid)) != ATTN_OK) return st;
  attn::CacheParams p = cache_params(cache, block_table, max_pages, cu_seqlens, start_lens, B, total);
  p.src_k = static_cast<const __nv_bfloat16*>(K);
  p.src_v = static_cast<const __nv_bfloat16*>(V);
  p.k_st = k_strides[0];
  p.k_sh = k_strides[1];
  p.v_st = v_strides[0];
  p.v_sh = v_strides[1];
  const int groups = cache->d == 128 ? attn::CacheTile<128>::kGroups : attn::CacheTile<64>::kGroups;
  p.step_t = groups / cache->num_heads;
  p.step_h = groups % cache->num_heads;
  int dev;
  uint32_t* status;
  if ((st = cache_device(&dev, &status, &p.page_word)) != ATTN_OK) return st;
  const bool f8 = cache->type == ATTN_CACHE_E4M3;
  const CacheKernel k = cache->d == 128
                            ? (f8 ? attn::attn_cache_write_kernel<128, true> : attn::attn_cache_write_kernel<128, false>)
                            : (f8 ? attn::attn_cache_write_kernel<64, true> : attn::attn_cache_write_kernel<64, false>);
  return launch_cache(k, grid, p, stream);
}

attn_status attn_cache_read(const attn_cache* cache, void* K, void* V, const int32_t* block_table, int max_pages,
                            const int32_t* cu_seqlens, const int32_t* start_lens, int B, int total, void* stream) {
  g_err[0] = '\0';
  attn_status st = check_cache(cache, max_pages);
  if (st != ATTN_OK) return st;
  if (B < 0 || total < 0) return fail(ATTN_ERR_BAD_SHAPE, "negative size (B=%d total=%d)", B, total);
  if (B == 0 || total == 0) return ATTN_OK;
  if (!K || !V) return fail(ATTN_ERR_NULLPTR, "K and V must not be NULL");
  if ((st = check_table(block_table, max_pages, cu_seqlens, start_lens)) != ATTN_OK) return st;
  if (odd16(K) || odd16(V)) return fail(ATTN_ERR_MISALIGNED, "K and V must be 16-byte aligned");
  unsigned grid;
  if ((st = cache_grid(cache, total, &grid)) != ATTN_OK) return st;
  attn::CacheParams p = cache_params(cache, block_table, max_pages, cu_seqlens, start_lens, B, total);
  p.dst_k = static_cast<__nv_bfloat16*>(K);
  p.dst_v = static_cast<__nv_bfloat16*>(V);
  int dev;
  uint32_t* status;
  if ((st = cache_device(&dev, &status, &p.page_word)) != ATTN_OK) return st;
  const bool f8 = cache->type == ATTN_CACHE_E4M3;
  const CacheKernel k = cache->d == 128
                            ? (f8 ? attn::attn_cache_read_kernel<128, true> : attn::attn_cache_read_kernel<128, false>)
                            : (f8 ? attn::attn_cache_read_kernel<64, true> : attn::attn_cache_read_kernel<64, false>);
  return launch_cache(k, grid, p, stream);
}

size_t attn_tree_workspace_bytes(int Hq, int Hkv, int max_seqlen_q, int d) {
  if ((d != 64 && d != 128) || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || max_seqlen_q < 1 ||
      max_seqlen_q > attn::kTreeMaxNodes)
    return 0;
  return use_tile_kernel(Hq / Hkv, max_seqlen_q) ? tree_space(attn::kTileRows, kTileMaxCtas, d).total
                                                 : tree_space(attn::kTreeRows, kTreeMaxCtas, d).total;
}

attn_status attn_fwd_tree(const void* Q, const attn_cache* cache, void* O, float* LSE, const int32_t* block_table,
                          int max_pages, const int32_t* cu_seqlens_q, const int32_t* ctx_lens,
                          const int64_t* tree_mask, int B, int Hq, int max_seqlen_q, int total_q, float scale,
                          void* workspace, size_t workspace_bytes, void* stream) {
  g_err[0] = '\0';
  attn_status st = check_cache(cache, max_pages);
  if (st != ATTN_OK) return st;
  if (B < 0 || Hq < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_q > attn::kTreeMaxNodes)
    return fail(ATTN_ERR_BAD_SHAPE, "B=%d Hq=%d total_q=%d max_seqlen_q=%d; max_seqlen_q must be in [0, %d]", B, Hq,
                total_q, max_seqlen_q, attn::kTreeMaxNodes);
  if (Hq > kMaxHeads) return fail(ATTN_ERR_BAD_SHAPE, "Hq=%d; at most %d", Hq, kMaxHeads);
  if (Hq % cache->num_heads != 0)
    return fail(ATTN_ERR_BAD_SHAPE, "Hq=%d must be a multiple of the cache's %d heads", Hq, cache->num_heads);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(ATTN_ERR_BAD_ARG, "scale must be finite and > 0");
  if (B == 0 || Hq == 0 || total_q == 0 || max_seqlen_q == 0) return ATTN_OK;
  if (!Q || !O || !LSE) return fail(ATTN_ERR_NULLPTR, "Q, O and LSE must not be NULL");
  if ((st = check_table(block_table, max_pages, cu_seqlens_q, ctx_lens)) != ATTN_OK) return st;
  if (odd16(Q) || odd16(O)) return fail(ATTN_ERR_MISALIGNED, "Q and O must be 16-byte aligned");
  if (odd_to(LSE, 4) || odd_to(tree_mask, 8))
    return fail(ATTN_ERR_MISALIGNED, "LSE must be 4-byte aligned, tree_mask 8-byte aligned");
  const size_t need = attn_tree_workspace_bytes(Hq, cache->num_heads, max_seqlen_q, cache->d);
  if (!workspace) return fail(ATTN_ERR_NULLPTR, "workspace must not be NULL (%zu B)", need);
  if (odd16(workspace)) return fail(ATTN_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  if (workspace_bytes < need)
    return fail(ATTN_ERR_BAD_ARG, "workspace of %zu B is smaller than the %zu B needed", workspace_bytes, need);
  attn::TreeParams p = {};
  int dev;
  if ((st = cache_device(&dev, &p.status, &p.page_word)) != ATTN_OK) return st;
  p.q = static_cast<const __nv_bfloat16*>(Q);
  p.o = static_cast<__nv_bfloat16*>(O);
  p.lse = LSE;
  p.table = block_table;
  p.cu = cu_seqlens_q;
  p.ctx = ctx_lens;
  p.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  p.v = cache->v;
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = cache->num_heads;
  p.G = Hq / cache->num_heads;
  p.max_q = max_seqlen_q;
  p.total_q = total_q;
  p.num_pages = cache->num_pages;
  p.page = cache->page_size;
  p.max_pages = max_pages;
  p.cap = max_pages * cache->page_size;
  p.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.timeout_ns = wait_limit_ns();
  p.fault_block = fault_block();
  const bool f8 = cache->type == ATTN_CACHE_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->d == 128)
    return f8 ? launch_tree_any<128, true>(cache, p, workspace, s, dev)
              : launch_tree_any<128, false>(cache, p, workspace, s, dev);
  return f8 ? launch_tree_any<64, true>(cache, p, workspace, s, dev)
            : launch_tree_any<64, false>(cache, p, workspace, s, dev);
}

attn_status attn_cache_check(void* stream) {
  g_err[0] = '\0';
  attn_status st = attn_status_sync(stream);
  if (st != ATTN_OK) return st;
  int dev;
  uint32_t* word = nullptr;
  if ((st = get_device(&dev)) != ATTN_OK) return st;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    word = g_page_addr[dev];
  }
  if (!word) return ATTN_OK;  // no cache call has run on this device
  uint32_t v = 0;
  if (cudaMemcpy(&v, word, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
    return fail(ATTN_ERR_LAUNCH, "page word read failed");
  if (!v) return ATTN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(word, 0, sizeof(v), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return fail(ATTN_ERR_LAUNCH, "page word clear failed");
  return fail(ATTN_ERR_BAD_PAGE, "a position had no page, or its block_table entry was outside the cache");
}

}  // extern "C"

// The library's one translation unit: the forward's entry points, then those of the paged cache.
#include "attn_api.cu"
#include "attn_cache_api.cuh"

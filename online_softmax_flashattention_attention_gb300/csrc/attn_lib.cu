// The library's one translation unit: the forward's entry points, those of the paged cache, and those
// for prompts and caches of bounded length.
#include "attn_api.cu"
#include "attn_cache_api.cuh"
#include "attn_prompt_api.cuh"

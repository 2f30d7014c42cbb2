// attn_lib.cu -- the library's one translation unit: the attention of whole
// tensors and packed batches, and the paged cache, which shares its device
// state and status word.
#include "attn_api.cu"

#include "attn_cache_api.cuh"

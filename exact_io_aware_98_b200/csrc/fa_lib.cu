// fa_lib.cu -- the translation unit of libfa: the attention entry points (fa_api.cu) and, on the
// same helpers, those of rotary positions and of the paged cache (fa_paged_api.cuh).
#include "fa_api.cu"

#include "fa_paged.cuh"
#include "fa_paged_cache.cuh"
#include "fa_paged_chunk_sm100.cuh"
#include "fa_paged_decode_sm100.cuh"
#include "fa_paged_simt.cuh"
#include "fa_rope.cuh"

#include "fa_paged_api.cuh"

// Instantiations of the tensor-core attention (prefill_impl.cuh) for chunks of new tokens over a paged cache: two row tiles sharing their keys.
#include "prefill_impl.cuh"

namespace pkv_prefill {
PKV_ATTN_INSTANTIATE(MODE_CHUNK, false)
PKV_ATTN_INSTANTIATE(MODE_CHUNK, true)
} // namespace pkv_prefill

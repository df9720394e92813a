// Instantiations of the tensor-core attention (prefill_impl.cuh) for chunks of few rows over a paged cache: one row tile, two streams of keys.
#include "prefill_impl.cuh"

namespace pkv_prefill {
PKV_ATTN_INSTANTIATE(MODE_STREAM, false)
PKV_ATTN_INSTANTIATE(MODE_STREAM, true)
} // namespace pkv_prefill

// Instantiations of the two-pipeline attention of chunks (chunk_stream.cuh): 16-bit caches, at most 128 rows.
#include "chunk_stream.cuh"

namespace pkv_prefill {
PKV_STREAM_INSTANTIATE(false, false)
} // namespace pkv_prefill

// Instantiations of the two-pipeline attention of chunks (chunk_stream.cuh): E4M3 caches, at most 128 rows.
#include "chunk_stream.cuh"

namespace pkv_prefill {
PKV_STREAM_INSTANTIATE(true, false)
} // namespace pkv_prefill

// Decode kernels with a sliding window and sinks: model dtype PKV_BF16, KV dtype PKV_BF16.
#include "decode_impl.cuh"

cudaError_t pkv_decode_window_bf16(const pkv_decode::Args &a, int D, int G, int grid, size_t smem, cudaStream_t st,
                                 bool merge) {
    return pkv_decode::dispatch<PKV_BF16, PKV_BF16, true>(a, D, G, grid, smem, st, merge);
}

int pkv_decode_window_occupancy_bf16(int D, int G, size_t smem) {
    return pkv_decode::occupancy_dispatch<PKV_BF16, PKV_BF16, true>(D, G, smem);
}

// Decode kernels with a sliding window and sinks: model dtype PKV_F16, KV dtype PKV_F16.
#include "decode_impl.cuh"

cudaError_t pkv_decode_window_f16(const pkv_decode::Args &a, int D, int G, int grid, size_t smem, cudaStream_t st,
                                 bool merge) {
    return pkv_decode::dispatch<PKV_F16, PKV_F16, true>(a, D, G, grid, smem, st, merge);
}

int pkv_decode_window_occupancy_f16(int D, int G, size_t smem) {
    return pkv_decode::occupancy_dispatch<PKV_F16, PKV_F16, true>(D, G, smem);
}

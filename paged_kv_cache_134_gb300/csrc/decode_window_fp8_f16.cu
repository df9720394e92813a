// Decode kernels with a sliding window and sinks: model dtype PKV_F16, KV dtype PKV_FP8_E4M3.
#include "decode_impl.cuh"

cudaError_t pkv_decode_window_fp8_f16(const pkv_decode::Args &a, int D, int G, int grid, size_t smem, cudaStream_t st,
                                 bool merge) {
    return pkv_decode::dispatch<PKV_F16, PKV_FP8_E4M3, true>(a, D, G, grid, smem, st, merge);
}

int pkv_decode_window_occupancy_fp8_f16(int D, int G, size_t smem) {
    return pkv_decode::occupancy_dispatch<PKV_F16, PKV_FP8_E4M3, true>(D, G, smem);
}

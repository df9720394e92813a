#include "decode_short.cuh"

cudaError_t pkv_short_fp8(const pkv_mma::Args &a, int mt, int D, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::dispatch_short<PKV_FP8_E4M3, PKV_F16>(a, D, st)
                         : pkv_mma::dispatch_short<PKV_FP8_E4M3, PKV_BF16>(a, D, st);
}

#include "decode_short.cuh"

cudaError_t pkv_short_16bit(const pkv_mma::Args &a, int mt, int D, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::dispatch_short<PKV_F16, PKV_F16>(a, D, st)
                         : pkv_mma::dispatch_short<PKV_BF16, PKV_BF16>(a, D, st);
}

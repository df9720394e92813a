#include "decode_mma.cuh"

cudaError_t pkv_mma_fp8_mass(const pkv_mma::Args &a, int mt, int D, int sms, bool merge, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::dispatch_mass<PKV_FP8_E4M3, PKV_F16>(a, D, sms, merge, st)
                         : pkv_mma::dispatch_mass<PKV_FP8_E4M3, PKV_BF16>(a, D, sms, merge, st);
}

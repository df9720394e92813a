#include "decode_mma.cuh"

cudaError_t pkv_mma_16bit_window(const pkv_mma::Args &a, int mt, int D, int sms, bool merge, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::dispatch_mass<PKV_F16, PKV_F16, false, true>(a, D, sms, merge, st)
                         : pkv_mma::dispatch_mass<PKV_BF16, PKV_BF16, false, true>(a, D, sms, merge, st);
}

#include "decode_int4.cuh"

cudaError_t pkv_mma_int4_mass(const pkv_mma::Args &a, int mt, int D, int sms, bool merge, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::dispatch_int4<PKV_F16, true>(a, D, sms, merge, st)
                         : pkv_mma::dispatch_int4<PKV_BF16, true>(a, D, sms, merge, st);
}

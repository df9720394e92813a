#include "decode_int4.cuh"

cudaError_t pkv_mma_int4(const pkv_mma::Args &a, int mt, int D, int sms, bool merge, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::dispatch_int4<PKV_F16, false>(a, D, sms, merge, st)
                         : pkv_mma::dispatch_int4<PKV_BF16, false>(a, D, sms, merge, st);
}

#include "chunk_few.cuh"

cudaError_t pkv_few_e4m3(const pkv_mma::FewArgs &a, int mt, int D, int sms, bool merge, cudaStream_t st) {
    return mt == PKV_F16 ? pkv_mma::launch_few<PKV_FP8_E4M3, PKV_F16>(a, D, sms, merge, st)
                         : pkv_mma::launch_few<PKV_FP8_E4M3, PKV_BF16>(a, D, sms, merge, st);
}

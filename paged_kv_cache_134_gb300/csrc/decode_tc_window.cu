// Instantiations of the tensor-core decode (decode_tc.cuh) with a sliding window and sinks, 16-bit caches.
#include "decode_tc.cuh"

cudaError_t pkv_decode_tc_window(const CUtensorMap &tkv, const CUtensorMap &tq, const pkv_decode::Args &a, int G, int mt,
                                 int grid, size_t smem, cudaStream_t st) {
    using namespace pkv_decode_tc;
#define PKV_TC_CASE(GG)                                                                                                \
    if (G == GG) {                                                                                                     \
        return mt == PKV_BF16 ? launch<GG, PKV_BF16, PKV_BF16, true>(tkv, tq, a, grid, smem, st)                       \
                              : launch<GG, PKV_F16, PKV_F16, true>(tkv, tq, a, grid, smem, st);                        \
    }
    PKV_TC_CASE(2)
    PKV_TC_CASE(4)
    PKV_TC_CASE(8)
#undef PKV_TC_CASE
    return cudaErrorInvalidValue;
}

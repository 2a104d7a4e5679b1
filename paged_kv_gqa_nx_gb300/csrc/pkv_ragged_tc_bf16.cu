// pkv_ragged_tc_bf16.cu -- the instances for bf16 rows of pkv_ragged_tc.h.
#include "pkv_ragged_tc.h"

namespace pkv {

cudaError_t launch_ragged_tc_bf16(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches,
                             cudaStream_t s) {
    return tc_t<bf16>(a, runs, n, first, n_stretches, s);
}

cudaError_t launch_ragged_tc(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches,
                             cudaStream_t s) {
    if (n <= 0 || n > kRaggedLarge || a.hd > kMaxHeadDim || !ragged_tc_takes(a)) return cudaErrorInvalidValue;
    return a.type == Elem::bf16 ? launch_ragged_tc_bf16(a, runs, n, first, n_stretches, s) : launch_ragged_tc_f16(a, runs, n, first, n_stretches, s);
}

}  // namespace pkv

// pkv_ragged_tc_f16.cu -- the instances for f16 rows of pkv_ragged_tc.h.
#include "pkv_ragged_tc.h"

namespace pkv {

cudaError_t launch_ragged_tc_f16(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches,
                             cudaStream_t s) {
    return tc_t<f16>(a, runs, n, first, n_stretches, s);
}

}  // namespace pkv

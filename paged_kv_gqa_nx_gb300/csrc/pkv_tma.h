// pkv_tma.h -- tensor maps of TMA loads: the driver's encoder, found at run time
// (the library links no driver), and the maps of an 8-bit pool.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace pkv {

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
cudaError_t encode_tiled(EncodeTiled *out);  // pkv_packed.cu

// An 8-bit pool's K and V as [block, layer][row of the block][kv head][hd], in
// boxes of sixteen rows of one head.
struct Q8Maps {
    CUtensorMap k, v;
    int n_layers, layer;
};

}  // namespace pkv

// pkv_half.h -- bf16 and f16 rows on the tensor cores (pkv_packed.cu, the
// ragged kernels): roundings, pairs in a register, warp-level MMAs and the
// loads of their operands.
#pragma once

#include "pkv_elem.h"

#include <cuda_fp16.h>
#include <type_traits>

namespace pkv {

using f16 = __half;

__device__ __forceinline__ void narrow(bf16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void narrow(f16 *p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ uint32_t pack2(bf16, float lo, float hi) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}
__device__ __forceinline__ uint32_t pack2(f16, float lo, float hi) {
    const __half2 t = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&t);
}
__device__ __forceinline__ float half_of(bf16, uint32_t w, int i) {
    return __uint_as_float(i ? w & 0xffff0000u : w << 16);
}
__device__ __forceinline__ float half_of(f16, uint32_t w, int i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return i ? f.y : f.x;
}
// the element's bits are an infinity or a NaN
template <class T>
__device__ __forceinline__ bool not_finite(uint32_t b16) {
    constexpr uint32_t e = std::is_same<T, bf16>::value ? 0x7f80u : 0x7c00u;
    return (b16 & e) == e;
}

template <class T>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, bf16>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kTrans>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *p) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    if constexpr (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
}

}  // namespace pkv

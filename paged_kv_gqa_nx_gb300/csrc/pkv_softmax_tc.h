// pkv_softmax_tc.h -- helpers of the tensor-core kernels whose softmax threads
// own a row of 128 scores (pkv_packed.cu, pkv_prefill_q8.cu): bounded waits, TMEM
// loads that stay in flight, packed f32 arithmetic, the issuing lane.
#pragma once

#include "pkv_tcgen05.h"

namespace pkv {
namespace tc {

// Bounded wait of the calling thread for the phase of the given parity: the
// clock is not read before the wait has gone on for a while (that read is
// slower than a whole uncontended wait).
__device__ __forceinline__ bool wait_phase(uint32_t mbar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t it = 0; it < (1u << 26); ++it) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(done)
            : "r"(mbar), "r"(parity)
            : "memory");
        if (done) return true;
        if ((it & 255u) == 255u) {
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > 1000000000ull) return false;
        }
    }
    return false;
}
// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool test_phase(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(mbar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ float ex2(float x) {  // 2^x to about 2^-22 relative; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// Columns x0 .. x0 + 31 of this thread's lane, issued without a wait; the
// registers belong to the load until tmem_ld_done has passed over them.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tie32(uint32_t *r) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
template <int N>
__device__ __forceinline__ void tmem_ld_done(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 32) tie32(r + i);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// pairs of f32 in one instruction: a * b + c, and a + b
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(f.x), "=f"(f.y) : "l"(x));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// The leading part of a row's running sums, out of the tensor core's reach: it
// rounds toward zero at every addition to a sum, so a long one loses steadily.
// Byte k of a word, h + 128, as h (2^23 + u is the float of bits 0x4b000000 | u):
__device__ __forceinline__ float aside(uint32_t w, int k) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | k)) - (8388608.f + 128.f);
}
// x (f32 bits; joined by what is set aside already, where there is some) becomes
// h * unit + x: h in hold's bytes, unit a power of two (returned) that makes the
// row's largest 32 to 64, x what that leaves, exactly, as a sum has 24 bits.  Only
// the first `width` of x count.
template <int N>
__device__ __forceinline__ float set_aside(uint32_t (&x)[N], uint32_t (&hold)[N / 4], float unit, bool join, int width) {
    if (join) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __float_as_uint(fmaf(aside(hold[i / 4], i & 3), unit, __uint_as_float(x[i])));
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < 16 || i < width) top = fmaxf(top, fabsf(__uint_as_float(x[i])));
    const int e = max(-100, min(100, static_cast<int>(__float_as_uint(top) >> 23) - 127 - 5));
    const float to = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    constexpr float kMagic = 12582912.f + 128.f;  // 1.5 * 2^23: a sum's low byte is the integer + 128
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        uint32_t t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float y = __uint_as_float(x[i + k]), r = fmaf(y, inv, kMagic);
            t[k] = __float_as_uint(r);
            x[i + k] = __float_as_uint(fmaf(kMagic - r, to, y));
        }
        hold[i / 4] = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
    }
    return to;
}
// One lane of a converged warp, chosen in a way that leaves the operands of the
// instructions it issues in uniform registers (a test of the lane number does
// not: eight MMAs then took 440 clocks to issue instead of 270).
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}\n" : "=r"(p));
    return p != 0;
}

}  // namespace tc
}  // namespace pkv

// pkv_q8.cu -- attention over an 8-bit pool with a scale per (block, layer, kv
// head): the split-K decode kernels and the split pass that makes the operand
// images of the tensor-core launches.
//
// A stored element u stands for (u - 128) * s, s a power of two, so every value
// is exact in f32 (and in f16 or bf16, which hold integers up to 2^11 and 2^8):
// the only rounding is the one made when the row was written.
//
//   scores   s_j = ks_j * sum_d q_d (u_jd - 128)      q pre-scaled by scale * log2(e)
//   output   o_d = sum_j 2^(s_j - m) vs_j (u_jd - 128) / sum_j 2^(s_j - m)
#include "pkv_elem.h"
#include "pkv_internal.h"
#include "pkv_rows.h"

#include <cuda_fp16.h>

namespace pkv {
namespace {

__device__ __forceinline__ float pow2f(int e) {  // 2^e, e in [-126, 127]
    return __int_as_float((e + 127) << 23);
}

// The block of position pos, or -1 (and the error flag) where the page index
// or the block id is out of range.
__device__ __forceinline__ int block_of(const PagedAddr &a, int slot, int pos, int32_t *err) {
    const int bi = a.bs_shift >= 0 ? (pos >> a.bs_shift) : (pos / a.bs);
    int blk = -1;
    if (bi < a.max_blocks) blk = __ldg(a.pt + static_cast<size_t>(slot) * a.max_blocks + bi);
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.n_blocks)) {
        flag_error(err, 1);
        return -1;
    }
    return blk;
}
__device__ __forceinline__ int block_off(const PagedAddr &a, int pos) {
    return a.bs_shift >= 0 ? (pos & (a.bs - 1)) : (pos % a.bs);
}

// --------------------------------------------------------- generic decode ----
//
// Any head width up to 256 and any group: CTA = 4 warps = one (unit, kv head,
// chunk of up to 16 query heads); warp w takes the unit's keys w, w + 4, ...,
// the lanes hold the dims d = lane, lane + 32, ....  Bound by the instructions
// it issues (a shuffle sum per key and head).

constexpr int kGW = 4, kGHeads = 16, kGDims = kMaxHeadDim / 32;

__global__ void __launch_bounds__(128) decode_q8_generic_kernel(AttnArgs a, Q8Addr q, int hpc) {
    extern __shared__ __align__(16) float sm[];
    const int n_chunks = (a.group + hpc - 1) / hpc;
    int b = blockIdx.x;
    const int chunk = b % n_chunks;
    b /= n_chunks;
    const int kvh = b % a.n_kv, ui = b / a.n_kv;
    const UnitDesc u = a.units[ui];
    const RowDesc rd = a.rows[u.row];
    const UnitRange ur = unit_range(u, rd, a.causal, a.split_keys);
    const int hd = a.hd, h0 = kvh * a.group + chunk * hpc, nh = min(hpc, a.group - chunk * hpc);
    float *qs = sm;                       // [hpc][hd]
    float *accs = qs + hpc * hd;          // [kGW][hpc][hd]
    float *ms = accs + kGW * hpc * hd;    // [kGW][hpc]
    float *ls = ms + kGW * hpc;           // [kGW][hpc]
    const float *qrow = a.Q + static_cast<size_t>(rd.q_row0 + u.qi) * (a.n_heads * hd) + static_cast<size_t>(h0) * hd;
    for (int t = threadIdx.x; t < nh * hd; t += blockDim.x) qs[t] = qrow[t] * a.scale_log2;
    for (int t = threadIdx.x; t < kGW * hpc * hd; t += blockDim.x) accs[t] = 0.f;
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m[kGHeads], l[kGHeads];
#pragma unroll
    for (int g = 0; g < kGHeads; ++g) m[g] = -INFINITY, l[g] = 0.f;
    float *acc = accs + warp * hpc * hd;
    for (int j = ur.kbeg + warp; j < ur.kend; j += kGW) {
        const int blk = block_of(q.a, rd.slot, j, a.err);
        if (blk < 0) continue;
        const size_t o = static_cast<size_t>(blk) * q.a.block_stride + q.a.layer_off +
                         static_cast<size_t>(block_off(q.a, j)) * q.a.kv_dim + static_cast<size_t>(kvh) * hd;
        const uint8_t *kr = static_cast<const uint8_t *>(q.a.k) + o, *vr = static_cast<const uint8_t *>(q.a.v) + o;
        const float ks = __ldg(q.ks + blk * q.scale_stride + kvh), vs = __ldg(q.vs + blk * q.scale_stride + kvh);
        float kx[kGDims], vx[kGDims];
#pragma unroll
        for (int i = 0; i < kGDims; ++i) {
            const int d = lane + 32 * i;
            kx[i] = d < hd ? static_cast<float>(static_cast<int>(kr[d]) - 128) : 0.f;
            vx[i] = d < hd ? static_cast<float>(static_cast<int>(vr[d]) - 128) : 0.f;
        }
#pragma unroll
        for (int g = 0; g < kGHeads; ++g) {
            if (g < nh) {
                float part = 0.f;
#pragma unroll
                for (int i = 0; i < kGDims; ++i)
                    if (lane + 32 * i < hd) part = fmaf(qs[g * hd + lane + 32 * i], kx[i], part);
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) part += __shfl_xor_sync(kFull, part, x);
                part *= ks;
                const float mn = fmaxf(m[g], part);
                const float alpha = mn == m[g] ? 1.f : exp2f(m[g] - mn);
                const float p = exp2f(part - mn);
                l[g] = fmaf(l[g], alpha, p);
                m[g] = mn;
                const float pv = p * vs;
#pragma unroll
                for (int i = 0; i < kGDims; ++i) {
                    const int d = lane + 32 * i;
                    if (d < hd) acc[g * hd + d] = fmaf(pv, vx[i], acc[g * hd + d] * alpha);
                }
            }
        }
    }
    if (lane == 0) {
#pragma unroll
        for (int g = 0; g < kGHeads; ++g)
            if (g < nh) {
                ms[warp * hpc + g] = m[g];
                ls[warp * hpc + g] = l[g];
            }
    }
    __syncthreads();

    for (int t = threadIdx.x; t < nh * hd; t += blockDim.x) {
        const int g = t / hd, d = t - g * hd;
        float M = -INFINITY;
        for (int w = 0; w < kGW; ++w) M = fmaxf(M, ms[w * hpc + g]);
        float num = 0.f, den = 0.f;
        for (int w = 0; w < kGW; ++w) {
            const float mw = ms[w * hpc + g];
            const float wt = mw == -INFINITY ? 0.f : exp2f(mw - M);
            if (ls[w * hpc + g] != 0.f) {  // a warp without keys has an empty state
                num = fmaf(wt, accs[(w * hpc + g) * hd + d], num);
                den = fmaf(wt, ls[w * hpc + g], den);
            }
        }
        const int h = h0 + g;
        if (u.item < 0) {
            a.out[static_cast<size_t>(rd.q_row0 + u.qi) * (a.n_heads * hd) + static_cast<size_t>(h) * hd + d] = num / den;
        } else {
            const size_t ph = static_cast<size_t>(a.merges[u.item].part0 + u.split) * a.n_heads + h;
            a.pacc[ph * hd + d] = num;
            if (d == 0) {
                a.pm[ph] = M;
                a.pl[ph] = den;
            }
        }
    }
}

cudaError_t launch_generic(const AttnArgs &a, const Q8Addr &q, cudaStream_t s) {
    const int hpc = a.group < kGHeads ? a.group : kGHeads;
    auto bytes = [](int n, int hd) { return (static_cast<size_t>(n) * hd * (1 + kGW) + 2 * kGW * n) * sizeof(float); };
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(decode_q8_generic_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(bytes(kGHeads, kMaxHeadDim)));
    });
    if (ce != cudaSuccess) return ce;
    const int n_chunks = (a.group + hpc - 1) / hpc;
    const long long grid = static_cast<long long>(a.n_units) * a.n_kv * n_chunks;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    decode_q8_generic_kernel<<<static_cast<unsigned>(grid), 128, bytes(hpc, a.hd), s>>>(a, q, hpc);
    return cudaGetLastError();
}

// -------------------------------------------------------------- split pass ----
//
// Operand images for the tensor-core launches (the layout of kImageBytes): one
// CTA per (64-key tile, kv head, K or V).  The tile's values go to shared
// memory as f32 (zero past the row's keys), the block finds their largest
// magnitude, and each value times the tile's power of two is an f16 value --
// seven bits, unless it lies more than 2^28 below the tile's largest -- so
// piece 1 is left out, as on the other narrow pools.

constexpr int kHDI = 128;

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__global__ void __launch_bounds__(256) split_q8_kernel(SplitArgs p, Q8Addr q) {
    extern __shared__ __align__(16) float raw[];
    __shared__ float wmax[8];
    const int part = blockIdx.x & 1;  // 0: K, 1: V
    const int ik = blockIdx.x >> 1, it = ik / p.n_kv, kvh = ik - it * p.n_kv;
    const SplitItem t = p.items[it];
    const RowDesc rd = p.rows[t.row];
    const int total_k = rd.past_len + rd.n_q, key0 = t.kt * kKeyTile;
    const int ld = part ? kHDI + 1 : kHDI;  // V is read transposed: an odd pitch has no bank conflicts
    const uint8_t *base = static_cast<const uint8_t *>(part ? q.a.v : q.a.k);
    const float *scales = part ? q.vs : q.ks;
    float mx = 0.f;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {  // 64 keys x 8 chunks of 16 elements
        const int i = threadIdx.x + 256 * pass, key = i >> 3, ch = i & 7, pos = key0 + key;
        uint4 u = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        float sc = 0.f;
        if (pos < total_k) {
            const int blk = block_of(q.a, rd.slot, pos, p.err);
            if (blk >= 0) {
                u = __ldg(reinterpret_cast<const uint4 *>(base + static_cast<size_t>(blk) * q.a.block_stride +
                                                          q.a.layer_off +
                                                          static_cast<size_t>(block_off(q.a, pos)) * q.a.kv_dim +
                                                          static_cast<size_t>(kvh) * kHDI + 16 * ch));
                sc = __ldg(scales + blk * q.scale_stride + kvh);
            }
        }
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float *d = raw + key * ld + 16 * ch;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float x = static_cast<float>(static_cast<int>(w[j >> 2] >> (8 * (j & 3)) & 255u) - 128) * sc;
            mx = fmaxf(mx, fabsf(x));
            d[j] = x;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = mx;
    __syncthreads();
    mx = wmax[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) mx = fmaxf(mx, wmax[w]);
    // the power of two that brings the largest magnitude into [2^14, 2^15)
    const int ex = max(-113, min(126, 14 - (static_cast<int>((__float_as_uint(mx) >> 23) & 255u) - 127)));
    const float sc = pow2f(ex);
    unsigned char *img = p.img + (static_cast<size_t>(t.slot) * p.n_kv + kvh) * kImageBytes;
    unsigned char *out = img + static_cast<size_t>(part) * 2 * kImagePlane;
    for (int c = threadIdx.x; c < static_cast<int>(kImagePlane / 16); c += blockDim.x) {
        float x[8];
        if (part == 0) {  // K: k-block c >> 9 (64 dims), key (c >> 3) & 63, swizzled chunk c & 7
            const int r = (c >> 3) & 63;
            const float *src = raw + r * kHDI + (c >> 9) * 64 + ((c & 7) ^ (r & 7)) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = src[j];
        } else {          // V^T: dim c >> 3, swizzled chunk c & 7 (8 keys)
            const int d = c >> 3, k0 = ((c & 7) ^ (d & 7)) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = raw[(k0 + j) * (kHDI + 1) + d];
        }
        *reinterpret_cast<uint4 *>(out + c * 16) =
            make_uint4(f16x2(x[0] * sc, x[1] * sc), f16x2(x[2] * sc, x[3] * sc), f16x2(x[4] * sc, x[5] * sc),
                       f16x2(x[6] * sc, x[7] * sc));
    }
    if (threadIdx.x == 0) reinterpret_cast<int32_t *>(img + kImageExpOff)[part] = ex;
}

}  // namespace

int q8_query_block(int, int) { return 1; }

cudaError_t launch_decode_q8(const AttnArgs &a, const Q8Addr &q, cudaStream_t s) { return launch_generic(a, q, s); }

cudaError_t launch_split_q8(const SplitArgs &a, const Q8Addr &q, cudaStream_t s) {
    constexpr size_t smem = static_cast<size_t>(kKeyTile) * (kHDI + 1) * sizeof(float);
    if (q.hd != kHDI) return cudaErrorInvalidValue;
    const long long grid = static_cast<long long>(a.n_items) * a.n_kv * 2;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    split_q8_kernel<<<static_cast<unsigned>(grid), 256, smem, s>>>(a, q);
    return cudaGetLastError();
}

}  // namespace pkv

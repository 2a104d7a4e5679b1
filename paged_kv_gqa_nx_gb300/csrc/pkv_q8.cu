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
#include "pkv_tcgen05.h"
#include "pkv_tma.h"

#include <algorithm>
#include <cuda_fp16.h>
#include <type_traits>
#include <utility>

namespace pkv {
namespace {

__device__ __forceinline__ float pow2f(int e) {  // 2^e, e in [-126, 127]
    return __int_as_float((e + 127) << 23);
}

// The block of position pos, or -1 (and the error flag) where the page index
// or the block id is out of range.  (Page table and scales are read through L2:
// a decode launch starts while the append before it still writes them, so they
// are not constant for its life, and a line of the SM's L1 may be older.)
__device__ __forceinline__ int block_of(const PagedAddr &a, int slot, int pos, int32_t *err) {
    const int bi = a.bs_shift >= 0 ? (pos >> a.bs_shift) : (pos / a.bs);
    int blk = -1;
    if (bi < a.max_blocks) blk = __ldcg(a.pt + static_cast<size_t>(slot) * a.max_blocks + bi);
    if (static_cast<unsigned>(blk) >= static_cast<unsigned>(a.n_blocks)) {
        flag_error(err, 1);
        return -1;
    }
    return blk;
}
__device__ __forceinline__ int block_off(const PagedAddr &a, int pos) {
    return a.bs_shift >= 0 ? (pos & (a.bs - 1)) : (pos % a.bs);
}

// ------------------------------------------------------------------ units ----

template <class B>
__device__ __forceinline__ Q8Unit unit_of(const Q8Args &a, const B &blob, int i) {
    const Q8Part p = blob_at(a.units, blob)[i];
    return Q8Unit{blob_at(a.blocks, blob)[p.block], p.kbeg, p.kend, p.rec};
}
// Waits for the end of the launch that this one was allowed to overlap.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// Whether this CTA's unit is the last of its block to finish; then every record
// of the block can be read (through L2: other SMs wrote them).
__device__ __forceinline__ bool last_of_block(const Q8Args &a, const Q8Unit &u, int part) {
    __shared__ bool last;
    __syncthreads();  // this CTA's records are written
    if (threadIdx.x == 0) {
        __threadfence();
        uint32_t *c = a.cnt + u.cnt + part;
        last = atomicAdd(c, 1u) == static_cast<uint32_t>(u.n_dec) - 1u;
        if (last) *c = 0;
        __threadfence();
    }
    __syncthreads();
    return last;
}
// One (query, head) of a block by one warp: out = sum_s 2^(m_s - M) acc_s / sum_s
// 2^(m_s - M) l_s over its records in ascending order.
__device__ __forceinline__ void join_records(const Q8Args &a, const Q8Unit &u, int qi, int h, int lane) {
    const int hd = a.hd;
    auto rec = [&](int s) { return static_cast<size_t>(u.part0 + qi * u.n_rec + s) * a.n_heads + h; };
    float M = -INFINITY, den = 0.f;
    for (int s = 0; s < u.n_rec; ++s) M = fmaxf(M, __ldcg(a.pm + rec(s)));
    for (int s = 0; s < u.n_rec; ++s) den = fmaf(exp2f(__ldcg(a.pm + rec(s)) - M), __ldcg(a.pl + rec(s)), den);
    float *o = a.out + static_cast<size_t>(u.q_row + qi) * (a.n_heads * hd) + static_cast<size_t>(h) * hd;
    for (int d = lane; d < hd; d += 32) {
        float num = 0.f;
#pragma unroll 4
        for (int s = 0; s < u.n_rec; ++s) num = fmaf(exp2f(__ldcg(a.pm + rec(s)) - M), __ldcg(a.pacc + rec(s) * hd + d), num);
        o[d] = num / den;
    }
}

// --------------------------------------------------------- generic decode ----
//
// Any head width up to 256 and any group: CTA = 4 warps = one (unit, kv head,
// chunk of up to 16 query heads); warp w takes the unit's keys w, w + 4, ...,
// the lanes hold the dims d = lane, lane + 32, ....  Bound by the instructions
// it issues (a shuffle sum per key and head): 64 sequences of 512 .. 4,096 with
// 32 heads of 160 over 8 in 1,320 us (0.2 TB/s).

constexpr int kGW = 4, kGHeads = 16, kGDims = kMaxHeadDim / 32;

template <class B>
__global__ void __launch_bounds__(128) decode_q8_generic_kernel(Q8Args a, Q8Addr q, int hpc,
                                                                const __grid_constant__ B blob) {
    extern __shared__ __align__(16) float sm[];
    const int n_chunks = (a.group + hpc - 1) / hpc;
    int b = blockIdx.x;
    const int chunk = b % n_chunks;
    b /= n_chunks;
    const int kvh = b % a.n_kv, ui = b / a.n_kv;
    const Q8Unit u = unit_of(a, blob, ui);  // one query
    const int hd = a.hd, h0 = kvh * a.group + chunk * hpc, nh = min(hpc, a.group - chunk * hpc);
    float *qs = sm;                       // [hpc][hd]
    float *accs = qs + hpc * hd;          // [kGW][hpc][hd]
    float *ms = accs + kGW * hpc * hd;    // [kGW][hpc]
    float *ls = ms + kGW * hpc;           // [kGW][hpc]
    const float *qrow = a.Q + static_cast<size_t>(u.q_row) * (a.n_heads * hd) + static_cast<size_t>(h0) * hd;
    for (int t = threadIdx.x; t < nh * hd; t += blockDim.x) qs[t] = qrow[t] * a.scale_log2;
    for (int t = threadIdx.x; t < kGW * hpc * hd; t += blockDim.x) accs[t] = 0.f;
    __syncthreads();
    wait_previous();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float m[kGHeads], l[kGHeads];
#pragma unroll
    for (int g = 0; g < kGHeads; ++g) m[g] = -INFINITY, l[g] = 0.f;
    float *acc = accs + warp * hpc * hd;
    for (int j = u.kbeg + warp; j < u.kend; j += kGW) {
        const int blk = block_of(q.a, u.slot, j, a.err);
        if (blk < 0) continue;
        const size_t o = static_cast<size_t>(blk) * q.a.block_stride + q.a.layer_off +
                         static_cast<size_t>(block_off(q.a, j)) * q.a.kv_dim + static_cast<size_t>(kvh) * hd;
        const uint8_t *kr = static_cast<const uint8_t *>(q.a.k) + o, *vr = static_cast<const uint8_t *>(q.a.v) + o;
        const float ks = __ldcg(q.ks + blk * q.scale_stride + kvh), vs = __ldcg(q.vs + blk * q.scale_stride + kvh);
        float kx[kGDims], vx[kGDims];
#pragma unroll
        for (int i = 0; i < kGDims; ++i) {
            const int d = lane + 32 * i;
            kx[i] = d < hd ? static_cast<float>(static_cast<int>(__ldcg(kr + d)) - 128) : 0.f;
            vx[i] = d < hd ? static_cast<float>(static_cast<int>(__ldcg(vr + d)) - 128) : 0.f;
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
        if (u.part0 < 0) {
            a.out[static_cast<size_t>(u.q_row) * (a.n_heads * hd) + static_cast<size_t>(h) * hd + d] = num / den;
        } else {
            const size_t ph = static_cast<size_t>(u.part0 + u.rec) * a.n_heads + h;
            a.pacc[ph * hd + d] = num;
            if (d == 0) {
                a.pm[ph] = M;
                a.pl[ph] = den;
            }
        }
    }
    if (u.part0 >= 0 && last_of_block(a, u, kvh * n_chunks + chunk))
        for (int g = warp; g < nh; g += kGW) join_records(a, u, 0, h0 + g, lane);
}

// A launch that may start while the one before it on the stream still runs.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

template <class B>
cudaError_t launch_generic(const Q8Args &a, const Q8Addr &q, const B &blob, cudaStream_t s) {
    const int hpc = a.group < kGHeads ? a.group : kGHeads;
    auto bytes = [](int n, int hd) { return (static_cast<size_t>(n) * hd * (1 + kGW) + 2 * kGW * n) * sizeof(float); };
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(decode_q8_generic_kernel<B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(bytes(kGHeads, kMaxHeadDim)));
    });
    if (ce != cudaSuccess) return ce;
    const int n_chunks = (a.group + hpc - 1) / hpc;
    const long long grid = static_cast<long long>(a.n_units) * a.n_kv * n_chunks;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_early(decode_q8_generic_kernel<B>, static_cast<unsigned>(grid), 128, bytes(hpc, a.hd), s, a, q, hpc, blob);
}

// ------------------------------------------------------------- fast decode ----
//
// Head widths that are multiples of 16 up to 128, any group: both products of
// a key tile on warp-level m16n8k16 MMAs (f16 operands, f32 accumulators) with
// the keys and the dims on the 16-row side, so no row of an MMA is wasted:
//
//   S^T [16 keys x 8]  = (U_K - 128) [16 x hd] . Q^T [hd x 8]
//   O^T [16 dims x 8] += (U_V - 128)^T [16 x keys] . W^T [keys x 8]
//
// The 8 columns are four (query, head) pairs with the two f16 pieces of each
// f32 value (x = x0 + x1, 22 significant bits): columns 2c and 2c + 1 hold
// pair c's pieces, so a lane owns whole pairs: lane 4g + c holds pair c's
// scores of keys g and g + 8 and needs no shuffle to add the pieces.  The f16
// pairs of W (a key's two pieces) become the B fragment of the second product
// by one 8 x 8 transpose (movmatrix).  Elements widen from bytes to f16 by two
// byte permutes (1024 + u) and two subtractions (1152) for four values, exact;
// the transposed loads of V hand out two dims x two keys a word, which the
// same permutes sort into even and odd dims.
//
// CTA = 4 warps = one (unit, kv head, block of pairs); warp w takes the unit's
// tiles w, w + 4, ... of 32 keys through its own two-stage cp.async ring and
// keeps its own online softmax per pair; the warps' states merge at the end.
// The reference maximum of a pair moves only where a score passes it by more
// than 2^8 (one warp vote per tile finds out); sums stay per lane until the
// end.  W = p * vs / 2^c with c an exponent of the warp that follows the
// largest V scale of the tiles (O holds 2^-c times the sum), which keeps W in
// f16's range: W <= 2^14 after a factor 2^6.  W's second piece ends at 2^-24, half
// a step of which is 2^-25; as 2^c is at most 2^6 above the tile's largest scale
// 2^e (or 2^-60 of the largest that the warp has seen), a key's term is off by
// 2^-25 * 127 * 2^c / 2^6 <= 2^-25 of the tile's largest value (127 * 2^e) whatever
// its own scale, besides the 2^-22 of itself that two pieces leave out.
//
// Shared memory rows keep their 16-byte chunks XOR-swizzled by the key, so
// that the 8 rows of an ldmatrix fall in distinct bank groups.
//
// Measured (32 heads over 8 of 128, pages of 16, append included): 256
// sequences of 128 .. 32,768 in 492 us (6.27 TB/s, 0.92 of the copy peak; the
// loads alone take 473), 64 of 512 .. 4,096 in 47.6, one of 700 in 12.3; with
// pages of 5 (cp.async instead of TMA) 63 against 59 us on a like batch.  Two
// stages and four warps: three stages leave 2 CTAs a SM (585 us at 256
// sequences against 486 at the time), 1, 2 and 6 warps were slower too.

constexpr int kW = 4;            // warps per CTA
constexpr int kT = 32;           // keys per tile
constexpr int kStages = 2;
constexpr float kGrowQ = 8.f;    // log2 headroom of the reference maximum
constexpr float kWScale = 64.f;  // W's factor: 2^8 * 2^6 = 2^14

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// bytes i and j of w as (u - 128) in the halves of an f16 pair: 0x6400 | u is 1024 + u
template <int kSel>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
    const uint32_t b = __byte_perm(w, 0x64646464u, kSel);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&b), __half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ float ex2f(float x) {  // 2^x to about 2^-22 relative; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// the two f16 pieces of x as a pair (x0 in the low half)
__device__ __forceinline__ uint32_t pieces2(float x) {
    const __half h0 = __float2half_rn(x);
    const __half2 h = __halves2half2(h0, __float2half_rn(x - __half2float(h0)));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, uint32_t n) {  // n = 16, or 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap *map, int head, int off, int page, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];\n" ::"r"(dst),
        "l"(map), "r"(0), "r"(head), "r"(off), "r"(page), "r"(mbar)
        : "memory");
}

// Columns of a CTA: pair x = 4 * nt + c of its block is (query qi + x / gb,
// head h0 + x % gb) with gb heads per block.
template <int HD>
struct FastQ8 {
    static constexpr int kStage = 2 * kT * HD;  // bytes: K rows, V rows
    static constexpr int kChunks = HD / 16;     // 16-byte chunks of a row
    // chunk c of key j sits at chunk position c ^ swz(j)
    static __device__ __forceinline__ int swz(int j) {
        return HD == 128 ? (j & 7) : HD == 64 ? ((j >> 1) & 3) : HD == 32 ? ((j >> 2) & 1) : 0;
    }
};

template <int HD, int NB, bool kTma, class B>
__global__ void __launch_bounds__(32 * kW, NB <= 2 ? 3 : 2)
    decode_q8_kernel(Q8Args a, Q8Addr q, int gb, const __grid_constant__ Q8Maps maps, const __grid_constant__ B blob) {
    using F = FastQ8<HD>;
    constexpr int NC = F::kChunks;
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *const smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smraw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ float2 sc_tile[kW][kStages][kT];  // K and V scales of a tile's keys
    __shared__ uint64_t bars[kW][kStages];       // tile landed (TMA loads)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int n_hb = (a.group + gb - 1) / gb;  // head blocks of a kv head
    int b = blockIdx.x;
    const int hb = b % n_hb;
    b /= n_hb;
    const int kvh = b % a.n_kv, ui = b / a.n_kv;
    const Q8Unit u = unit_of(a, blob, ui);
    const int h0 = kvh * a.group + hb * gb, nh = min(gb, a.group - hb * gb);
    const int nq = u.nq, kbeg = u.kbeg, kend = u.kend;
    const int n_tiles = (kend - kbeg + kT - 1) / kT;
    const int my_n = warp < n_tiles ? (n_tiles - warp + kW - 1) / kW : 0;
    unsigned char *wbase = smem + warp * kStages * F::kStage;
    const uint32_t wbase_s = static_cast<uint32_t>(__cvta_generic_to_shared(wbase));
    const uint8_t *const kp = static_cast<const uint8_t *>(q.a.k), *const vp = static_cast<const uint8_t *>(q.a.v);

    // Tile loads.  Lane j finds key j's block a tile ahead of the copies and its
    // scales a tile ahead of their use, so that no lookup is waited for; the lanes
    // copy the rows' chunks, K and V, each a 16-byte cp.async (zeros past the
    // unit, and where the page lookup failed, with scale 0).
    // With whole sixteens of keys in every page, lanes 0 and 1 load their half of
    // a tile, K and V, as one TMA box each (a page's sixteen rows of this head, in
    // the same swizzle), and each half has one scale.
    auto find = [&](int kl) {  // the block of this lane's key (half) in tile kl, or -1
        const int pos = kbeg + (warp + kl * kW) * kT + (kTma ? 16 * lane : lane);
        return kl < my_n && pos < kend && (!kTma || lane < 2) ? block_of(q.a, u.slot, pos, a.err) : -1;
    };
    auto scales_of = [&](int blk) {
        return blk >= 0 ? make_float2(__ldcg(q.ks + blk * q.scale_stride + kvh), __ldcg(q.vs + blk * q.scale_stride + kvh))
                        : make_float2(0.f, 0.f);
    };
    auto load_tile = [&](int kl, int st, int blk) {
        const uint32_t dst = wbase_s + st * F::kStage;
        if constexpr (kTma) {
            if (lane < 2) {
                const int off = block_off(q.a, kbeg + (warp + kl * kW) * kT + 16 * lane);
                const uint32_t bar = static_cast<uint32_t>(__cvta_generic_to_shared(&bars[warp][st]));
                if (blk >= 0) {
                    tc::mbar_expect_tx(bar, 2 * 16 * HD);
                    tma_page(dst + lane * 16 * HD, &maps.k, kvh, off, blk * maps.n_layers + maps.layer, bar);
                    tma_page(dst + (kT + lane * 16) * HD, &maps.v, kvh, off, blk * maps.n_layers + maps.layer, bar);
                } else {
                    tc::mbar_arrive(bar);  // the half keeps what it holds: its keys are masked, its scale is 0
                }
            }
            return;
        }
        const int pos = kbeg + (warp + kl * kW) * kT + lane;
        const int64_t off = blk < 0 ? -1
                                    : static_cast<int64_t>(blk) * q.a.block_stride + q.a.layer_off +
                                          static_cast<int64_t>(block_off(q.a, pos)) * q.a.kv_dim +
                                          static_cast<int64_t>(kvh) * HD;
#pragma unroll
        for (int i = 0; i < NC; ++i) {  // kT * NC chunks over 32 lanes, K and V
            const int x = lane + 32 * i, j = x / NC, ch = x - j * NC;
            const int64_t o = __shfl_sync(kFull, off, j);
            const uint32_t d = dst + j * HD + ((ch ^ F::swz(j)) << 4), n = o >= 0 ? 16u : 0u;
            cp_async16z(d, kp + (o >= 0 ? o + 16 * ch : 0), n);
            cp_async16z(d + kT * HD, vp + (o >= 0 ? o + 16 * ch : 0), n);
        }
    };
    if constexpr (kTma) {
        if (lane < kStages) tc::mbar_init(static_cast<uint32_t>(__cvta_generic_to_shared(&bars[warp][lane])), 2);
        tc::fence_proxy_async();  // the barriers (this warp's own), before TMA uses them
        __syncwarp();
    }

    // Q^T fragments: pair x's pieces in columns 2c, 2c + 1 of n-tile x / 4.  As
    // a B fragment lane 4g + c holds column g = pair g / 2, piece g % 2, dims
    // 16s + 4c + (0, 1 | 2, 3) (the order in which ldmatrix hands out a row's
    // bytes).  Each pair is scaled by a power of two that puts its largest
    // entry into [2^14, 2^15).  The queries are no work of the launch before
    // this one, the pages may be; the first tile loads while the pieces are made.
    float qv[NB][NC][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int x = 4 * nb + (g >> 1), qi = x / gb, hi = x - qi * gb;
        const bool on = qi < nq && hi < nh;
        const float *row = a.Q + static_cast<size_t>(u.q_row + (on ? qi : 0)) * (a.n_heads * HD) +
                           static_cast<size_t>(h0 + (on ? hi : 0)) * HD;
#pragma unroll
        for (int s = 0; s < NC; ++s) {
            const float4 t = on ? __ldg(reinterpret_cast<const float4 *>(row + 16 * s + 4 * c)) : make_float4(0.f, 0.f, 0.f, 0.f);
            qv[nb][s][0] = t.x, qv[nb][s][1] = t.y, qv[nb][s][2] = t.z, qv[nb][s][3] = t.w;
        }
    }
    wait_previous();
    int blk_next;
    float2 sc_cur, sc_next = make_float2(0.f, 0.f);
    {
        const int blk = find(0);
        blk_next = find(1);
        if (0 < my_n) load_tile(0, 0, blk);
        if constexpr (!kTma) cp_async_commit();
        sc_cur = scales_of(blk);
    }
    uint32_t qf[NB][NC][2];
    float qinv[NB];  // of this lane's own pair, 4 * nb + c
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float mx = 0.f;
#pragma unroll
        for (int s = 0; s < NC; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qv[nb][s][i] *= a.scale_log2;
                mx = fmaxf(mx, fabsf(qv[nb][s][i]));
            }
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
        int e = 0;
        if (mx > 0.f && mx <= 3.4e38f)
            e = max(-126, min(126, 14 - (static_cast<int>((__float_as_uint(mx) >> 23) & 255u) - 127)));
        const float up = pow2f(e);
        qinv[nb] = __shfl_sync(kFull, pow2f(-e), 8 * c);  // lane 8c holds columns of pair c
#pragma unroll
        for (int s = 0; s < NC; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t p0 = pieces2(qv[nb][s][2 * i] * up), p1 = pieces2(qv[nb][s][2 * i + 1] * up);
                qf[nb][s][i] = __byte_perm(p0, p1, (g & 1) ? 0x7632 : 0x5410);  // this column's piece of both dims
            }
    }

    // ldmatrix addresses of this lane: matrix mi = lane / 8, row mr of it
    //   K: keys 8 (mi & 1) + mr, chunk + (mi >> 1);  V (transposed): the same
    const int mi = lane >> 3, mr = lane & 7, key_of = 8 * (mi & 1) + mr, ch_of = mi >> 1;
    // chunk pair s / 2 of key key_of (and of key_of + 16: the swizzle repeats
    // every eight keys); the last pair of an odd chunk count reads the last twice
    uint32_t at[(NC + 1) / 2];
#pragma unroll
    for (int s = 0; s < NC; s += 2) at[s / 2] = key_of * HD + ((min(s + ch_of, NC - 1) ^ F::swz(key_of)) << 4);
    bool landed = true;

    float m_run[NB], l_run[NB], o[NB][NC][4];
    int c_exp = 0, c_top = -126;  // O holds 2^-c_exp times the sum (and kWScale); c_top: the largest exponent seen
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        m_run[nb] = -INFINITY;
        l_run[nb] = 0.f;
#pragma unroll
        for (int s = 0; s < NC; ++s) o[nb][s][0] = o[nb][s][1] = o[nb][s][2] = o[nb][s][3] = 0.f;
    }
    // keys that this lane's pairs see: below lim
    int lim[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        const int qi = (4 * nb + c) / gb;
        lim[nb] = a.causal ? min(kend, u.see0 + min(qi, nq - 1)) : kend;
    }

    for (int k = 0; k < my_n; ++k) {
        if (k + 1 < my_n) load_tile(k + 1, (k + 1) % kStages, blk_next);
        if constexpr (!kTma) cp_async_commit();
        sc_next = scales_of(blk_next);
        blk_next = find(k + 2);
        const int st = k % kStages;
        float ksc[2], vsc2[2];  // TMA: of the tile's halves
        if constexpr (kTma) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ksc[h] = __shfl_sync(kFull, sc_cur.x, h);
                vsc2[h] = __shfl_sync(kFull, sc_cur.y, h);
            }
            landed = __all_sync(kFull, tc::mbar_wait(static_cast<uint32_t>(__cvta_generic_to_shared(&bars[warp][st])),
                                                     (k / kStages) & 1));
            if (!landed) {  // one more bounded wait for the copies in flight, this tile's and the next's
                for (int t = k; t <= k + 1 && t < my_n; ++t)
                    tc::mbar_wait(static_cast<uint32_t>(__cvta_generic_to_shared(&bars[warp][t % kStages])),
                                  (t / kStages) & 1);
                break;
            }
        } else {
            sc_tile[warp][st][lane] = sc_cur;
            cp_async_wait<1>();
            __syncwarp();
        }
        sc_cur = sc_next;
        const int pos0 = kbeg + (warp + k * kW) * kT;
        const uint32_t Ks = wbase_s + st * F::kStage, Vs = Ks + kT * HD;

        float sv[NB][4];  // scores of keys g, g + 8, g + 16, g + 24
#pragma unroll
        for (int kg = 0; kg < 2; ++kg) {
            float acc[NB][4];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) acc[nb][0] = acc[nb][1] = acc[nb][2] = acc[nb][3] = 0.f;
#pragma unroll
            for (int s = 0; s < NC; s += 2) {
                uint32_t r[4];
                ldsm4(r, Ks + at[s / 2] + 16 * kg * HD);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (s + h >= NC) continue;
                    const uint32_t af[4] = {widen2<0x4140>(r[2 * h]), widen2<0x4140>(r[2 * h + 1]),
                                            widen2<0x4342>(r[2 * h]), widen2<0x4342>(r[2 * h + 1])};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_f16(acc[nb], af, qf[nb][s + h][0], qf[nb][s + h][1]);
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                sv[nb][2 * kg] = acc[nb][0] + acc[nb][1];
                sv[nb][2 * kg + 1] = acc[nb][2] + acc[nb][3];
            }
        }
        // scales and mask; the maximum's move, when some lane asks for it
        float vsc[4];
        bool grow = false;
        float es = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 sc = kTma ? make_float2(ksc[i >> 1], vsc2[i >> 1]) : sc_tile[warp][st][g + 8 * i];
            vsc[i] = sc.y;
            es = fmaxf(es, sc.y);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float x = sv[nb][i] * (qinv[nb] * sc.x);
                sv[nb][i] = pos0 + g + 8 * i < lim[nb] ? x : -INFINITY;
                grow = grow || sv[nb][i] > m_run[nb] + kGrowQ;
            }
        }
        // the tile's largest V scale (a power of two, the same in every lane)
        const int e_tile = static_cast<int>(__reduce_max_sync(kFull, __float_as_uint(es) >> 23)) - 127;
        c_top = max(c_top, e_tile);
        const int want = max(e_tile, c_top - 60);  // O keeps within f32 when c goes down
        const bool first = k == 0;
        const bool move_c = first || want > c_exp || want < c_exp - 6;
        if (move_c || __any_sync(kFull, grow)) {
            const int c_new = move_c ? max(want, -126) : c_exp;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float top = fmaxf(fmaxf(sv[nb][0], sv[nb][1]), fmaxf(sv[nb][2], sv[nb][3]));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
                const float mn = top > m_run[nb] + kGrowQ || m_run[nb] == -INFINITY ? top : m_run[nb];
                const float al = mn == m_run[nb] || m_run[nb] == -INFINITY ? 1.f : ex2f(m_run[nb] - mn);
                m_run[nb] = mn;
                l_run[nb] *= al;
                if (!first) {
                    // a lane's accumulators belong to pair c's columns
                    const int d = c_exp - c_new;  // two exact steps
                    const float f1 = pow2f(d / 2), f2 = pow2f(d - d / 2) * al;
#pragma unroll
                    for (int s = 0; s < NC; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[nb][s][i] = o[nb][s][i] * f1 * f2;
                }
            }
            c_exp = c_new;
        }
        // W, its pieces transposed into B fragments: bf[nb][kg] = keys 16 kg + (0-7 | 8-15)
        uint32_t bf[NB][4];
        const float down = pow2f(-c_exp);  // c_exp in [-126, 122]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float vw = vsc[i] * down * kWScale;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const float p = ex2f(sv[nb][i] - (m_run[nb] == -INFINITY ? 0.f : m_run[nb]));
                l_run[nb] += p;
                bf[nb][i] = transpose8(pieces2(sv[nb][i] == -INFINITY ? 0.f : p * vw));
            }
        }
        // O^T += (U_V - 128)^T W^T
#pragma unroll
        for (int kg = 0; kg < 2; ++kg) {
#pragma unroll
            for (int s = 0; s < NC; s += 2) {
                uint32_t r[4];
                ldsm4t(r, Vs + at[s / 2] + 16 * kg * HD);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (s + h >= NC) continue;
                    // rows 0-7: the chunk's even dims, rows 8-15: its odd dims
                    const uint32_t af[4] = {widen2<0x4240>(r[2 * h]), widen2<0x4341>(r[2 * h]),
                                            widen2<0x4240>(r[2 * h + 1]), widen2<0x4341>(r[2 * h + 1])};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) mma_f16(o[nb][s + h], af, bf[nb][2 * kg], bf[nb][2 * kg + 1]);
                }
            }
        }
        __syncwarp();
    }
    if constexpr (!kTma) cp_async_wait<0>();
    if (!landed && lane == 0) flag_error(a.err, 2);
    __syncthreads();  // every warp is done with its stages

    // publish each warp's (O, m, l), pair by pair: O[pair][dim] behind one another
    constexpr int NP = 4 * NB;
    float *R = reinterpret_cast<float *>(smem) + warp * NP * (HD + 2);
    const float o1 = pow2f(c_exp / 2) * (1.f / kWScale), o2 = pow2f(c_exp - c_exp / 2);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        float l = l_run[nb];
        l += __shfl_xor_sync(kFull, l, 4);
        l += __shfl_xor_sync(kFull, l, 8);
        l += __shfl_xor_sync(kFull, l, 16);
        float *Rp = R + (4 * nb + c) * (HD + 2);
#pragma unroll
        for (int s = 0; s < NC; ++s) {
            Rp[16 * s + 2 * g] = (o[nb][s][0] + o[nb][s][1]) * o1 * o2;
            Rp[16 * s + 2 * g + 1] = (o[nb][s][2] + o[nb][s][3]) * o1 * o2;
        }
        if (g == 0) {
            Rp[HD] = m_run[nb];
            Rp[HD + 1] = l;
        }
    }
    __syncthreads();
    for (int x = warp; x < NP; x += kW) {  // warp per pair
        const int qi = x / gb, hi = x - qi * gb;
        if (qi >= nq || hi >= nh) continue;
        const float *R0 = reinterpret_cast<const float *>(smem) + x * (HD + 2);
        float M = -INFINITY, den = 0.f, wt[kW];
#pragma unroll
        for (int w = 0; w < kW; ++w) M = fmaxf(M, R0[w * NP * (HD + 2) + HD]);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            // a warp that saw no key of the pair has l = 0 (one that saw only NaN
            // scores has no maximum either, and l = NaN)
            const float mw = R0[w * NP * (HD + 2) + HD], lw = R0[w * NP * (HD + 2) + HD + 1];
            wt[w] = lw == 0.f ? 0.f : mw == -INFINITY ? 1.f : exp2f(mw - M);
            if (wt[w] != 0.f) den = fmaf(wt[w], lw, den);
        }
        const int h = h0 + hi;
        const size_t ph = u.part0 < 0 ? 0 : static_cast<size_t>(u.part0 + qi * u.n_rec + u.rec) * a.n_heads + h;
        float *dst = u.part0 < 0 ? a.out + static_cast<size_t>(u.q_row + qi) * (a.n_heads * HD) + static_cast<size_t>(h) * HD
                                 : a.pacc + ph * HD;
        for (int d = lane; d < HD; d += 32) {
            float num = 0.f;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float *Rw = R0 + w * NP * (HD + 2);
                if (wt[w] != 0.f) num = fmaf(wt[w], Rw[d], num);
            }
            dst[d] = u.part0 < 0 ? num / den : num;
        }
        if (u.part0 >= 0 && lane == 0) {
            a.pm[ph] = M;
            a.pl[ph] = den;
        }
    }
    if (u.part0 >= 0 && last_of_block(a, u, kvh * n_hb + hb))
        for (int x = warp; x < NP; x += kW) {
            const int qi = x / gb, hi = x - qi * gb;
            if (qi < nq && hi < nh) join_records(a, u, qi, h0 + hi, lane);
        }
}

template <int HD, int NB, bool kTma, class B>
cudaError_t launch_fast(const Q8Args &a, const Q8Addr &q, int gb, const B &blob, cudaStream_t s) {
    using F = FastQ8<HD>;
    constexpr size_t smem = static_cast<size_t>(kW) * kStages * F::kStage + 1024;  // + alignment slack
    static_assert(smem - 1024 >= static_cast<size_t>(kW) * 4 * NB * (HD + 2) * sizeof(float), "the merge fits the stages");
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(decode_q8_kernel<HD, NB, kTma, B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(smem));
    });
    if (ce != cudaSuccess) return ce;
    const long long grid = static_cast<long long>(a.n_units) * a.n_kv * ((a.group + gb - 1) / gb);
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    Q8Maps maps{};
    if (kTma) {
        maps = *static_cast<const Q8Maps *>(q.maps);
        maps.layer = static_cast<int>(q.a.layer_off / (static_cast<int64_t>(q.a.bs) * q.a.kv_dim));
    }
    return launch_early(decode_q8_kernel<HD, NB, kTma, B>, static_cast<unsigned>(grid), 32 * kW, smem, s, a, q, gb, maps, blob);
}

// Heads per CTA and queries per unit: up to 16 (query, head) pairs share a
// unit's keys.  A group of more than 16 heads is cut into blocks of 16.
bool fast_shape(int head_dim) { return head_dim % 16 == 0 && head_dim <= 128; }
int heads_per_block(int group) { return group < 16 ? group : 16; }

template <int HD, class B>
cudaError_t launch_fast_hd(const Q8Args &a, const Q8Addr &q, const B &blob, cudaStream_t s) {
    const int gb = heads_per_block(a.group);
    // the widest unit of the call decides; a unit of fewer pairs leaves columns idle
    const int pairs = gb * a.max_q;
    if constexpr (HD == 64 || HD == 128)
        if (q.maps) {
            if (pairs <= 4) return launch_fast<HD, 1, true>(a, q, gb, blob, s);
            if (pairs <= 8) return launch_fast<HD, 2, true>(a, q, gb, blob, s);
            return launch_fast<HD, 4, true>(a, q, gb, blob, s);
        }
    if (pairs <= 4) return launch_fast<HD, 1, false>(a, q, gb, blob, s);
    if (pairs <= 8) return launch_fast<HD, 2, false>(a, q, gb, blob, s);
    return launch_fast<HD, 4, false>(a, q, gb, blob, s);
}

template <class B>
cudaError_t launch_decode_with(const Q8Args &a, const Q8Addr &q, const B &blob, cudaStream_t s) {
    switch (fast_shape(a.hd) ? a.hd : 0) {
        case 16: return launch_fast_hd<16>(a, q, blob, s);
        case 32: return launch_fast_hd<32>(a, q, blob, s);
        case 48: return launch_fast_hd<48>(a, q, blob, s);
        case 64: return launch_fast_hd<64>(a, q, blob, s);
        case 80: return launch_fast_hd<80>(a, q, blob, s);
        case 96: return launch_fast_hd<96>(a, q, blob, s);
        case 112: return launch_fast_hd<112>(a, q, blob, s);
        case 128: return launch_fast_hd<128>(a, q, blob, s);
        default: return launch_generic(a, q, blob, s);
    }
}

// -------------------------------------------------------------- split pass ----
//
// Operand images for the tensor-core launches (the layout of kImageBytes): one
// CTA per (64-key tile, kv head).  The images' power of two needs no look at
// the values: with 2^t the tile's largest scale every magnitude is at most
// 127 * 2^t, so 2^(8 - t) brings them below 2^15, and (u - 128) * 2^(8 - t + e)
// is an f16 value -- seven bits times a factor of at least 2^-24, the smallest
// f16, where the key's scale 2^e lies at most 2^32 below the tile's; below that the
// factor rounds to 0 -- so piece 1 is left out, as on the other narrow pools.  K goes straight to its image; V's bytes turn
// through shared memory.  Bound by the images' writes: 24 us for 320 tiles of 8
// heads of 128 (42 MB read, 84 MB written).

constexpr int kVPitch = 132;  // bytes from key to key: four keys on, another bank

// four bytes as (u - 128) times the pair of powers of two s2, in f16 (exact)
__device__ __forceinline__ uint2 widen4(uint32_t w, __half2 s2) {
    const uint32_t lo = widen2<0x4140>(w), hi = widen2<0x4342>(w);
    const __half2 a = __hmul2(*reinterpret_cast<const __half2 *>(&lo), s2), b = __hmul2(*reinterpret_cast<const __half2 *>(&hi), s2);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

template <bool kWide>  // head width 128
__global__ void __launch_bounds__(256) split_q8_kernel(SplitArgs p, Q8Addr q) {
    static_assert(sizeof(kFull) == 4 && kFull == 0xffffffffu, "the shuffles below are whole warps'");
    const int hd = kWide ? 128 : q.hd;
    __shared__ __align__(16) uint8_t vs[kKeyTile * kVPitch];
    __shared__ int64_t row_of[kKeyTile];
    __shared__ __half kf[kKeyTile], vf[kKeyTile];  // each key's factor
    __shared__ float top[2][2];
    const int it = blockIdx.x / p.n_kv, kvh = blockIdx.x - it * p.n_kv;
    const SplitItem t = p.items[it];
    const RowDesc rd = p.rows[t.row];
    const int tid = threadIdx.x;
    float ks = 0.f, vsc = 0.f;
    if (tid < kKeyTile) {  // two warps: the keys' rows and scales
        const int pos = t.kt * kKeyTile + tid;
        int64_t o = -1;
        if (pos < rd.past_len + rd.n_q) {
            const int blk = block_of(q.a, rd.slot, pos, p.err);
            if (blk >= 0) {
                o = static_cast<int64_t>(blk) * q.a.block_stride + q.a.layer_off +
                    static_cast<int64_t>(block_off(q.a, pos)) * q.a.kv_dim + static_cast<int64_t>(kvh) * hd;
                ks = __ldg(q.ks + blk * q.scale_stride + kvh);
                vsc = __ldg(q.vs + blk * q.scale_stride + kvh);
            }
        }
        row_of[tid] = o;
        float mk = ks, mv = vsc;  // fmaxf passes over a NaN scale
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) {
            mk = fmaxf(mk, __shfl_xor_sync(kFull, mk, x));
            mv = fmaxf(mv, __shfl_xor_sync(kFull, mv, x));
        }
        if ((tid & 31) == 0) top[0][tid >> 5] = mk, top[1][tid >> 5] = mv;
    }
    __syncthreads();
    int ex[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float m = fmaxf(top[i][0], top[i][1]);
        ex[i] = max(-113, min(126, 8 - (static_cast<int>((__float_as_uint(m) >> 23) & 255u) - 127)));
    }
    if (tid < kKeyTile) {
        // scale * 2^ex <= 2^8; f16 keeps 2^-24, and a NaN
        kf[tid] = __float2half_rn(ks * pow2f(ex[0]));
        vf[tid] = __float2half_rn(vsc * pow2f(ex[1]));
    }
    // V's and K's bytes (and zeros, u = 128, past the row's keys), all on the way at
    // once.  K: k-block c >> 9 (64 dims), key (c >> 3) & 63, swizzled chunk c & 7
    constexpr int kKC = static_cast<int>(kImagePlane / 16) / 256;
    uint4 vw[2];
    uint2 kw[kKC];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int key = (tid + 256 * i) >> 3, ch = tid & 7;
        const int64_t o = row_of[key];
        vw[i] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
        if (o >= 0 && 16 * ch < hd) vw[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(q.a.v) + o + 16 * ch));
    }
#pragma unroll
    for (int i = 0; i < kKC; ++i) {
        const int c = tid + 256 * i, r = (c >> 3) & 63, dim = (c >> 9) * 64 + ((c & 7) ^ (r & 7)) * 8;
        const int64_t o = row_of[r];
        kw[i] = make_uint2(0x80808080u, 0x80808080u);
        if (o >= 0 && dim < hd) kw[i] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(q.a.k) + o + dim));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t *d = reinterpret_cast<uint32_t *>(vs + ((tid + 256 * i) >> 3) * kVPitch + 16 * (tid & 7));
        d[0] = vw[i].x, d[1] = vw[i].y, d[2] = vw[i].z, d[3] = vw[i].w;
    }
    __syncthreads();
    unsigned char *img = p.img + (static_cast<size_t>(t.slot) * p.n_kv + kvh) * kImageBytes;
#pragma unroll
    for (int i = 0; i < kKC; ++i) {
        const int c = tid + 256 * i, r = (c >> 3) & 63, dim = (c >> 9) * 64 + ((c & 7) ^ (r & 7)) * 8;
        if (dim >= hd) continue;
        const __half2 f = __half2half2(kf[r]);
        const uint2 a = widen4(kw[i].x, f), b = widen4(kw[i].y, f);
        *reinterpret_cast<uint4 *>(img + c * 16) = make_uint4(a.x, a.y, b.x, b.y);
    }
    // V^T: four dims d .. d + 3 of eight keys k0 .. at a time: a word of each key,
    // each dim's eight values together one chunk of the image (dim row, chunk
    // k0 / 8 at its swizzled place)
    if (tid < 2) reinterpret_cast<int32_t *>(img + kImageExpOff)[tid] = ex[tid];
    const int d = 4 * (tid >> 3), k0 = 8 * (tid & 7);
    if (d >= hd) return;
    uint32_t w[8];
    __half2 f[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint32_t *>(vs + (k0 + j) * kVPitch + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __halves2half2(vf[k0 + 2 * j], vf[k0 + 2 * j + 1]);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // byte x of two keys' words beside one another
            const uint32_t two = __byte_perm(w[2 * j], w[2 * j + 1], x | (4 + x) << 4);
            const uint32_t h = widen2<0x4140>(two);
            const __half2 z = __hmul2(*reinterpret_cast<const __half2 *>(&h), f[j]);
            y[j] = *reinterpret_cast<const uint32_t *>(&z);
        }
        const int dd = d + x;
        *reinterpret_cast<uint4 *>(img + 2 * kImagePlane + (dd * 8 + ((k0 >> 3) ^ (dd & 7))) * 16) =
            make_uint4(y[0], y[1], y[2], y[3]);
    }
}

}  // namespace

int q8_query_block(int head_dim, int group) {
    return fast_shape(head_dim) ? std::max(1, 16 / heads_per_block(group)) : 1;
}

cudaError_t make_q8_maps(Q8Maps *m, const Q8Addr &q, int n_layers, bool *usable) {
    *usable = false;
    m->n_layers = n_layers;
    if ((q.hd != 64 && q.hd != 128) || q.a.bs % 16 != 0 ||
        static_cast<int64_t>(q.a.n_blocks) * n_layers > 0x7fffffff)
        return cudaSuccess;
    EncodeTiled f;
    const cudaError_t e = encode_tiled(&f);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(q.hd), static_cast<cuuint64_t>(q.n_kv),
                                static_cast<cuuint64_t>(q.a.bs), static_cast<cuuint64_t>(q.a.n_blocks) * n_layers};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(q.hd), static_cast<cuuint64_t>(q.a.kv_dim),
                                   static_cast<cuuint64_t>(q.a.bs) * q.a.kv_dim};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(q.hd), 1, 16, 1}, one[4] = {1, 1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (f(i ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, i ? q.a.v : q.a.k, dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, q.hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    *usable = true;
    return cudaSuccess;
}

int q8_counters(int head_dim, int group, int n_kv) {
    const int per = fast_shape(head_dim) ? heads_per_block(group) : group < kGHeads ? group : kGHeads;
    return n_kv * ((group + per - 1) / per);
}

cudaError_t launch_decode_q8(const Q8Args &a, const Q8Addr &q, cudaStream_t s) {
    return with_blob(a.blob, a.blob_n, [&](const auto &b) { return launch_decode_with(a, q, b, s); });
}

cudaError_t launch_split_q8(const SplitArgs &a, const Q8Addr &q, cudaStream_t s) {
    if (q.hd % 16 != 0 || q.hd > 128) return cudaErrorInvalidValue;
    const long long grid = static_cast<long long>(a.n_items) * a.n_kv;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (q.hd == 128) split_q8_kernel<true><<<static_cast<unsigned>(grid), 256, 0, s>>>(a, q);
    else split_q8_kernel<false><<<static_cast<unsigned>(grid), 256, 0, s>>>(a, q);
    return cudaGetLastError();
}

}  // namespace pkv

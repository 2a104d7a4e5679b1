// pkv_packed.cu -- attention over whole prompts packed behind one another
// (bf16 or f16 rows, grouped heads, causal or not).
//
//   o[i, h] = sum_j p_ij v[j, h / G] / sum_j p_ij,  p_ij = 2^(s_ij - m_i),
//   s_ij = scale * log2(e) * <q[i, h], k[j, h / G]>
//
// over the keys j of query i's own sequence, j <= i where causal.  Scores,
// running maxima, sums and the output accumulate in f32 in one pass over the
// keys; the output is rounded once.
//
// The sequences' places travel in the launch's parameters, longest sequence
// first, so a call needs no upload and no scratch and can be captured into a
// graph.
#include "pkv_elem.h"
#include "pkv_half.h"
#include "pkv_internal.h"
#include "pkv_packed_tc.h"

namespace pkv {
namespace {

using namespace tc;

// ---------------------------------------------------------------- general ----
//
// Any head width up to 256, any strides and alignment, any scale.  CTA = 4 warps
// = 64 queries of one head, 16 a warp; keys go through shared memory 32 at a
// time (rows padded with zeros to DP dims, and by 16 bytes, so that ldmatrix
// meets no bank twice); both products on m16n8k16 MMAs:
//
//   S [16 x 32] = Q K^T          A, B by ldmatrix
//   O [16 x DP] += P V           A from S's accumulators, B by transposed ldmatrix
//
// Scores are scaled in f32.  In sequences of more than kLongKeys each tile's
// products have a sum of their own, added to O in f32, as the tensor core would
// round O toward zero twice a tile (10% of the launch, in an instance of its own).
// A key that a query does not see has probability 0;
// as zero times an infinity is NaN, a tile that some row does not see whole is
// looked over, and where it holds a value that is not finite its products are
// made one by one, over the keys that the row sees.
//
// Measured (causal, 32 heads over 8, 24 prompts of 16 .. 4,096): 95 TFLOP/s at
// 160-wide heads (3.65 ms; f32 products from shared memory took 67.7), 108 at
// 256 (16 heads), 76 at 128 off 16-byte boundaries (element loads).  Bound by
// the loads, which wait for the tile before them: two to five CTAs a SM overlap.

constexpr int kGQ = 64, kGK = 32;

template <int DP>
struct GenCfg {
    static constexpr int kPitch = DP + 8;  // elements
    static constexpr size_t kSmem = static_cast<size_t>(kGQ + 2 * kGK) * kPitch * 2 + kGQ * (kGK + 1) * sizeof(float);
};

// Rows 0 .. rows - 1 of hd elements into padded shared rows, zeros elsewhere;
// whether a value was not finite (of this thread's).
template <class T, int DP, bool kVec>
__device__ __forceinline__ bool load_rows(unsigned short *dst, const T *src, int64_t stride, int rows, int n_rows, int hd) {
    bool bad = false;
    if constexpr (kVec) {
        for (int i = threadIdx.x; i < n_rows * (DP / 8); i += 128) {
            const int r = i / (DP / 8), c = i - r * (DP / 8);
            uint4 x = make_uint4(0, 0, 0, 0);
            if (r < rows && 8 * c < hd) x = __ldg(reinterpret_cast<const uint4 *>(src + r * stride + 8 * c));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) bad = bad || not_finite<T>(w[k]) || not_finite<T>(w[k] >> 16);
            *reinterpret_cast<uint4 *>(dst + r * GenCfg<DP>::kPitch + 8 * c) = x;
        }
    } else {
        for (int i = threadIdx.x; i < n_rows * DP; i += 128) {
            const int r = i / DP, d = i - r * DP;
            unsigned short x = 0;
            if (r < rows && d < hd) x = __ldg(reinterpret_cast<const unsigned short *>(src) + r * stride + d);
            bad = bad || not_finite<T>(x);
            dst[r * GenCfg<DP>::kPitch + d] = x;
        }
    }
    return bad;
}

template <class T, int DP, bool kVec, bool kLong, int N>
__global__ void __launch_bounds__(128) packed_general_kernel(const __grid_constant__ PackedArgs a,
                                                             const __grid_constant__ PackedSeqs<N> l) {
    using C = GenCfg<DP>;
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned short *Qs = reinterpret_cast<unsigned short *>(smraw), *Ks = Qs + kGQ * C::kPitch, *Vs = Ks + kGK * C::kPitch;
    float *Ps = reinterpret_cast<float *>(Vs + kGK * C::kPitch);  // [kGQ][kGK + 1], of tiles made one by one
    const int hd = a.hd, h = blockIdx.x % a.n_heads, t = blockIdx.x / a.n_heads;
    const int s = seq_of_tile(l, t);
    const int len = l.len[s];
    const int q0 = (l.tile0[s + 1] - l.tile0[s] - 1 - (t - l.tile0[s])) * kGQ;  // the last queries, with the most keys, first
    const int64_t row0 = l.start[s];
    const int kvh = h / (a.n_heads / a.n_kv);
    const T *Q = static_cast<const T *>(a.Q) + (row0 + q0) * a.q_stride + static_cast<int64_t>(h) * hd;
    const T *K = static_cast<const T *>(a.K) + row0 * a.k_stride + static_cast<int64_t>(kvh) * hd;
    const T *V = static_cast<const T *>(a.V) + row0 * a.v_stride + static_cast<int64_t>(kvh) * hd;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, mi = lane >> 3, mr = lane & 7;
    load_rows<T, DP, kVec>(Qs, Q, a.q_stride, min(kGQ, len - q0), kGQ, hd);
    // rows g and g + 8 of the warp's sixteen: the keys that they see, running maximum and sum
    int lim[2];
    float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int q = q0 + 16 * warp + g + 8 * x;
        lim[x] = q >= len ? 0 : a.causal ? q + 1 : len;
    }
    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    const int kend = a.causal ? min(len, q0 + kGQ) : len;  // keys that the tile sees
    const int whole = a.causal ? q0 + 1 : len;             // keys that all of its rows see
    for (int k0 = 0; k0 < kend; k0 += kGK) {
        __syncthreads();
        load_rows<T, DP, kVec>(Ks, K + k0 * a.k_stride, a.k_stride, min(kGK, len - k0), kGK, hd);
        const bool odd = load_rows<T, DP, kVec>(Vs, V + k0 * a.v_stride, a.v_stride, min(kGK, len - k0), kGK, hd);
        const bool single = __syncthreads_or(odd && k0 + kGK > whole);
        float sc[kGK / 8][4];
#pragma unroll
        for (int i = 0; i < kGK / 8; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
        for (int d = 0; d < DP; d += 16) {
            uint32_t qa[4];  // rows mr (+ 8), dims d (+ 8)
            ldsm4<false>(qa, Qs + (16 * warp + mr + 8 * (mi & 1)) * C::kPitch + d + 8 * (mi >> 1));
#pragma unroll
            for (int n = 0; n < kGK / 16; ++n) {
                uint32_t kb[4];
                ldsm4<false>(kb, Ks + (16 * n + mr + 8 * (mi >> 1)) * C::kPitch + d + 8 * (mi & 1));
                mma16<T>(sc[2 * n], qa, kb[0], kb[1]);
                mma16<T>(sc[2 * n + 1], qa, kb[2], kb[3]);
            }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kGK / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = k0 + 8 * i + 2 * c + (e & 1);
                sc[i][e] = key < lim[e >> 1] ? sc[i][e] * a.scale_log2 : -INFINITY;
                top[e >> 1] = fmaxf(top[e >> 1], sc[i][e]);
            }
        uint32_t p[kGK / 16][4];  // as A: keys 16 n + (2c, 2c + 1) and + 8, rows g and g + 8
        float al[2], ps[2] = {0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
            const float mn = fmaxf(m[x], top[x]);
            al[x] = mn == m[x] ? 1.f : ex2(m[x] - mn);
            m[x] = mn;
        }
#pragma unroll
        for (int i = 0; i < kGK / 8; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float mn = m[e >> 1];
                sc[i][e] = sc[i][e] == -INFINITY ? 0.f : ex2(sc[i][e] - (mn == -INFINITY ? 0.f : mn));
                ps[e >> 1] += sc[i][e];
            }
            p[i >> 1][2 * (i & 1)] = pack2(T{}, sc[i][0], sc[i][1]);
            p[i >> 1][2 * (i & 1) + 1] = pack2(T{}, sc[i][2], sc[i][3]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) sum[x] = fmaf(sum[x], al[x], ps[x]);
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] *= al[0], o[i][1] *= al[0], o[i][2] *= al[1], o[i][3] *= al[1];
        if (!single) {
            const bool own = kLong && len > kLongKeys;  // the tile's products in sums of their own
#pragma unroll
            for (int d = 0; d < DP; d += 16) {
                float t[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[0][e] = own ? 0.f : o[d / 8][e], t[1][e] = own ? 0.f : o[d / 8 + 1][e];
#pragma unroll
                for (int n = 0; n < kGK / 16; ++n) {
                    uint32_t vb[4];
                    ldsm4<true>(vb, Vs + (16 * n + mr + 8 * (mi & 1)) * C::kPitch + d + 8 * (mi >> 1));
                    mma16<T>(t[0], p[n], vb[0], vb[1]);
                    mma16<T>(t[1], p[n], vb[2], vb[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[d / 8][e] = own ? o[d / 8][e] + t[0][e] : t[0][e];
                    o[d / 8 + 1][e] = own ? o[d / 8 + 1][e] + t[1][e] : t[1][e];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kGK / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    Ps[(16 * warp + g + 8 * (e >> 1)) * (kGK + 1) + 8 * i + 2 * c + (e & 1)] =
                        half_of(T{}, p[i >> 1][2 * (i & 1) + (e >> 1)], e & 1);
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < kGK; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (k0 + k >= lim[x]) continue;
                    const float pk = Ps[(16 * warp + g + 8 * x) * (kGK + 1) + k];
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        const uint32_t v = *reinterpret_cast<const uint32_t *>(Vs + k * C::kPitch + 8 * i + 2 * c);
                        o[i][2 * x] = fmaf(pk, half_of(T{}, v, 0), o[i][2 * x]);
                        o[i][2 * x + 1] = fmaf(pk, half_of(T{}, v, 1), o[i][2 * x + 1]);
                    }
                }
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        const int q = q0 + 16 * warp + g + 8 * x;
        if (q >= len) continue;
        T *out = static_cast<T *>(a.out) + (row0 + q) * a.o_stride + static_cast<int64_t>(h) * hd;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (8 * i + 2 * c + e < hd) narrow(out + 8 * i + 2 * c + e, o[i][2 * x + e] / sum[x]);
    }
}

template <int N>
void fill_seqs(PackedSeqs<N> &l, const int32_t *start, const int32_t *len, int32_t n, int32_t tile) {
    l.n = n;
    int32_t at = 0;
    for (int32_t i = 0; i < n; ++i) {
        l.start[i] = start[i];
        l.len[i] = len[i];
        l.tile0[i] = at;
        at += (len[i] + tile - 1) / tile;
    }
    l.tile0[n] = at;
}

template <class T, int DP, bool kVec, bool kLong, int N>
cudaError_t launch_general_n(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    PackedSeqs<N> l;
    fill_seqs(l, start, len, n, kGQ);
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(packed_general_kernel<T, DP, kVec, kLong, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(GenCfg<DP>::kSmem));
    });
    if (ce != cudaSuccess) return ce;
    const long long grid = static_cast<long long>(l.tile0[n]) * a.n_heads;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    packed_general_kernel<T, DP, kVec, kLong, N><<<static_cast<unsigned>(grid), 128, GenCfg<DP>::kSmem, s>>>(a, l);
    return cudaGetLastError();
}

template <int D, class T, int N, bool kLong>
__global__ void __launch_bounds__(kTcThreads, 1)
    packed_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ PackedArgs a,
                     const __grid_constant__ PackedSeqs<N> l, int log_p) {
    packed_tc<D, T, kLong, WholePrompts<N>>(mq, mk, mv, mk, mv, a, l, log_p);
}

// Whether the tensor-core kernel takes the call: TMA's alignment rules, a
// positive finite scale (the kernel masks with -inf before it scales).
bool tc_takes(const PackedArgs &a) {
    auto ok = [](const void *p, int64_t stride) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0 && stride < (1LL << 38);
    };
    return a.hd % 8 == 0 && a.hd <= 128 && ok(a.Q, a.q_stride) && ok(a.K, a.k_stride) && ok(a.V, a.v_stride) &&
           ok(a.out, a.o_stride) && a.scale_log2 > 0.f && a.scale_log2 <= 3e38f;
}

template <int D, class T, int N, bool kLong>
cudaError_t launch_tc_n(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    using C = TcCfg<D>;
    static PerDeviceOnce configured;  // the attributes are per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        // setmaxnreg.inc waits for registers of the launch's own: launch only
        // if the kernel starts with what the split was sized for
        cudaFuncAttributes fa{};
        cudaError_t e = cudaFuncGetAttributes(&fa, packed_tc_kernel<D, T, N, kLong>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kTcLaunchRegs || fa.maxThreadsPerBlock < kTcThreads) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(packed_tc_kernel<D, T, N, kLong>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(C::kSmem));
    });
    if (ce != cudaSuccess) return ce;
    const int group = a.n_heads / a.n_kv;
    int log_p = 0;
    while (log_p < 4 && group % (2 << log_p) == 0) ++log_p;
    EncodeTiled f;
    cudaError_t e = encode_tiled(&f);
    CUtensorMap mq, mk, mv;
    if (e == cudaSuccess) e = rows_map(&mq, f, a.type, a.hd, a.n_tokens, a.Q, a.q_stride, a.n_heads, 1 << log_p, 128 >> log_p);
    if (e == cudaSuccess) e = rows_map(&mk, f, a.type, a.hd, a.n_tokens, a.K, a.k_stride, a.n_kv, 1, kKeys);
    if (e == cudaSuccess) e = rows_map(&mv, f, a.type, a.hd, a.n_tokens, a.V, a.v_stride, a.n_kv, 1, kKeys);
    if (e != cudaSuccess) return e;
    PackedSeqs<N> l;
    fill_seqs(l, start, len, n, 2 * (128 >> log_p));
    const long long grid = static_cast<long long>(l.tile0[n]) * (a.n_heads >> log_p);
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    PackedArgs b = a;
    b.out32 = a.hd % 16 == 0 && a.o_stride % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    packed_tc_kernel<D, T, N, kLong><<<static_cast<unsigned>(grid), kTcThreads, C::kSmem, s>>>(mq, mk, mv, b, l, log_p);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_tc(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    const bool few = n <= 64;
    if (len[0] > kLongKeys)  // the longest
        return a.hd <= 64 ? launch_tc_n<64, T, kPackedSeqs, true>(a, start, len, n, s)
                          : launch_tc_n<128, T, kPackedSeqs, true>(a, start, len, n, s);
    if (a.hd <= 64)
        return few ? launch_tc_n<64, T, 64, false>(a, start, len, n, s) : launch_tc_n<64, T, kPackedSeqs, false>(a, start, len, n, s);
    return few ? launch_tc_n<128, T, 64, false>(a, start, len, n, s) : launch_tc_n<128, T, kPackedSeqs, false>(a, start, len, n, s);
}

template <class T, int DP>
cudaError_t launch_general_d(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    auto ok = [](const void *p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; };
    const bool vec = a.hd % 8 == 0 && ok(a.Q, a.q_stride) && ok(a.K, a.k_stride) && ok(a.V, a.v_stride);
    if (len[0] > kLongKeys)  // the longest
        return vec ? launch_general_n<T, DP, true, true, kPackedSeqs>(a, start, len, n, s)
                   : launch_general_n<T, DP, false, true, kPackedSeqs>(a, start, len, n, s);
    return vec ? launch_general_n<T, DP, true, false, kPackedSeqs>(a, start, len, n, s)
               : launch_general_n<T, DP, false, false, kPackedSeqs>(a, start, len, n, s);
}
template <class T>
cudaError_t launch_general(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    if (a.hd <= 64) return launch_general_d<T, 64>(a, start, len, n, s);
    if (a.hd <= 128) return launch_general_d<T, 128>(a, start, len, n, s);
    if (a.hd <= 192) return launch_general_d<T, 192>(a, start, len, n, s);
    return launch_general_d<T, 256>(a, start, len, n, s);
}

}  // namespace

cudaError_t encode_tiled(EncodeTiled *out) {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled f = known.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (!p || q != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        f = reinterpret_cast<EncodeTiled>(p);
        known.store(f, std::memory_order_release);
    }
    *out = f;
    return cudaSuccess;
}

cudaError_t launch_packed(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n_seqs,
                          cudaStream_t s) {
    if (n_seqs <= 0 || n_seqs > kPackedSeqs) return cudaErrorInvalidValue;
    if (tc_takes(a)) {
        if (a.type == Elem::bf16) return launch_tc<bf16>(a, start, len, n_seqs, s);
        if (a.type == Elem::f16) return launch_tc<f16>(a, start, len, n_seqs, s);
    }
    if (a.type == Elem::bf16) return launch_general<bf16>(a, start, len, n_seqs, s);
    if (a.type == Elem::f16) return launch_general<f16>(a, start, len, n_seqs, s);
    return cudaErrorInvalidValue;
}

}  // namespace pkv

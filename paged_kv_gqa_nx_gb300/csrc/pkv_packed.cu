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
#include "pkv_internal.h"

#include <cuda_fp16.h>

namespace pkv {
namespace {

using f16 = __half;

__device__ __forceinline__ float widen(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(f16 x) { return __half2float(x); }
__device__ __forceinline__ void narrow(bf16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void narrow(f16 *p, float x) { *p = __float2half_rn(x); }

// The sequence of query tile `t` (tiles of the list's sequences in order).
template <int N>
__device__ __forceinline__ int seq_of_tile(const PackedSeqs<N> &l, int t) {
    int lo = 0, hi = l.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.tile0[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---------------------------------------------------------------- general ----
//
// Any head width up to 256, any strides and alignment.  CTA = 128 threads = 32
// queries of one head; four neighbouring threads share a query.  Keys go
// through shared memory 32 at a time; thread t of a query scores keys t, t + 4,
// ... and owns the output dims t, t + 4, ....  A key that a query does not see
// is skipped, never multiplied by a zero probability, so infinities and NaN
// there do not reach it.  Bound by the shared-memory reads of its products.

constexpr int kGQ = 32, kGK = 32, kGOwn = kMaxHeadDim / 4;

template <class T, int N>
__global__ void __launch_bounds__(128) packed_general_kernel(const __grid_constant__ PackedArgs a,
                                                             const __grid_constant__ PackedSeqs<N> l) {
    extern __shared__ __align__(16) float sm[];
    const int hd = a.hd, pitch = hd + 1;
    float *Qs = sm, *Ks = Qs + kGQ * pitch, *Vs = Ks + kGK * pitch, *Ps = Vs + kGK * pitch;  // Ps: [kGQ][kGK + 1]
    const int h = blockIdx.x % a.n_heads, t = blockIdx.x / a.n_heads;
    const int s = seq_of_tile(l, t);
    const int len = l.len[s];
    const int n_tiles = l.tile0[s + 1] - l.tile0[s];
    const int q0 = (n_tiles - 1 - (t - l.tile0[s])) * kGQ;  // the last queries, with the most keys, first
    const int64_t row0 = l.start[s];
    const int kvh = h / (a.n_heads / a.n_kv);
    const T *Q = static_cast<const T *>(a.Q) + row0 * a.q_stride + static_cast<int64_t>(h) * hd;
    const T *K = static_cast<const T *>(a.K) + row0 * a.k_stride + static_cast<int64_t>(kvh) * hd;
    const T *V = static_cast<const T *>(a.V) + row0 * a.v_stride + static_cast<int64_t>(kvh) * hd;
    const int tid = threadIdx.x, qi = tid >> 2, part = tid & 3;
    const bool valid = q0 + qi < len;
    for (int i = tid; i < kGQ * hd; i += 128) {
        const int r = i / hd, d = i - r * hd;
        Qs[r * pitch + d] = q0 + r < len ? widen(Q[(q0 + r) * a.q_stride + d]) * a.scale_log2 : 0.f;
    }
    const int lim = !valid ? 0 : a.causal ? q0 + qi + 1 : len;             // keys this query sees
    const int kend = a.causal ? min(len, q0 + kGQ) : len;                  // keys the tile sees
    float m = -INFINITY, sum = 0.f, o[kGOwn];
#pragma unroll
    for (int i = 0; i < kGOwn; ++i) o[i] = 0.f;
    for (int k0 = 0; k0 < kend; k0 += kGK) {
        const int nk = min(kGK, kend - k0);
        __syncthreads();
        for (int i = tid; i < nk * hd; i += 128) {
            const int r = i / hd, d = i - r * hd;
            Ks[r * pitch + d] = widen(K[(k0 + r) * a.k_stride + d]);
            Vs[r * pitch + d] = widen(V[(k0 + r) * a.v_stride + d]);
        }
        __syncthreads();
        const int see = min(nk, lim - k0);  // keys of the tile below the query's limit
        float sc[kGK / 4];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < kGK / 4; ++j) {
            const int k = part + 4 * j;
            sc[j] = -INFINITY;
            if (k < see) {
                float x = 0.f;
                for (int d = 0; d < hd; ++d) x = fmaf(Qs[qi * pitch + d], Ks[k * pitch + d], x);
                sc[j] = x;
            }
            top = fmaxf(top, sc[j]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m, top);
        const float al = mn == m ? 1.f : exp2f(m - mn);
        float ps = 0.f;
#pragma unroll
        for (int j = 0; j < kGK / 4; ++j) {
            const int k = part + 4 * j;
            const float p = k < see ? exp2f(sc[j] - (mn == -INFINITY ? 0.f : mn)) : 0.f;
            Ps[qi * (kGK + 1) + k] = p;
            ps += p;
        }
        ps += __shfl_xor_sync(0xffffffffu, ps, 1);
        ps += __shfl_xor_sync(0xffffffffu, ps, 2);
        sum = fmaf(sum, al, ps);
        m = mn;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kGOwn; ++i) o[i] *= al;
        for (int k = 0; k < see; ++k) {
            const float p = Ps[qi * (kGK + 1) + k];
#pragma unroll
            for (int i = 0; i < kGOwn; ++i)
                if (part + 4 * i < hd) o[i] = fmaf(p, Vs[k * pitch + part + 4 * i], o[i]);
        }
    }
    if (!valid) return;
    T *out = static_cast<T *>(a.out) + (row0 + q0 + qi) * a.o_stride + static_cast<int64_t>(h) * hd;
#pragma unroll
    for (int i = 0; i < kGOwn; ++i)
        if (part + 4 * i < hd) narrow(out + part + 4 * i, o[i] / sum);
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

template <class T, int N>
cudaError_t launch_general_n(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    PackedSeqs<N> l;
    fill_seqs(l, start, len, n, kGQ);
    const size_t smem = (static_cast<size_t>(kGQ + 2 * kGK) * (a.hd + 1) + kGQ * (kGK + 1)) * sizeof(float);
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(packed_general_kernel<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>((static_cast<size_t>(kGQ + 2 * kGK) * (kMaxHeadDim + 1) +
                                                      kGQ * (kGK + 1)) * sizeof(float)));
    });
    if (ce != cudaSuccess) return ce;
    const long long grid = static_cast<long long>(l.tile0[n]) * a.n_heads;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    packed_general_kernel<T, N><<<static_cast<unsigned>(grid), 128, smem, s>>>(a, l);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_general(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n, cudaStream_t s) {
    if (n <= 64) return launch_general_n<T, 64>(a, start, len, n, s);
    return launch_general_n<T, kPackedSeqs>(a, start, len, n, s);
}

}  // namespace

cudaError_t launch_packed(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n_seqs,
                          cudaStream_t s) {
    if (n_seqs <= 0 || n_seqs > kPackedSeqs) return cudaErrorInvalidValue;
    if (a.type == Elem::bf16) return launch_general<bf16>(a, start, len, n_seqs, s);
    if (a.type == Elem::f16) return launch_general<f16>(a, start, len, n_seqs, s);
    return cudaErrorInvalidValue;
}

}  // namespace pkv

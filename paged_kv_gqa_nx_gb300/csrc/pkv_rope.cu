// pkv_rope.cu -- rotary positions with several axes on packed query and key rows.
//
//   y[i]     = x[i] cos a_i - x[i + r] sin a_i
//   y[i + r] = x[i] sin a_i + x[i + r] cos a_i,    a_i = pos[axis_i][t] * f_i
//
// r pairs a head, each with a frequency f_i and one of the row's positions; the
// inverse turns by -a_i.
//
// The angle is kept in turns, as a fraction of 2^64: position * step mod 2^64
// is exact however far the position, for a step cut to whole 2^-64 turns (an
// f32 angle of position 100,000 is off by 4e-3, and f64 sines would take longer
// than the rows: 150 operations a pair at 1/50 of the f32 rate).  The nearest
// quarter turn is taken off in whole numbers, the rest, at most an eighth of a
// turn, goes through sincospi in f32.
//
// A thread takes one piece of a row's pairs (16 bytes of each half of a head)
// for several heads: its cosines and sines stay in registers, and all its loads
// are on their way before the sines, which the block computes once a row, are
// there.  What bounds it is one read and one write of every row.
#include "pkv_half.h"
#include "pkv_ragged.h"

#include <algorithm>

namespace pkv {
namespace {

constexpr int kThreads = 256, kMaxRows = 32, kHeads = 4;  // of a block, of a block, of a thread at a time

template <int B>
struct Piece;
template <>
struct Piece<16> {
    using type = uint4;
};
template <>
struct Piece<8> {
    using type = uint2;
};
template <>
struct Piece<4> {
    using type = uint32_t;
};
template <>
struct Piece<2> {
    using type = unsigned short;
};

__device__ __forceinline__ float widen(const float *p, int i) { return p[i]; }
__device__ __forceinline__ float widen(const bf16 *p, int i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float widen(const f16 *p, int i) { return __half2float(p[i]); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
template <class T>
__device__ __forceinline__ void put(T *p, float x) {
    narrow(p, x);
}

// cos and sin of a fraction of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t turn) {
    const uint64_t near = turn + (uint64_t{1} << 61);
    const uint32_t quarter = static_cast<uint32_t>(near >> 62);
    const float rest = static_cast<float>(static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62)));
    float s, c;
    sincospif(rest * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    return quarter & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// E elements a piece; the block takes n_tok rows, each by `lanes` threads a piece.
template <class T, int E>
__global__ void __launch_bounds__(kThreads, 3) rope_packed_kernel(const __grid_constant__ RopePacked a, int n_tok, int lanes) {
    using P = typename Piece<E * sizeof(T)>::type;
    extern __shared__ float2 cs[];  // [n_tok][n_pairs]
    const int r = a.n_pairs, tid = threadIdx.x, per_head = r / E, per_row = per_head * lanes;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * n_tok;
    const int rows = static_cast<int>(min(static_cast<int64_t>(n_tok), a.n_rows - row0));
    const int mine = tid / per_row, in_row = tid - mine * per_row, lane = in_row / per_head, pair = (in_row - lane * per_head) * E;
    const bool works = mine < rows;
    const int64_t row = row0 + (works ? mine : 0);
    const int heads = a.heads[0] + a.heads[1];
    auto src = [&](int h) {
        const int w = h >= a.heads[0];
        return static_cast<const T *>(a.src[w]) + row * a.src_stride[w] + static_cast<int64_t>(w ? h - a.heads[0] : h) * a.hd + pair;
    };
    auto dst = [&](int h) {
        const int w = h >= a.heads[0];
        return static_cast<T *>(a.dst[w]) + row * a.dst_stride[w] + static_cast<int64_t>(w ? h - a.heads[0] : h) * a.hd + pair;
    };
    P x[kHeads], y[kHeads];
    auto load = [&](int h0) {
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (works && h0 + k * lanes < heads) {
                const T *p = src(h0 + k * lanes);
                x[k] = *reinterpret_cast<const P *>(p);
                y[k] = *reinterpret_cast<const P *>(p + r);
            }
    };
    load(lane);
    for (int i = tid; i < rows * r; i += blockDim.x) {
        const int t = i / r, p = i - t * r;
        const int64_t pos = __ldg(a.pos + a.axis[p] * a.pos_stride + row0 + t);
        const uint64_t turn = static_cast<uint64_t>(pos) * a.step[p];
        cs[i] = cos_sin(a.inverse ? 0 - turn : turn);
    }
    __syncthreads();
    if (works) {
        float2 f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = cs[mine * r + pair + e];
        for (int h0 = lane; h0 < heads; h0 += kHeads * lanes) {
            if (h0 != lane) load(h0);
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                if (h0 + k * lanes >= heads) continue;
                const T *px = reinterpret_cast<const T *>(&x[k]), *py = reinterpret_cast<const T *>(&y[k]);
                P s, t;
                T *ps = reinterpret_cast<T *>(&s), *pt = reinterpret_cast<T *>(&t);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float p0 = widen(px, e), p1 = widen(py, e);
                    put(ps + e, fmaf(p0, f[e].x, -(p1 * f[e].y)));
                    put(pt + e, fmaf(p0, f[e].y, p1 * f[e].x));
                }
                T *p = dst(h0 + k * lanes);
                *reinterpret_cast<P *>(p) = s;
                *reinterpret_cast<P *>(p + r) = t;
            }
        }
    }
    // columns that are not turned
    const int rest = a.hd - 2 * r;
    if (rest > 0) {
        for (int i = tid; i < rows * heads * rest; i += blockDim.x) {
            const int t = i / (heads * rest), v = i - t * heads * rest, h = v / rest;
            const int w = h >= a.heads[0], hh = w ? h - a.heads[0] : h;
            if (a.src[w] == a.dst[w]) continue;
            const int64_t at = static_cast<int64_t>(hh) * a.hd + 2 * r + (v - h * rest);
            static_cast<T *>(a.dst[w])[(row0 + t) * a.dst_stride[w] + at] =
                static_cast<const T *>(a.src[w])[(row0 + t) * a.src_stride[w] + at];
        }
    }
}

template <class T, int E>
cudaError_t launch_e(const RopePacked &a, cudaStream_t s) {
    // As many threads a row as give each its kHeads heads at most, where that fits
    // a block; a block's rows fewer where the launch would not reach every SM twice.
    const int per_head = a.n_pairs / E, heads = a.heads[0] + a.heads[1];
    const int lanes = std::max(1, std::min((heads + kHeads - 1) / kHeads, kThreads / per_head));
    const int per_row = per_head * lanes;
    const int n_tok = std::max(1, std::min({kThreads / per_row, kMaxRows, a.n_rows / (2 * kSMs)}));
    const int64_t grid = (static_cast<int64_t>(a.n_rows) + n_tok - 1) / n_tok;
    const size_t smem = sizeof(float2) * n_tok * a.n_pairs;
    rope_packed_kernel<T, E><<<static_cast<unsigned>(grid), (n_tok * per_row + 31) / 32 * 32, smem, s>>>(a, n_tok, lanes);
    return cudaGetLastError();
}
template <class T>
cudaError_t launch_t(const RopePacked &a, cudaStream_t s) {
    // the largest piece on whose boundaries pairs, heads and rows all start
    uint64_t bits = static_cast<uint64_t>(a.n_pairs | a.hd) * sizeof(T);
    for (int w = 0; w < 2; ++w)
        if (a.heads[w])
            bits |= reinterpret_cast<uintptr_t>(a.src[w]) | reinterpret_cast<uintptr_t>(a.dst[w]) |
                    static_cast<uint64_t>(a.src_stride[w] | a.dst_stride[w]) * sizeof(T);
    if (bits % 16 == 0) return launch_e<T, 16 / sizeof(T)>(a, s);
    if (bits % 8 == 0) return launch_e<T, 8 / sizeof(T)>(a, s);
    return launch_e<T, 1>(a, s);
}

}  // namespace

cudaError_t launch_rope_packed(const RopePacked &a, cudaStream_t s) {
    if (a.n_rows <= 0 || a.n_pairs <= 0 || a.n_pairs > kRopePairs) return cudaErrorInvalidValue;
    if (a.type == Elem::f32) return launch_t<float>(a, s);
    return a.type == Elem::bf16 ? launch_t<bf16>(a, s) : launch_t<f16>(a, s);
}

}  // namespace pkv

// pkv_rope.cu -- rotary positions with several axes on packed query and key rows.
//
//   y[i]     = x[i] cos a_i - x[i + r] sin a_i
//   y[i + r] = x[i] sin a_i + x[i + r] cos a_i,    a_i = pos[axis_i][t] * f_i
//
// r pairs a head, each with a frequency f_i and one of the row's positions; the
// inverse turns by -a_i.
//
// The angle is kept in turns, as a fraction of 2^64: position * step mod 2^64
// is exact however far the position (an f32 angle of position 100,000 is off by
// 4e-3, and f64 sines would take longer than the rows: 150 operations a pair at
// 1/50 of the f32 rate).  The nearest quarter turn is taken off in whole
// numbers, the rest, at most an eighth of a turn, goes through sincospi in f32.
//
// A block computes its rows' sines once for all heads, with the first of its
// loads on the way, and turns each pair of 16-byte pieces in registers; what
// bounds it is one read and one write of every row.
#include "pkv_half.h"
#include "pkv_ragged.h"

namespace pkv {
namespace {

constexpr int kThreads = 256, kMaxRows = 4, kUnroll = 4;

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

// E elements a piece; n_tok rows a block.
template <class T, int E>
__global__ void __launch_bounds__(kThreads) rope_packed_kernel(const __grid_constant__ RopePacked a, int n_tok) {
    using P = typename Piece<E * sizeof(T)>::type;
    __shared__ float2 cs[kMaxRows][kRopePairs];
    const int r = a.n_pairs, tid = threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * n_tok;
    const int rows = static_cast<int>(min(static_cast<int64_t>(n_tok), a.n_rows - row0));
    const int per_head = r / E, heads = a.heads[0] + a.heads[1], per_row = heads * per_head, units = rows * per_row;

    struct At {
        const T *src;
        T *dst;
        int row, pair;
    };
    auto place = [&](int u) {
        const int row = u / per_row, v = u - row * per_row, h = v / per_head, j = v - h * per_head;
        const int w = h >= a.heads[0], hh = w ? h - a.heads[0] : h;
        const int64_t in_row = static_cast<int64_t>(hh) * a.hd + E * j;
        return At{static_cast<const T *>(a.src[w]) + (row0 + row) * a.src_stride[w] + in_row,
                  static_cast<T *>(a.dst[w]) + (row0 + row) * a.dst_stride[w] + in_row, row, E * j};
    };
    bool ready = false;
    for (int u0 = tid; u0 < units || !ready; u0 += kUnroll * kThreads) {
        P x[kUnroll], y[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * kThreads;
            if (u < units) {
                const At at = place(u);
                x[k] = *reinterpret_cast<const P *>(at.src);
                y[k] = *reinterpret_cast<const P *>(at.src + r);
            }
        }
        if (!ready) {
            for (int i = tid; i < rows * r; i += kThreads) {
                const int row = i / r, p = i - row * r;
                const int64_t pos = __ldg(a.pos + a.axis[p] * a.pos_stride + row0 + row);
                const uint64_t turn = static_cast<uint64_t>(pos) * a.step[p];
                cs[row][p] = cos_sin(a.inverse ? 0 - turn : turn);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int u = u0 + k * kThreads;
            if (u >= units) continue;
            const At at = place(u);
            P s, t;
            const T *px = reinterpret_cast<const T *>(&x[k]), *py = reinterpret_cast<const T *>(&y[k]);
            T *ps = reinterpret_cast<T *>(&s), *pt = reinterpret_cast<T *>(&t);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float2 f = cs[at.row][at.pair + e];
                const float p0 = widen(px, e), p1 = widen(py, e);
                put(ps + e, fmaf(p0, f.x, -(p1 * f.y)));
                put(pt + e, fmaf(p0, f.y, p1 * f.x));
            }
            *reinterpret_cast<P *>(at.dst) = s;
            *reinterpret_cast<P *>(at.dst + r) = t;
        }
    }
    // columns that are not turned
    const int rest = a.hd - 2 * r;
    if (rest > 0) {
        for (int i = tid; i < rows * heads * rest; i += kThreads) {
            const int row = i / (heads * rest), v = i - row * heads * rest, h = v / rest;
            const int w = h >= a.heads[0], hh = w ? h - a.heads[0] : h;
            if (a.src[w] == a.dst[w]) continue;
            const int64_t at = static_cast<int64_t>(hh) * a.hd + 2 * r + (v - h * rest);
            static_cast<T *>(a.dst[w])[(row0 + row) * a.dst_stride[w] + at] =
                static_cast<const T *>(a.src[w])[(row0 + row) * a.src_stride[w] + at];
        }
    }
}

template <class T, int E>
cudaError_t launch_e(const RopePacked &a, cudaStream_t s) {
    // A row a block while that fills the GPU no more than twice.
    const int n_tok = a.n_rows <= 8 * 152 ? 1 : kMaxRows;
    const int64_t grid = (static_cast<int64_t>(a.n_rows) + n_tok - 1) / n_tok;
    rope_packed_kernel<T, E><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, n_tok);
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

// pkv_ragged_rows.cu -- attention of few query rows over many keys, for packed
// bf16 / f16 rows (single tokens of cross attention, sequences behind a shared
// prefix, head widths and alignments that the tensor-core tiles do not take),
// and the join of partial records.
//
//   o[i, h] = sum_j p_ij v[j, h / G] / sum_j p_ij,  p_ij = 2^(s_ij - m_i),
//   s_ij = scale * log2(e) * <q[i, h], k[j, h / G]>
//
// A unit is 16 R query rows ((query, head of the group) pairs, which share
// their keys) of one kv head and one split of the keys: the shared prefix's
// rows, then the run's own.  Its four warps take the 16-key tiles in turn, each
// with its own ring of tiles (cp.async, no block-wide barrier in the loop), its
// own running maximum and sum; they are joined in shared memory at the end.
//
//   S [16 x 16] = Q K^T     m16n8k16, A and B by ldmatrix
//   O [16 x DP] += P V      A from S's accumulators, B by transposed ldmatrix
//
// What bounds it is reading K and V once: a tile of 8 KB (128-wide heads) has
// 16 MMAs for S and 32 for O.  So P is not rounded to 16 bits: it goes in as two
// pieces, p = hi + lo, each of the type, and what is left of p beyond them is
// 2^-16 (bf16) or 2^-22 of it.  The tensor core rounds its sums toward zero, so
// each tile's products have a sum of their own, added to O in f32.
// The reference maximum moves only where a tile's passes it by 2^8.
//
// Shared memory holds a tile's rows without padding; the 16-byte chunk c of
// row r sits at c ^ (r % 8), so that ldmatrix meets no bank twice.
#include "pkv_half.h"
#include "pkv_ragged.h"

namespace pkv {
namespace {

constexpr int kTile = 16;    // keys of a tile
constexpr int kRowWarps = 4;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kHeadroom = 8.f;

template <int DP, int R>
struct RowCfg {
    static constexpr int kPitch = DP * 2;                     // bytes of a row
    static constexpr int kStage = 2 * kTile * kPitch;         // K and V of a tile
    static constexpr int kStages = DP <= 64 ? 6 : 3;          // 128 KB of K and V on the way a SM
    static constexpr int kQ = 16 * R * kPitch;
    static constexpr size_t kSmem = static_cast<size_t>(kQ) + kRowWarps * kStages * kStage;
    static_assert(static_cast<size_t>(kRowWarps) * 16 * R * DP * 4 <= kSmem, "the warps' outputs");
};

__device__ __forceinline__ float pow2(float x) {  // 2^x to about 2^-22 relative; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// 16 bytes, or zeros where `there` is false (nothing is read then)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_launch_before() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void let_next_launch_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <class R, int N>
__device__ __forceinline__ int run_of(const RunList<R, N> &l, int u) {
    int lo = 0, hi = l.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.unit0[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Rows [16][DP] of K or V at tile `t0` (keys of the prefix, then of the run)
// into shared memory, zeros past `end`.
template <class T, int DP, bool kVec>
__device__ __forceinline__ void load_tile(unsigned char *dst, const T *pre, int64_t pre_stride, int n_pre, const T *own,
                                          int64_t own_stride, int t0, int end, int hd, int lane) {
    constexpr int kChunks = DP / 8;
    if constexpr (kVec) {
        constexpr int kRows = 32 / kChunks > 0 ? 32 / kChunks : 1;  // rows a pass of the warp covers
        constexpr int kAcross = kChunks > 32 ? kChunks / 32 : 1;
        static_assert(kAcross == 1, "a row is at most 32 chunks");
        const int c = lane % kChunks, r0 = lane / kChunks;
        if (8 * c >= hd) return;
        const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
#pragma unroll
        for (int i = 0; i < kTile / kRows; ++i) {
            const int r = r0 + i * kRows, key = t0 + r;
            const bool there = key < end;
            const int k = there ? key : t0;
            const T *src = k < n_pre ? pre + k * pre_stride : own + (k - n_pre) * own_stride;
            copy16(base + r * (DP * 2) + ((c ^ (r & 7)) << 4), src + 8 * c, there);
        }
    } else {
#pragma unroll 1
        for (int i = lane; i < kTile * DP; i += 32) {
            const int r = i / DP, d = i % DP, key = t0 + r;
            unsigned short x = 0;
            if (key < end && d < hd) {
                const T *src = key < n_pre ? pre + key * pre_stride : own + (key - n_pre) * own_stride;
                x = __ldg(reinterpret_cast<const unsigned short *>(src) + d);
            }
            *reinterpret_cast<unsigned short *>(dst + r * (DP * 2) + (((d >> 3) ^ (r & 7)) << 4) + 2 * (d & 7)) = x;
        }
    }
}

template <class T, int DP, int R, bool kVec, int N>
__global__ void __launch_bounds__(32 * kRowWarps, DP <= 128 ? 2 : 1)
    ragged_rows_kernel(const __grid_constant__ RaggedArgs a, const __grid_constant__ RunList<RaggedRun, N> l) {
    using C = RowCfg<DP, R>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float sm_m[kRowWarps][16 * R], sm_l[kRowWarps][16 * R];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3, mi = lane >> 3, mr = lane & 7;
    const int G = a.n_heads / a.n_kv, hd = a.hd;
    let_next_launch_start();

    // the unit: neighbouring blocks take the kv heads of the same keys
    const int ri = run_of(l, blockIdx.x);
    const RaggedRun run = l.run[ri];
    int u = blockIdx.x - l.unit0[ri];
    const int kvh = u % a.n_kv;
    u /= a.n_kv;
    const int rows = run.nq * G, n_blocks = ragged_row_units(rows, R);
    const int split = u / n_blocks, row0 = (u - split * n_blocks) * 16 * R;
    const int n_rows = min(16 * R, rows - row0);
    const int first = row0 / G, last = (row0 + n_rows - 1) / G;  // queries of the block

    const int total = a.n_pre + run.nk;
    const int per = ((total + run.ns - 1) / run.ns + kTile * kRowWarps - 1) / (kTile * kRowWarps) * (kTile * kRowWarps);
    const long long beg = static_cast<long long>(split) * per;
    const int kb = static_cast<int>(min(beg, static_cast<long long>(total)));
    const int seen = a.n_pre + min(run.nk, run.off + last + 1);  // keys that some row sees
    const int whole = a.n_pre + min(run.nk, run.off + first + 1);  // keys that all rows see
    const int end = static_cast<int>(min(static_cast<long long>(min(total, seen)), beg + per));

    const T *Kp = static_cast<const T *>(a.Kp) + static_cast<int64_t>(kvh) * hd;
    const T *Vp = static_cast<const T *>(a.Vp) + static_cast<int64_t>(kvh) * hd;
    const T *K = static_cast<const T *>(a.K) + run.k0 * a.k_stride + static_cast<int64_t>(kvh) * hd;
    const T *V = static_cast<const T *>(a.V) + run.k0 * a.v_stride + static_cast<int64_t>(kvh) * hd;

    unsigned char *Qs = smem, *ring = smem + C::kQ + warp * C::kStages * C::kStage;
    if (kVec && hd < DP) {  // columns that no copy writes
        const int pad = (DP - hd) / 8;
        for (int i = lane; i < C::kStages * 2 * kTile * pad; i += 32) {
            const int r = i / pad, ch = hd / 8 + i % pad;
            *reinterpret_cast<uint4 *>(ring + r * C::kPitch + ((ch ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        }
    }
    auto load = [&](int stage, int t0) {
        unsigned char *p = ring + stage * C::kStage;
        load_tile<T, DP, kVec>(p, Kp, a.kp_stride, a.n_pre, K, a.k_stride, t0, end, hd, lane);
        load_tile<T, DP, kVec>(p + C::kStage / 2, Vp, a.vp_stride, a.n_pre, V, a.v_stride, t0, end, hd, lane);
    };
    // the block's query rows, zeros behind them
    for (int i = tid; i < 16 * R * DP / 8; i += 32 * kRowWarps) {
        const int r = i / (DP / 8), ch = i % (DP / 8);
        const bool there = r < n_rows && 8 * ch < hd;
        const int qi = (row0 + (there ? r : 0)) / G, h = kvh * G + (row0 + (there ? r : 0)) % G;
        const T *q = static_cast<const T *>(a.Q) + (static_cast<int64_t>(run.q0) + qi) * a.q_stride + static_cast<int64_t>(h) * hd;
        unsigned char *dst = Qs + r * C::kPitch + ((ch ^ (r & 7)) << 4);
        if constexpr (kVec) {
            copy16(static_cast<uint32_t>(__cvta_generic_to_shared(dst)), q + (there ? 8 * ch : 0), there);
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (there && 8 * ch + k < hd)
                    w[k / 2] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short *>(q) + 8 * ch + k)) << (16 * (k & 1));
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    copies_commit();
    const int t_first = kb + warp * kTile, n_tiles = end > t_first ? (end - t_first + kTile * kRowWarps - 1) / (kTile * kRowWarps) : 0;
    auto fill = [&] {
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            if (i < n_tiles) load(i, t_first + i * kTile * kRowWarps);
            copies_commit();
        }
    };
    fill();
    copies_wait<C::kStages - 1>();
    __syncthreads();

    int lim[2 * R];  // rows g and g + 8 of each sixteen: keys that they see
    float m[2 * R], sum[2 * R], o[R][DP / 8][4];
#pragma unroll
    for (int x = 0; x < 2 * R; ++x) {
        const int r = row0 + 8 * x + g;
        lim[x] = r < rows ? a.n_pre + min(run.nk, run.off + r / G + 1) : 0;
    }
    bool careful = false;
    for (;;) {
#pragma unroll
        for (int x = 0; x < 2 * R; ++x) m[x] = -INFINITY, sum[x] = 0.f;
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
        int stage = 0;
#pragma unroll 1
        for (int it = 0; it < n_tiles; ++it) {
            const int t0 = t_first + it * kTile * kRowWarps;
            copies_wait<C::kStages - 2>();
            __syncwarp();  // the tile has landed, and the slot of the one before it has been read
            const int next = it + C::kStages - 1;
            if (next < n_tiles) load(stage == 0 ? C::kStages - 1 : stage - 1, t_first + next * kTile * kRowWarps);
            copies_commit();
            unsigned char *Ks = ring + stage * C::kStage, *Vs = Ks + C::kStage / 2;
            // ---- scores ----
            float sc[R][2][4];
#pragma unroll
            for (int x = 0; x < R; ++x)
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[x][i][0] = sc[x][i][1] = sc[x][i][2] = sc[x][i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                uint32_t kb4[4];  // keys mr (+ 8 by mi / 2), dims 16 k (+ 8 by mi % 2)
                ldsm4<false>(kb4, Ks + (mr + 8 * (mi >> 1)) * C::kPitch + (((2 * k + (mi & 1)) ^ mr) << 4));
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    uint32_t qa[4];
                    ldsm4<false>(qa, Qs + (16 * x + mr + 8 * (mi & 1)) * C::kPitch + (((2 * k + (mi >> 1)) ^ mr) << 4));
                    mma16<T>(sc[x][0], qa, kb4[0], kb4[1]);
                    mma16<T>(sc[x][1], qa, kb4[2], kb4[3]);
                }
            }
            // ---- softmax: reference, probabilities, sum ----
            uint32_t hi[R][4], lo[R][4];  // as A: keys (2c, 2c + 1) and + 8, rows g and g + 8
#pragma unroll
            for (int x = 0; x < R; ++x) {
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = t0 + 8 * i + 2 * c + (e & 1);
                        sc[x][i][e] = key < min(lim[2 * x + (e >> 1)], end) ? sc[x][i][e] * a.scale_log2 : -INFINITY;
                        top[e >> 1] = fmaxf(top[e >> 1], sc[x][i][e]);
                    }
                bool move = false;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    top[y] = fmaxf(top[y], __shfl_xor_sync(kAll, top[y], 1));
                    top[y] = fmaxf(top[y], __shfl_xor_sync(kAll, top[y], 2));
                    move = move || top[y] > m[2 * x + y] + kHeadroom || (m[2 * x + y] == -INFINITY && top[y] != -INFINITY);
                }
                if (__any_sync(kAll, move)) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float mn = fmaxf(m[2 * x + y], top[y]);
                        const float f = mn == m[2 * x + y] ? 1.f : pow2(m[2 * x + y] - mn);
                        m[2 * x + y] = mn;
                        sum[2 * x + y] *= f;
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i) o[x][i][2 * y] *= f, o[x][i][2 * y + 1] *= f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float ref = m[2 * x + (e >> 1)];
                        sc[x][i][e] = pow2(sc[x][i][e] - (ref == -INFINITY ? 0.f : ref));
                        sum[2 * x + (e >> 1)] += sc[x][i][e];
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t h = pack2(T{}, sc[x][i][2 * y], sc[x][i][2 * y + 1]);
                        hi[x][2 * i + y] = h;
                        lo[x][2 * i + y] = pack2(T{}, sc[x][i][2 * y] - half_of(T{}, h, 0), sc[x][i][2 * y + 1] - half_of(T{}, h, 1));
                    }
                }
            }
            // ---- output ----
            // Zero times an infinity is NaN: where some row does not see all of the
            // tile, values of V that are not finite are added one by one, to the rows
            // that see them, and leave the tile.
            if (careful || min(t0 + kTile, end) > whole) {
                constexpr uint32_t kE = std::is_same<T, bf16>::value ? 0x7f807f80u : 0x7c007c00u;
                constexpr uint32_t kOne = std::is_same<T, bf16>::value ? 0x00800080u : 0x04000400u;
                uint32_t seen = 0;  // a half's exponent is all ones where adding one to it reaches the sign bit
                for (int i = lane; i < kTile * DP / 8; i += 32) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(Vs + 16 * i);
                    seen |= ((y.x & kE) + kOne) | ((y.y & kE) + kOne) | ((y.z & kE) + kOne) | ((y.w & kE) + kOne);
                }
                if (__any_sync(kAll, seen & 0x80008000u)) {
#pragma unroll 1
                    for (int k = 0; k < kTile; ++k)
#pragma unroll
                        for (int x = 0; x < 2 * R; ++x) {
                            const float mine = k & 8 ? (k & 1 ? sc[x >> 1][1][2 * (x & 1) + 1] : sc[x >> 1][1][2 * (x & 1)])
                                                     : (k & 1 ? sc[x >> 1][0][2 * (x & 1) + 1] : sc[x >> 1][0][2 * (x & 1)]);
                            const float p = __shfl_sync(kAll, mine, (lane & ~3) | ((k & 7) >> 1));
                            if (t0 + k >= min(lim[x], end)) continue;
#pragma unroll
                            for (int i = 0; i < DP / 8; ++i) {
                                const uint32_t v = *reinterpret_cast<const uint32_t *>(Vs + k * C::kPitch + ((i ^ (k & 7)) << 4) + 4 * c);
                                float *at = &o[x >> 1][i][2 * (x & 1)];
                                if (not_finite<T>(v)) at[0] = fmaf(p, half_of(T{}, v, 0), at[0]);
                                if (not_finite<T>(v >> 16)) at[1] = fmaf(p, half_of(T{}, v, 1), at[1]);
                            }
                        }
                    __syncwarp();
                    for (int i = lane; i < kTile * DP / 2; i += 32) {
                        uint32_t *w = reinterpret_cast<uint32_t *>(Vs) + i;
                        if (not_finite<T>(*w)) *w &= 0xffff0000u;
                        if (not_finite<T>(*w >> 16)) *w &= 0xffffu;
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int k = 0; k < DP / 16; ++k) {
                uint32_t vb[4];  // keys mr (+ 8 by mi % 2), dims 16 k (+ 8 by mi / 2)
                ldsm4<true>(vb, Vs + (mr + 8 * (mi & 1)) * C::kPitch + (((2 * k + (mi >> 1)) ^ mr) << 4));
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    float t[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                    mma16<T>(t[0], hi[x], vb[0], vb[1]);
                    mma16<T>(t[1], hi[x], vb[2], vb[3]);
                    mma16<T>(t[0], lo[x], vb[0], vb[1]);
                    mma16<T>(t[1], lo[x], vb[2], vb[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][2 * k][e] += t[0][e], o[x][2 * k + 1][e] += t[1][e];
                }
            }
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }
        copies_wait<0>();
        // An infinity in V meets both pieces of P, of which one may be zero or
        // negative.  A warp that ends with a NaN goes over its keys again with an
        // eye on V; a row without such a value in sight comes out the same.
        if (careful) break;
        bool bad = false;
#pragma unroll
        for (int x = 0; x < R; ++x)
#pragma unroll
            for (int i = 0; i < DP / 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) bad = bad || o[x][i][e] != o[x][i][e];
        if (!__any_sync(kAll, bad)) break;
        careful = true;
        __syncwarp();
        fill();
    }

    // ---- the warps' parts ----
#pragma unroll
    for (int x = 0; x < 2 * R; ++x) {
        sum[x] += __shfl_xor_sync(kAll, sum[x], 1);
        sum[x] += __shfl_xor_sync(kAll, sum[x], 2);
        if (c == 0) {
            sm_m[warp][8 * x + g] = m[x];
            sm_l[warp][8 * x + g] = sum[x];
        }
    }
    __syncthreads();  // (all rings have been read)
    float *part = reinterpret_cast<float *>(smem);  // [warp][16 R][DP], a row's 16-byte chunks rotated by the row
#pragma unroll
    for (int x = 0; x < 2 * R; ++x) {
        const int r = 8 * x + g;
        float top = sm_m[0][r];
#pragma unroll
        for (int w = 1; w < kRowWarps; ++w) top = fmaxf(top, sm_m[w][r]);
        const float f = pow2(m[x] - (top == -INFINITY ? 0.f : top));
        float *dst = part + (warp * 16 * R + r) * DP;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
            *reinterpret_cast<float2 *>(dst + ((8 * i + 2 * c + 8 * r) & (DP - 1))) =
                make_float2(o[x >> 1][i][2 * (x & 1)] * f, o[x >> 1][i][2 * (x & 1) + 1] * f);
    }
    __syncthreads();
    const int64_t H = a.n_heads;
    for (int i = tid; i < n_rows * (DP / 4); i += 32 * kRowWarps) {
        const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
        if (d >= hd) continue;
        float top = sm_m[0][r], L = 0.f;
#pragma unroll
        for (int w = 1; w < kRowWarps; ++w) top = fmaxf(top, sm_m[w][r]);
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            L += sm_l[w][r] * pow2(sm_m[w][r] - (top == -INFINITY ? 0.f : top));
            const float4 y = *reinterpret_cast<const float4 *>(part + (w * 16 * R + r) * DP + ((d + 8 * r) & (DP - 1)));
            v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
        }
        const int qi = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
        if (run.rec0 >= 0) {
            const int64_t rec = (static_cast<int64_t>(run.rec0) + static_cast<int64_t>(qi) * run.ns + split) * H + h;
            if (d == 0) a.pm[rec] = top, a.pl[rec] = L;
            float *dst = a.pacc + rec * hd + d;
            if constexpr (kVec) {
                *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (d + k < hd) dst[k] = v[k];
            }
        } else {
            const float inv = L == 0.f ? 0.f : 1.f / L;  // a row without keys is 0
            T *dst = static_cast<T *>(a.out) + (static_cast<int64_t>(run.q0) + qi) * a.o_stride + static_cast<int64_t>(h) * hd + d;
            if constexpr (kVec) {
                *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2(T{}, v[0] * inv, v[1] * inv), pack2(T{}, v[2] * inv, v[3] * inv));
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (d + k < hd) narrow(dst + k, v[k] * inv);
            }
        }
    }
    wait_launch_before();  // so that the join behind this launch has both
}

// One (query, head) a block: its records' maximum and sum, then four warps add
// every fourth record's output.
template <class T, int N>
__global__ void __launch_bounds__(128)
    ragged_join_kernel(const __grid_constant__ RaggedArgs a, const __grid_constant__ RunList<JoinRun, N> l) {
    __shared__ float part[4][256];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % a.n_heads, t = blockIdx.x / a.n_heads;
    const int ri = run_of(l, t), qi = t - l.unit0[ri];
    const JoinRun run = l.run[ri];
    const int64_t own = run.rec0 + static_cast<int64_t>(qi) * run.ns, pre = run.pre0 + static_cast<int64_t>(qi) * run.pns;
    const int n = run.ns + run.pns;
    auto record = [&](int x) { return (x < run.ns ? own + x : pre + (x - run.ns)) * a.n_heads + h; };
    wait_launch_before();
    float top = -INFINITY;
    for (int x = lane; x < n; x += 32) top = fmaxf(top, a.pm[record(x)]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, s));
    const float ref = top == -INFINITY ? 0.f : top;
    float L = 0.f;
    for (int x = lane; x < n; x += 32) L += a.pl[record(x)] * pow2(a.pm[record(x)] - ref);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(kAll, L, s);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    float o[2][4] = {};
    const bool vec = (a.hd & 3) == 0;
    for (int x = warp; x < n; x += 4) {
        const int64_t r = record(x);
        if (a.pl[r] == 0.f) continue;  // no key of the split is seen: no output was written
        const float f = pow2(a.pm[r] - ref);
        const float *src = a.pacc + r * a.hd;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int d = 4 * lane + 128 * j;
            if (d >= a.hd) continue;
            if (vec) {
                const float4 y = *reinterpret_cast<const float4 *>(src + d);
                o[j][0] = fmaf(f, y.x, o[j][0]), o[j][1] = fmaf(f, y.y, o[j][1]);
                o[j][2] = fmaf(f, y.z, o[j][2]), o[j][3] = fmaf(f, y.w, o[j][3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (d + k < a.hd) o[j][k] = fmaf(f, src[d + k], o[j][k]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) part[warp][4 * lane + 128 * j + k] = o[j][k];
    __syncthreads();
    T *dst = static_cast<T *>(a.out) + (static_cast<int64_t>(run.q0) + qi) * a.o_stride + static_cast<int64_t>(h) * a.hd;
    for (int d = tid; d < a.hd; d += 128) narrow(dst + d, (part[0][d] + part[1][d] + part[2][d] + part[3][d]) * inv);
}

// A launch that may overlap the one in front of it, or a plain one.
template <class K, class... A>
cudaError_t start(K *kernel, long long grid, int threads, size_t smem, bool overlap, cudaStream_t s, const A &...args) {
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int DP, int R, bool kVec, int N>
cudaError_t rows_n(const RaggedArgs &a, const RaggedRun *runs, int32_t n, cudaStream_t s) {
    using C = RowCfg<DP, R>;
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(ragged_rows_kernel<T, DP, R, kVec, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(C::kSmem));
    });
    if (ce != cudaSuccess) return ce;
    RunList<RaggedRun, N> l;
    l.n = n;
    long long at = 0;
    for (int32_t i = 0; i < n; ++i) {
        l.run[i] = runs[i];
        l.unit0[i] = static_cast<int32_t>(at);
        at += static_cast<long long>(ragged_row_units(runs[i].nq * (a.n_heads / a.n_kv), R)) * runs[i].ns * a.n_kv;
        if (at > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    }
    l.unit0[n] = static_cast<int32_t>(at);
    return start(ragged_rows_kernel<T, DP, R, kVec, N>, at, 32 * kRowWarps, C::kSmem, a.overlap, s, a, l);
}
template <class T, int DP, int R, bool kVec>
cudaError_t rows_l(const RaggedArgs &a, const RaggedRun *runs, int32_t n, cudaStream_t s) {
    if (kVec && n <= kRaggedSmall) return rows_n<T, DP, R, kVec, kVec ? kRaggedSmall : kRaggedLarge>(a, runs, n, s);
    return rows_n<T, DP, R, kVec, kRaggedLarge>(a, runs, n, s);
}
template <class T>
cudaError_t rows_t(const RaggedArgs &a, const RaggedRun *runs, int32_t n, int wide, cudaStream_t s) {
    if (!a.vec) {
        if (a.hd <= 64) return rows_l<T, 64, 1, false>(a, runs, n, s);
        if (a.hd <= 128) return rows_l<T, 128, 1, false>(a, runs, n, s);
        return rows_l<T, 256, 1, false>(a, runs, n, s);
    }
    if (a.hd <= 64) return wide == 2 ? rows_l<T, 64, 2, true>(a, runs, n, s) : rows_l<T, 64, 1, true>(a, runs, n, s);
    if (a.hd <= 128) return wide == 2 ? rows_l<T, 128, 2, true>(a, runs, n, s) : rows_l<T, 128, 1, true>(a, runs, n, s);
    return rows_l<T, 256, 1, true>(a, runs, n, s);
}

template <class T, int N>
cudaError_t join_n(const RaggedArgs &a, const JoinRun *runs, int32_t n, cudaStream_t s) {
    RunList<JoinRun, N> l;
    l.n = n;
    long long at = 0;
    for (int32_t i = 0; i < n; ++i) {
        l.run[i] = runs[i];
        l.unit0[i] = static_cast<int32_t>(at);
        at += runs[i].nq;
        if (at > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    }
    l.unit0[n] = static_cast<int32_t>(at);
    return start(ragged_join_kernel<T, N>, at * a.n_heads, 128, 0, true, s, a, l);
}
template <class T>
cudaError_t join_t(const RaggedArgs &a, const JoinRun *runs, int32_t n, cudaStream_t s) {
    return n <= kRaggedSmall ? join_n<T, kRaggedSmall>(a, runs, n, s) : join_n<T, kRaggedLarge>(a, runs, n, s);
}

}  // namespace

cudaError_t launch_ragged_rows(const RaggedArgs &a, const RaggedRun *runs, int32_t n, int wide, cudaStream_t s) {
    if (n <= 0 || n > kRaggedLarge || a.hd > kMaxHeadDim) return cudaErrorInvalidValue;
    return a.type == Elem::bf16 ? rows_t<bf16>(a, runs, n, wide, s) : rows_t<f16>(a, runs, n, wide, s);
}

cudaError_t launch_ragged_join(const RaggedArgs &a, const JoinRun *runs, int32_t n, cudaStream_t s) {
    if (n <= 0 || n > kRaggedLarge || a.hd > kMaxHeadDim) return cudaErrorInvalidValue;
    return a.type == Elem::bf16 ? join_t<bf16>(a, runs, n, s) : join_t<f16>(a, runs, n, s);
}

}  // namespace pkv

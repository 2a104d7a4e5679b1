// pkv_ragged_rows.cu -- attention of few query rows over many keys, for packed
// bf16 / f16 rows (single tokens of cross attention, sequences behind a shared
// prefix, head widths and alignments that the tensor-core tiles do not take),
// and the join of partial records.
//
//   o[i, h] = sum_j p_ij v[j, h / G] / sum_j p_ij,  p_ij = 2^(s_ij - m_i),
//   s_ij = scale * log2(e) * <q[i, h], k[j, h / G]>
//
// A unit is 8 W query rows ((query, head of the group) pairs, which share their
// keys) of one kv head and one split of the keys: the shared prefix's rows,
// then the run's own.  Its two warps take the key tiles in turn, each with its
// own ring of tiles (cp.async, no block-wide barrier in the loop), its own running
// maximum and sum; they are joined in shared memory at the end.
//
// Small launches have a cluster of blocks a unit, a split each, and join them
// through each other's shared memory: one launch.  Larger ones write partial records
// that the join launch combines.
//
//   S^T [16 keys x 8] = K Q^T       m16n8k16, A by ldmatrix, B held in registers
//   O^T [16 dims x 8] += V^T P^T    A by transposed ldmatrix, B from S^T by movmatrix
//
// Keys and dims lie on the MMA's 16-row side, so that a single token's heads (4 of a group)
// fill half of the other side and not a quarter.  What has to bound it is reading K and V
// once: 8 KB a tile of 128-wide heads.  So P is not rounded to 16 bits: it goes in as two
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

// Warps of a block.  With two, and four blocks a SM, more units are in their first loads and last joins while
// others read than with four and two (64 runs of 170 keys, 8 kv heads: 9.1 us, 12.5).
constexpr int kRowWarps = 2;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kHeadroom = 8.f;

template <int DP, int W>
struct RowCfg {
    static constexpr int kTile = DP <= 64 ? 32 : 16;          // keys
    static constexpr int kPitch = DP * 2;                     // bytes of a row
    static constexpr int kStage = 2 * kTile * kPitch;         // K and V of a tile: 8 KB (16 of wide heads)
    static constexpr int kStages = 3;                         // 128 KB of K and V on the way a SM
    static constexpr size_t kRing = static_cast<size_t>(kRowWarps) * kStages * kStage;
    static constexpr int kPart = DP + 4;                      // floats of an output row of a warp's part
    static constexpr size_t kParts = sizeof(float) * (kRowWarps + 1) * 8 * W * kPart;  // the warps', and the block's
    static constexpr size_t kSmem = kRing > kParts ? kRing : kParts;
};

__device__ __forceinline__ float pow2(float x) {  // 2^x to about 2^-22 relative; 0 for -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
// or zeros where `there` is false (nothing is read then)
__device__ __forceinline__ void copy16_if(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
// Blocks of a cluster: their number, this one's place, a barrier over all of
// them, and shared memory of another.
__device__ __forceinline__ int cluster_size() {
    uint32_t x;
    asm("mov.u32 %0, %%cluster_nctarank;\n" : "=r"(x));
    return static_cast<int>(x);
}
__device__ __forceinline__ int cluster_rank() {
    uint32_t x;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(x));
    return static_cast<int>(x);
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t in_block(const void *p, int rank) {
    uint32_t y;
    asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(y) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    return y;
}
__device__ __forceinline__ float ld_block(uint32_t a) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(x) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ float4 ld_block4(uint32_t a) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(a) : "memory");
    return x;
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

// 8 x 8 elements of the warp, transposed.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

// Key rows as the two stretches they lie in, of one kv head.
template <class T>
struct KeyRows {
    const T *pre, *own;  // own: of the key behind the prefix
    int64_t pre_stride, own_stride;
    int n_pre;
    __device__ __forceinline__ const T *row(int key) const {
        return key < n_pre ? pre + key * pre_stride : own + (key - n_pre) * own_stride;
    }
};

// Rows [kTile][DP] of K or V from key `t0` on into shared memory, zeros from `end` on.
template <class T, int DP, int kTile, bool kVec>
__device__ __forceinline__ void load_tile(unsigned char *dst, const KeyRows<T> &rows, int t0, int end, int hd, int lane) {
    if constexpr (kVec) {
        constexpr int kChunks = DP / 8, kRows = 32 / kChunks;  // chunks of a row, rows that the warp copies at a time
        const int c = lane % kChunks, r0 = lane / kChunks;
        if (8 * c >= hd) return;
        const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(dst)) + r0 * (DP * 2);
        const bool pre = t0 + kTile <= rows.n_pre;
        if (t0 + kTile <= end && (pre || t0 >= rows.n_pre)) {  // rows at one stride
            const T *src = pre ? rows.pre + (t0 + r0) * rows.pre_stride : rows.own + (t0 - rows.n_pre + r0) * rows.own_stride;
            const int64_t step = (pre ? rows.pre_stride : rows.own_stride) * kRows;
            src += 8 * c;
#pragma unroll
            for (int i = 0; i < kTile / kRows; ++i, src += step)
                copy16(base + i * kRows * (DP * 2) + ((c ^ ((r0 + i * kRows) & 7)) << 4), src);
            return;
        }
#pragma unroll 1
        for (int i = 0; i < kTile / kRows; ++i) {
            const int r = r0 + i * kRows, key = t0 + r;
            copy16_if(base + i * kRows * (DP * 2) + ((c ^ (r & 7)) << 4), rows.row(key < end ? key : t0) + 8 * c, key < end);
        }
    } else {
#pragma unroll 1
        for (int i = lane; i < kTile * DP; i += 32) {
            const int r = i / DP, d = i % DP, key = t0 + r;
            unsigned short x = 0;
            if (key < end && d < hd) x = __ldg(reinterpret_cast<const unsigned short *>(rows.row(key)) + d);
            *reinterpret_cast<unsigned short *>(dst + r * (DP * 2) + (((d >> 3) ^ (r & 7)) << 4) + 2 * (d & 7)) = x;
        }
    }
}

template <class T, int DP, int W, bool kVec, int N>
__global__ void __launch_bounds__(32 * kRowWarps, DP <= 128 ? 4 : 2)
    ragged_rows_kernel(const __grid_constant__ RaggedArgs a, const __grid_constant__ RunList<RaggedRun, N> l) {
    using C = RowCfg<DP, W>;
    constexpr int kTile = C::kTile, kStep = kTile * kRowWarps, MT = kTile / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ float sm_m[kRowWarps][8 * W], sm_l[kRowWarps][8 * W];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3, mi = lane >> 3, mr = lane & 7;
    const int G = a.n_heads / a.n_kv, hd = a.hd;
    let_next_launch_start();

    // the unit: neighbouring blocks take the kv heads of the same keys
    const int n_ranks = cluster_size(), rank = cluster_rank(), unit = blockIdx.x / n_ranks;
    const int ri = run_of(l, unit);
    const RaggedRun run = l.run[ri];
    int u = unit - l.unit0[ri];
    const int kvh = u % a.n_kv;
    u /= a.n_kv;
    const int rows = run.nq * G, n_blocks = ragged_row_units(rows, W), ns = n_ranks > 1 ? n_ranks : run.ns;
    const int split = n_ranks > 1 ? rank : u / n_blocks, row0 = u % n_blocks * 8 * W;
    const int n_rows = min(8 * W, rows - row0);
    const int first = row0 / G, last = (row0 + n_rows - 1) / G;  // queries of the block

    const int n_pre = run.kind == kOnPrefix ? 0 : a.n_pre, total = n_pre + run.nk;
    // a cluster's blocks have few keys each: whole tiles; otherwise as many tiles a warp
    const int grain = n_ranks > 1 ? kTile : kStep, per = ((total + ns - 1) / ns + grain - 1) / grain * grain;
    const int kb = static_cast<int>(min(static_cast<long long>(split) * per, static_cast<long long>(total)));
    const int seen = n_pre + min(run.nk, run.off + last + 1);    // keys that some row sees
    const int whole = n_pre + min(run.nk, run.off + first + 1);  // keys that all rows see
    const int end = static_cast<int>(min(static_cast<long long>(seen), static_cast<long long>(kb) + per));

    const int64_t head = static_cast<int64_t>(kvh) * hd;
    KeyRows<T> K{static_cast<const T *>(a.Kp) + head, static_cast<const T *>(a.K) + run.k0 * a.k_stride + head, a.kp_stride, a.k_stride, n_pre};
    KeyRows<T> V{static_cast<const T *>(a.Vp) + head, static_cast<const T *>(a.V) + run.k0 * a.v_stride + head, a.vp_stride, a.v_stride, n_pre};
    if (run.kind == kOnPrefix) {
        K.own = K.pre, K.own_stride = K.pre_stride;
        V.own = V.pre, V.own_stride = V.pre_stride;
    }

    unsigned char *ring = smem + warp * C::kStages * C::kStage;
    if (kVec && hd < DP) {  // columns that no copy writes
        const int pad = (DP - hd) / 8;
        for (int i = lane; i < C::kStages * 2 * kTile * pad; i += 32) {
            const int r = i / pad, ch = hd / 8 + i % pad;
            *reinterpret_cast<uint4 *>(ring + r * C::kPitch + ((ch ^ (r & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        }
    }
    auto load = [&](int stage, int t0) {
        unsigned char *p = ring + stage * C::kStage;
        load_tile<T, DP, kTile, kVec>(p, K, t0, end, hd, lane);
        load_tile<T, DP, kTile, kVec>(p + C::kStage / 2, V, t0, end, hd, lane);
    };
    const int t_first = kb + warp * kTile, n_tiles = end > t_first ? (end - t_first + kStep - 1) / kStep : 0;
    auto fill = [&] {
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            if (i < n_tiles) load(i, t_first + i * kStep);
            copies_commit();
        }
    };
    fill();

    // Q as B: query rows g of each eight, dims 2c, 2c + 1 and + 8 of each sixteen
    uint32_t q[W][DP / 16][2];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int r = 8 * w + g;
        const bool there = r < n_rows;
        const int qi = (row0 + (there ? r : 0)) / G, h = kvh * G + (row0 + (there ? r : 0)) % G;
        const T *src = static_cast<const T *>(a.Q) + (static_cast<int64_t>(run.q0) + qi) * a.q_stride + static_cast<int64_t>(h) * hd;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = 16 * k + 8 * e + 2 * c;
                uint32_t x = 0;
                if (there && d < hd) {
                    if constexpr (kVec) {
                        x = __ldg(reinterpret_cast<const unsigned int *>(src + d));
                    } else {
                        x = __ldg(reinterpret_cast<const unsigned short *>(src) + d);
                        if (d + 1 < hd) x |= static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short *>(src) + d + 1)) << 16;
                    }
                }
                q[w][k][e] = x;
            }
    }
    int lim[W][2];  // rows 2c and 2c + 1 of each eight: keys that they see
    float m[W][2], sum[W][2], o[W][DP / 16][4];
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int r = row0 + 8 * w + 2 * c + y;
            lim[w][y] = r < rows ? min(end, n_pre + min(run.nk, run.off + r / G + 1)) : 0;
        }
    bool careful = false;
    for (;;) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            m[w][0] = m[w][1] = -INFINITY;
            sum[w][0] = sum[w][1] = 0.f;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) o[w][i][0] = o[w][i][1] = o[w][i][2] = o[w][i][3] = 0.f;
        }
        int stage = 0;
#pragma unroll 1
        for (int it = 0; it < n_tiles; ++it) {
            const int t0 = t_first + it * kStep;
            copies_wait<C::kStages - 2>();
            __syncwarp();  // the tile has landed, and the slot of the one before it has been read
            const int next = it + C::kStages - 1;
            if (next < n_tiles) load(stage == 0 ? C::kStages - 1 : stage - 1, t_first + next * kStep);
            copies_commit();
            unsigned char *Ks = ring + stage * C::kStage, *Vs = Ks + C::kStage / 2;
            // ---- scores: keys g and g + 8 of each sixteen, rows 2c and 2c + 1 ----
            float sc[MT][W][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int w = 0; w < W; ++w) sc[t][w][0] = sc[t][w][1] = sc[t][w][2] = sc[t][w][3] = 0.f;
#pragma unroll
            for (int k = 0; k < DP / 16; ++k)
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    uint32_t ka[4];  // keys mr (+ 8 by mi % 2), dims 16 k (+ 8 by mi / 2)
                    ldsm4<false>(ka, Ks + (16 * t + mr + 8 * (mi & 1)) * C::kPitch + (((2 * k + (mi >> 1)) ^ mr) << 4));
#pragma unroll
                    for (int w = 0; w < W; ++w) mma16<T>(sc[t][w], ka, q[w][k][0], q[w][k][1]);
                }
            // ---- softmax: reference, probabilities, sum ----
            const bool part = t0 + kTile > whole || t0 + kTile > end;
            uint32_t hi[MT][W][2], lo[MT][W][2];  // as B
#pragma unroll
            for (int w = 0; w < W; ++w) {
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[t][w][e] *= a.scale_log2;
                        if (part && t0 + 16 * t + 8 * (e >> 1) + g >= lim[w][e & 1]) sc[t][w][e] = -INFINITY;
                        top[e & 1] = fmaxf(top[e & 1], sc[t][w][e]);
                    }
                if (__any_sync(kAll, top[0] > m[w][0] + kHeadroom || top[1] > m[w][1] + kHeadroom)) {  // (-inf: any score passes it)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top[y] = fmaxf(top[y], __shfl_xor_sync(kAll, top[y], x));
                        const float mn = fmaxf(m[w][y], top[y]);
                        const float f = mn == m[w][y] ? 1.f : pow2(m[w][y] - mn);
                        m[w][y] = mn;
                        sum[w][y] *= f;
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) o[w][i][y] *= f, o[w][i][2 + y] *= f;
                    }
                }
                const float ref[2] = {m[w][0] == -INFINITY ? 0.f : m[w][0], m[w][1] == -INFINITY ? 0.f : m[w][1]};
#pragma unroll
                for (int t = 0; t < MT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[t][w][e] = pow2(sc[t][w][e] - ref[e & 1]);
                        sum[w][e & 1] += sc[t][w][e];
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float p0 = sc[t][w][2 * e], p1 = sc[t][w][2 * e + 1];
                        const uint32_t h = pack2(T{}, p0, p1);
                        hi[t][w][e] = turned(h);
                        lo[t][w][e] = turned(pack2(T{}, p0 - half_of(T{}, h, 0), p1 - half_of(T{}, h, 1)));
                    }
                }
            }
            // ---- output: dims g and g + 8 of each sixteen, rows 2c and 2c + 1 ----
            // Zero times an infinity is NaN: where some row does not see all of the
            // tile, values of V that are not finite are added one by one, to the rows
            // that see them, and leave the tile.
            if (careful || min(t0 + kTile, end) > whole) {
                constexpr uint32_t kE = std::is_same<T, bf16>::value ? 0x7f807f80u : 0x7c007c00u;
                constexpr uint32_t kOne = std::is_same<T, bf16>::value ? 0x00800080u : 0x04000400u;
                uint32_t odd = 0;  // a half's exponent is all ones where adding one to it reaches the sign bit
                for (int i = lane; i < kTile * DP / 8; i += 32) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(Vs + 16 * i);
                    odd |= ((y.x & kE) + kOne) | ((y.y & kE) + kOne) | ((y.z & kE) + kOne) | ((y.w & kE) + kOne);
                }
                if (__any_sync(kAll, odd & 0x80008000u)) {
#pragma unroll 1
                    for (int k = 0; k < kTile; ++k)
#pragma unroll
                        for (int w = 0; w < W; ++w)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                float mine = sc[0][w][y];
                                if (k & 8) mine = sc[0][w][2 + y];
                                if constexpr (MT == 2) {
                                    if (k & 16) mine = k & 8 ? sc[1][w][2 + y] : sc[1][w][y];
                                }
                                const float p = __shfl_sync(kAll, mine, 4 * (k & 7) + c);
                                if (t0 + k >= lim[w][y]) continue;
#pragma unroll
                                for (int i = 0; i < DP / 8; ++i) {
                                    const uint32_t v = *reinterpret_cast<const unsigned short *>(Vs + k * C::kPitch + ((i ^ (k & 7)) << 4) + 2 * g);
                                    float &at = o[w][i >> 1][2 * (i & 1) + y];
                                    if (not_finite<T>(v)) at = fmaf(p, half_of(T{}, v, 0), at);
                                }
                            }
                    __syncwarp();
                    for (int i = lane; i < kTile * DP / 2; i += 32) {
                        uint32_t *v = reinterpret_cast<uint32_t *>(Vs) + i;
                        if (not_finite<T>(*v)) *v &= 0xffff0000u;
                        if (not_finite<T>(*v >> 16)) *v &= 0xffffu;
                    }
                    __syncwarp();
                }
            }
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                float t4[W][4];
#pragma unroll
                for (int w = 0; w < W; ++w) t4[w][0] = t4[w][1] = t4[w][2] = t4[w][3] = 0.f;
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    uint32_t va[4];  // keys mr (+ 8 by mi / 2), dims 16 i (+ 8 by mi % 2)
                    ldsm4<true>(va, Vs + (16 * t + mr + 8 * (mi >> 1)) * C::kPitch + (((2 * i + (mi & 1)) ^ mr) << 4));
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        mma16<T>(t4[w], va, hi[t][w][0], hi[t][w][1]);
                        mma16<T>(t4[w], va, lo[t][w][0], lo[t][w][1]);
                    }
                }
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[w][i][e] += t4[w][e];
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
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) bad = bad || o[w][i][e] != o[w][i][e];
        if (!__any_sync(kAll, bad)) break;
        careful = true;
        __syncwarp();
        fill();
    }

    // ---- the warps' parts ----
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) sum[w][y] += __shfl_xor_sync(kAll, sum[w][y], x);
            if (g == 0) {
                sm_m[warp][8 * w + 2 * c + y] = m[w][y];
                sm_l[warp][8 * w + 2 * c + y] = sum[w][y];
            }
        }
    __syncthreads();  // (all rings have been read)
    float *out = reinterpret_cast<float *>(smem);  // [warp][8 W][kPart]
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int r = 8 * w + 2 * c + y;
            float top = sm_m[0][r];
#pragma unroll
            for (int x = 1; x < kRowWarps; ++x) top = fmaxf(top, sm_m[x][r]);
            const float f = pow2(m[w][y] - (top == -INFINITY ? 0.f : top));
            float *dst = out + (warp * 8 * W + r) * C::kPart + g;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                dst[16 * i] = o[w][i][y] * f;
                dst[16 * i + 8] = o[w][i][2 + y] * f;
            }
        }
    __syncthreads();
    // four dims of a row, over the block's warps
    auto of_block = [&](int r, int d, float &top, float &L, float (&v)[4]) {
        top = sm_m[0][r];
        L = 0.f;
#pragma unroll
        for (int w = 1; w < kRowWarps; ++w) top = fmaxf(top, sm_m[w][r]);
        v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            L += sm_l[w][r] * pow2(sm_m[w][r] - (top == -INFINITY ? 0.f : top));
            const float4 y = *reinterpret_cast<const float4 *>(out + (w * 8 * W + r) * C::kPart + d);
            v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
        }
    };
    const int64_t H = a.n_heads;
    float *joined = out + kRowWarps * 8 * W * C::kPart;
    if (n_ranks > 1) {
        for (int i = tid; i < n_rows * (DP / 4); i += 32 * kRowWarps) {
            const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
            if (d >= hd) continue;
            float top, L, v[4];
            of_block(r, d, top, L, v);
            *reinterpret_cast<float4 *>(joined + r * C::kPart + d) = make_float4(v[0], v[1], v[2], v[3]);
            if (d == 0) joined[r * C::kPart + DP] = top, joined[r * C::kPart + DP + 1] = L;
        }
        cluster_sync();
    }
    wait_launch_before();  // so that the join behind this launch has both
    for (int i = (n_ranks > 1 ? rank * 32 * kRowWarps : 0) + tid; i < n_rows * (DP / 4); i += n_ranks * 32 * kRowWarps) {
        const int r = i / (DP / 4), d = 4 * (i % (DP / 4));
        if (d >= hd) continue;
        float top, L, v[4];
        if (n_ranks > 1) {
            top = -INFINITY, L = 0.f;
            v[0] = v[1] = v[2] = v[3] = 0.f;
            for (int x = 0; x < n_ranks; ++x) top = fmaxf(top, ld_block(in_block(joined + r * C::kPart + DP, x)));
            for (int x = 0; x < n_ranks; ++x) {
                const uint32_t at = in_block(joined + r * C::kPart, x);
                const float f = pow2(ld_block(at + 4 * DP) - (top == -INFINITY ? 0.f : top));
                const float4 y = ld_block4(at + 4 * d);
                L += f * ld_block(at + 4 * DP + 4);
                v[0] = fmaf(f, y.x, v[0]), v[1] = fmaf(f, y.y, v[1]), v[2] = fmaf(f, y.z, v[2]), v[3] = fmaf(f, y.w, v[3]);
            }
        } else {
            of_block(r, d, top, L, v);
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
            continue;
        }
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
    if (n_ranks > 1) cluster_sync();  // the others may still read this block's part
}

// The records of a (query, head), by one warp or, where there are few of them, by
// the four of a block (`together`).  A lane takes a record's maximum and sum, then
// the records' outputs are added, kBatch on the way at a time: what it takes is
// the latency of two dependent reads, and a warp's own instructions (64 queries
// behind 8,192 keys, 14 records of each of 2,048 rows and heads: the three launches
// take 47 us with one read after another, 39 with four at a time by four warps, 35 so).
template <class T, int N, int J>  // J: 128 dims each
__global__ void __launch_bounds__(128, 4)
    ragged_join_kernel(const __grid_constant__ RaggedArgs a, const __grid_constant__ RunList<JoinRun, N> l, int together) {
    constexpr int kBatch = J == 1 ? 12 : 6;
    __shared__ __align__(16) float part[4][128 * J];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t H = a.n_heads;
    const uint32_t item = together ? blockIdx.x : 4 * blockIdx.x + warp;  // (rows times heads stay below 2^31)
    const int first = together ? warp : 0, step = together ? 4 : 1;  // of this warp's records
    const int t = static_cast<int>(item / static_cast<uint32_t>(a.n_heads)), h = static_cast<int>(item % static_cast<uint32_t>(a.n_heads));
    if (t >= l.unit0[l.n]) return;  // (whole blocks, where warps meet below)
    const int ri = run_of(l, t), qi = t - l.unit0[ri];
    const JoinRun run = l.run[ri];
    const int64_t own = (run.rec0 + static_cast<int64_t>(qi) * run.ns) * H + h, pre = (run.pre0 + static_cast<int64_t>(qi) * run.pns) * H + h;
    const int n = run.ns + run.pns;
    auto record = [&](int x) { return (x < run.ns ? own : pre - run.ns * H) + x * H; };
    const float *own_out = a.pacc + own * a.hd + 4 * lane, *pre_out = a.pacc + (pre - run.ns * H) * a.hd + 4 * lane;
    const int64_t out_step = H * a.hd;
    wait_launch_before();
    float m0 = -INFINITY, l0 = 0.f;  // of the lane's first record
    if (lane < n) {
        const int64_t r = record(lane);
        m0 = __ldcg(a.pm + r), l0 = __ldcg(a.pl + r);
    }
    float top = m0;
    for (int x = 32 + lane; x < n; x += 32) top = fmaxf(top, __ldcg(a.pm + record(x)));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, s));
    const float ref = top == -INFINITY ? 0.f : top;
    float L = 0.f, o[J][4] = {};
    const bool vec = (a.hd & 3) == 0;
    for (int x0 = 0; x0 < n; x0 += 32) {
        if (x0 > 0) {
            m0 = -INFINITY, l0 = 0.f;
            if (x0 + lane < n) {
                const int64_t r = record(x0 + lane);
                m0 = __ldcg(a.pm + r), l0 = __ldcg(a.pl + r);
            }
        }
        // A record without a key in sight (sum 0) holds no output and is passed over: -1.  One whose weight
        // is 0 counts: what it holds may be infinite, and 0 times that is NaN however the keys are split.
        const float f = l0 == 0.f ? -1.f : pow2(m0 - ref);
        L = fmaf(l0, f, L);
        const int m = min(32, n - x0);
        for (int y0 = first; y0 < m; y0 += kBatch * step) {
            float w[kBatch];
            float4 v[kBatch][J];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const int y = y0 + e * step;
                w[e] = __shfl_sync(kAll, f, y & 31);
                if (y >= m) w[e] = -1.f;
                const int x = x0 + min(y, m - 1);
                const float *src = (x < run.ns ? own_out : pre_out) + x * out_step;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    v[e][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w[e] < 0.f) continue;
                    const int left = a.hd - 4 * lane - 128 * j;
                    if (vec) {
                        if (left > 0) v[e][j] = __ldcg(reinterpret_cast<const float4 *>(src + 128 * j));
                    } else {
                        if (left > 0) v[e][j].x = __ldcg(src + 128 * j);
                        if (left > 1) v[e][j].y = __ldcg(src + 128 * j + 1);
                        if (left > 2) v[e][j].z = __ldcg(src + 128 * j + 2);
                        if (left > 3) v[e][j].w = __ldcg(src + 128 * j + 3);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    o[j][0] = fmaf(w[e], v[e][j].x, o[j][0]), o[j][1] = fmaf(w[e], v[e][j].y, o[j][1]);
                    o[j][2] = fmaf(w[e], v[e][j].z, o[j][2]), o[j][3] = fmaf(w[e], v[e][j].w, o[j][3]);
                }
        }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(kAll, L, s);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    T *dst = static_cast<T *>(a.out) + (static_cast<int64_t>(run.q0) + qi) * a.o_stride + static_cast<int64_t>(h) * a.hd;
#pragma unroll
    for (int j = 0; j < J; ++j)
        *reinterpret_cast<float4 *>(&part[warp][4 * lane + 128 * j]) = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
    if (together) {
        __syncthreads();
        for (int d = threadIdx.x; d < a.hd; d += 128) narrow(dst + d, (part[0][d] + part[1][d] + part[2][d] + part[3][d]) * inv);
    } else {
        __syncwarp();
        for (int d = lane; d < a.hd; d += 32) narrow(dst + d, part[warp][d] * inv);
    }
}

// A launch that may overlap the one in front of it, or a plain one.
template <class K, class... A>
cudaError_t start(K *kernel, long long grid, int cluster, int threads, size_t smem, bool overlap, cudaStream_t s, const A &...args) {
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2] = {};
    if (overlap) {
        at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(cluster);
        at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    cfg.attrs = at;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <class T, int DP, int W, bool kVec, int N>
cudaError_t rows_n(const RaggedArgs &a, const RaggedRun *runs, int32_t n, cudaStream_t s) {
    using C = RowCfg<DP, W>;
    static PerDeviceOnce configured;  // the attribute is per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        return cudaFuncSetAttribute(ragged_rows_kernel<T, DP, W, kVec, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(C::kSmem));
    });
    if (ce != cudaSuccess) return ce;
    RunList<RaggedRun, N> l;
    l.n = n;
    long long at = 0;
    for (int32_t i = 0; i < n; ++i) {
        l.run[i] = runs[i];
        l.unit0[i] = static_cast<int32_t>(at);
        at += static_cast<long long>(ragged_row_units(runs[i].nq * (a.n_heads / a.n_kv), W)) * runs[i].ns * a.n_kv;
        if (at > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    }
    l.unit0[n] = static_cast<int32_t>(at);
    return start(ragged_rows_kernel<T, DP, W, kVec, N>, at * a.cluster, a.cluster, 32 * kRowWarps, C::kSmem, a.overlap, s, a, l);
}
template <class T, int DP, int W, bool kVec>
cudaError_t rows_l(const RaggedArgs &a, const RaggedRun *runs, int32_t n, cudaStream_t s) {
    if (kVec && n <= kRaggedSmall) return rows_n<T, DP, W, kVec, kVec ? kRaggedSmall : kRaggedLarge>(a, runs, n, s);
    return rows_n<T, DP, W, kVec, kRaggedLarge>(a, runs, n, s);
}
template <class T, int DP>
cudaError_t rows_d(const RaggedArgs &a, const RaggedRun *runs, int32_t n, int wide, cudaStream_t s) {
    if (!a.vec) return wide == 2 ? rows_l<T, DP, 2, false>(a, runs, n, s) : cudaErrorInvalidValue;
    if (wide == 1) return rows_l<T, DP, 1, true>(a, runs, n, s);
    if (wide == 2) return rows_l<T, DP, 2, true>(a, runs, n, s);
    if constexpr (DP <= 128) return rows_l<T, DP, 4, true>(a, runs, n, s);
    return cudaErrorInvalidValue;
}
template <class T>
cudaError_t rows_t(const RaggedArgs &a, const RaggedRun *runs, int32_t n, int wide, cudaStream_t s) {
    if (a.hd <= 64) return rows_d<T, 64>(a, runs, n, wide, s);
    if (a.hd <= 128) return rows_d<T, 128>(a, runs, n, wide, s);
    return rows_d<T, 256>(a, runs, n, wide, s);
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
    const int together = at * a.n_heads <= 2 * kSMs;
    const long long grid = together ? at * a.n_heads : (at * a.n_heads + 3) / 4;
    if (a.hd > 128) return start(ragged_join_kernel<T, N, 2>, grid, 1, 128, 0, true, s, a, l, together);
    return start(ragged_join_kernel<T, N, 1>, grid, 1, 128, 0, true, s, a, l, together);
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

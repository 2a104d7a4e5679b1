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
#include "pkv_softmax_tc.h"
#include "pkv_tcgen05.h"
#include "pkv_tma.h"

#include <cuda_fp16.h>
#include <type_traits>

namespace pkv {
namespace {

using f16 = __half;
using namespace tc;

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

// ------------------------------------------------------------ tensor cores ----
//
// A piece of work = two tiles of 128 query rows of one sequence (two softmax
// chains that share every K/V tile).  The grid has a block per piece, and a
// block that runs takes over further pieces from blocks that have not started
// (the loading warp asks once a piece's last load is on its way), so that the loads of the next piece and its
// first QK run under the last softmax and the output of this one: a block per
// piece spent ~14,000 of ~29,000 clocks of an average piece of a ragged batch
// outside its loop.  A tile is 128/P consecutive tokens x P heads of
// one kv head, P the largest power of two (at most 16) that divides the group,
// so the rows of a tile need the same keys and a causal tile's masked corner
// is only 128/P tokens deep.  Row m of chain c is token m / P, head m % P, TMEM
// lane m and thread m of warps 4c .. 4c + 3.
//
//   S_c [128 x 128] = Q_c K_j^T    A, B from shared memory (K-major)
//   O_c [128 x D]  += P_c V_j      A from TMEM (P over S, two values a column),
//                                  B from shared memory (V as stored: MN-major)
//
// Warps 8 and 10 issue chain 0's and chain 1's MMAs, warp 9 the TMA loads
// (Q once; K_0, V_0, K_1, ... through a ring of slots).  A chain runs QK(j),
// softmax(j), PV(j) and QK(j + 1) back to back; while one chain's softmax runs,
// the tensor core works on the other's products.  The issuing warps take turns:
// without turns the core interleaved both chains' MMAs, so both softmaxes ran
// at once and then both waited.  P of tile j is read by PV(j) before QK(j + 1),
// issued by the same thread, writes over it.
//
// Probabilities are rounded to the operand type (half a step: 2^-8 relative to p
// in bf16, 2^-11 in f16 and 2^-25 absolute for f16 below 2^-14; the outputs, of the
// same type, are rounded by as much); sums use them unrounded.  On random rows
// the output is 1.15 to 1.36 times as far from 64 bits as one of f32 probabilities.
// The reference maximum moves, and O is rescaled, only where a tile's maximum
// passes it by more than 2^8, which keeps every p at most 256.
//
// The tensor core rounds its f32 sums toward zero, which on values of one sign
// takes 7e-9 of an output a key: 1.1e-4 of it at 16,384 keys, 4.3e-4 at 65,536 and
// 1.3e-3 at 200,000, past f16's half step (4.9e-4).  In sequences of more than
// kLongKeys the leading part of O therefore goes to registers after every kHold key
// tiles, a byte a dim in units of the row's own power of two, and O goes on from the
// rest: 7.3e-5 at 65,536 keys and 8.8e-5 at 200,000.  It costs 2 to 3% of such a
// launch (40,000 tokens: 7.93 -> 8.16 ms), and in a kernel for all lengths 2% of a
// ragged batch, so that a launch without a long sequence has an instance without
// it.  What a sequence's rows return goes by its own length alone.
//
// A zero probability times an infinity is NaN, so V rows behind a sequence's
// end or in a query's future must not hold one: on the (at most two) tiles
// that some row of the CTA does not see whole, the compute threads of one chain
// replace values that are not finite by 0 and, where they found any, every
// thread adds those products for the keys that its row does see.
//
// Measured: 16,384 tokens, causal, 32 heads over 8 of 128, f16: 1,356 us (1,622
// TFLOP/s; 2,400 clocks a pair of tiles and key tile, of which the MMAs take
// 2,048).  24 prompts of 16 .. 4,096, bf16: 84 us, 4.4 key tiles a piece, 3,000
// clocks each and 5,000 to 6,000 a piece for its first scores and its output.
// 64-wide heads, 16 prompts of 64 .. 1,024: 49 to 57 us, 2,600 clocks a key tile
// (a third score buffer, with scores two steps ahead, gave 58).  Also not taken:
// pieces of one tile (ragged 114: twice the reads of K and V), a part of the
// exponentials on the FMA units (1,409 us and more on the long prompt).
constexpr int kKeys = 128;  // keys per tile
constexpr int kTcThreads = 384;
constexpr int kWarpMma0 = 8, kWarpLoad = 9, kWarpSpare = 11;  // warp 10: chain 1's MMAs
// registers per thread: at launch, then of warps 8-11 and of the compute warps
constexpr int kTcLaunchRegs = 168, kTcOtherRegs = 88, kTcComputeRegs = 208;
static_assert(256 * kTcComputeRegs + 128 * kTcOtherRegs <= kTcThreads * kTcLaunchRegs, "register split");
constexpr uint32_t kTcCols = 512;           // O_c at c * 128, S_c / P_c at 256 + c * 128
constexpr int kPassLeft = 2;                // MMAs of QK still to issue when the turn passes
constexpr float kGrow = 8.f;                // log2 headroom of the reference maximum
constexpr int kLongKeys = 16384;            // in a longer sequence O's leading part is set aside
constexpr int kHold = 64;                   // after every so many key tiles

template <int D>
struct TcCfg {
    static constexpr uint32_t kTile = kKeys * D * 2;         // bytes of a Q, K or V tile
    static constexpr uint32_t kBlock = kKeys * 128;          // 64 columns of it
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr size_t kSmem = (2 + kSlots) * kTile + 1024;  // + alignment slack
};

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
        : "memory");
}
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
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n" : "=r"(r) : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
    return r;
}
// Shared-memory matrix descriptor of a V tile, MN-major with 128-byte swizzle:
// 64 columns of a key in 128 bytes, 8 keys 1024 bytes apart (stride offset),
// the next 64 columns kBlock bytes on (leading offset).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t block) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(block >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
// Instruction descriptor: f32 accumulator, M = 128, A K-major, B K- or MN-major.
template <class T>
__host__ __device__ constexpr uint32_t idesc16(uint32_t n, bool b_mn) {
    constexpr uint32_t f = std::is_same<T, bf16>::value ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// Asks for the index of a block of this grid that has not started yet: if there
// is one it will not start, and this block does its work.  The 16-byte answer
// comes with 16 bytes of the barrier's transaction count.
__device__ __forceinline__ void ask_work(uint32_t answer, uint32_t mbar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
                     answer),
                 "r"(mbar)
                 : "memory");
}
// The answer: a block's index, or -1.
__device__ __forceinline__ int work_of(uint32_t answer) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}\n"
        : "=r"(got), "=r"(x)
        : "r"(answer)
        : "memory");
    return got ? static_cast<int>(x) : -1;
}

// What block index w of the grid stands for.
struct Piece {
    int len, row0, q0, h0, kvh;  // sequence, first token of chain 0's tile, heads
    int n0, n1, look0;           // key tiles of each chain; tiles from look0 on hold a key that some row does not see
    __device__ __forceinline__ int n_max() const { return max(n0, n1); }
    __device__ __forceinline__ int looks() const { return max(0, n_max() - look0); }
};
template <int N>
__device__ __forceinline__ Piece piece_of(const PackedArgs &a, const PackedSeqs<N> &l, int log_p, int w) {
    Piece p;
    const int TQ = 128 >> log_p, n_ht = a.n_heads >> log_p;
    const int t = w / n_ht, ht = w - t * n_ht, s = seq_of_tile(l, t);
    p.len = l.len[s];
    p.row0 = l.start[s];
    // the last queries, which see the most keys, come first
    p.q0 = (l.tile0[s + 1] - l.tile0[s] - 1 - (t - l.tile0[s])) * 2 * TQ;
    p.h0 = ht << log_p;
    p.kvh = p.h0 / (a.n_heads / a.n_kv);
    const int kend0 = a.causal ? min(p.len, p.q0 + TQ) : p.len;
    const int kend1 = p.q0 + TQ >= p.len ? 0 : a.causal ? min(p.len, p.q0 + 2 * TQ) : p.len;
    p.n0 = (kend0 + kKeys - 1) / kKeys;
    p.n1 = (kend1 + kKeys - 1) / kKeys;
    p.look0 = a.causal ? p.q0 / kKeys : p.len / kKeys;
    return p;
}

// Barriers.  Every role counts ring items (K_0, V_0, K_1, ... of one piece after
// another; item i in slot i % NS), tiles of its chain, pieces of its chain and
// looked-over tiles alike, and takes phases from those counts.
//   full[slot] / free[slot]  item landed / both issuing warps' reads of it done
//   q[c] / qfree[c]          Q_c landed / the piece's last QK_c done
//   s[c]                     QK_c done: S_c readable
//   p[c]                     P_c written (four warps) and the chain's turn (one)
//   o[c] / ofree[c]          the piece's last PV_c done / O_c read (four warps)
//   go[x], look[x]           V of a partly seen tile loaded / looked over
//   answer                   the number of a further piece
//   work[x] / wfree[x]       piece handed out / read by the other ten warps
template <int D, class T, int N, bool kLong>
__global__ void __launch_bounds__(kTcThreads, 1)
    packed_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ PackedArgs a,
                     const __grid_constant__ PackedSeqs<N> l, int log_p) {
    using C = TcCfg<D>;
    constexpr int NS = C::kSlots;
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smraw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *ring = sm + 2 * C::kTile;  // Q_c at c * kTile
    __shared__ uint64_t bar_full[NS], bar_free[NS], bar_q[2], bar_qfree[2], bar_s[2], bar_p[2], bar_o[2], bar_ofree[2];
    __shared__ uint64_t bar_go[4], bar_look[4], bar_answer, bar_work[2], bar_wfree[2];
    __shared__ __align__(16) uint4 answer;
    __shared__ int4 pieces_s[2][2];  // decoded by the loading warp for the others
    __shared__ uint32_t tslot, dirty[4], held[2];  // held[c]: O_c already holds something before PV(0)

    // (values that the compiler knows to be the same in a warp stay in uniform
    // registers, where the MMA instructions want their operands)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    auto wait_w = [&](uint64_t *bar, uint32_t parity) {  // bounded; the warp agrees on the outcome
        return __all_sync(0xffffffffu, wait_phase(smem_u32(bar), parity & 1u)) != 0;
    };
    auto slot = [](uint32_t i) { return static_cast<int>(i % NS); };
    auto rph = [](uint32_t i) { return i / NS; };

    if (warp == 0) {
        tmem_alloc(smem_u32(&tslot), kTcCols);
        tmem_relinquish();
    }
    if (tid == 32 * kWarpLoad) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&bar_full[i]), 1);
            mbar_init(smem_u32(&bar_free[i]), 2);
        }
        for (int c = 0; c < 2; ++c) {
            mbar_init(smem_u32(&bar_q[c]), 1);
            mbar_init(smem_u32(&bar_qfree[c]), 1);
            mbar_init(smem_u32(&bar_s[c]), 1);
            mbar_init(smem_u32(&bar_p[c]), 5);
            mbar_init(smem_u32(&bar_o[c]), 1);
            mbar_init(smem_u32(&bar_ofree[c]), 4);
            mbar_init(smem_u32(&bar_work[c]), 1);
            mbar_init(smem_u32(&bar_wfree[c]), 10);
            held[c] = 0;
        }
        mbar_init(smem_u32(&bar_answer), 1);
        for (int x = 0; x < 4; ++x) {
            mbar_init(smem_u32(&bar_go[x]), 1);
            mbar_init(smem_u32(&bar_look[x]), 4);
            dirty[x] = 0;
        }
        fence_proxy_async();  // the barriers, before the asynchronous units use them
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = __shfl_sync(0xffffffffu, tslot, 0);
    bool ok = true;
    uint32_t wi = 0;  // pieces taken from the loading warp
    // The next piece (false: none is left, or a wait ran out).
    auto next_piece = [&](Piece &p) {
        const int x = wi & 1;
        ok = ok && wait_w(&bar_work[x], wi >> 1);
        if (!ok) return false;
        const int4 u = pieces_s[x][0], v = pieces_s[x][1];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_wfree[x]));
        ++wi;
        auto same = [](int y) { return __shfl_sync(0xffffffffu, y, 0); };
        p = Piece{same(u.x), same(u.y), same(u.z), same(u.w), same(v.x), same(v.y), same(v.z), same(v.w)};
        return p.len > 0;
    };

    if (warp >= 8) {
        setmaxnreg_dec<kTcOtherRegs>();
        if (warp == kWarpSpare) {
            // nothing to do
        } else if (warp == kWarpLoad) {
            // ---------------- loads (lane 0): of each piece K_0, Q, V_0, K_1, ... ----------------
            uint32_t it = 0, lk = 0, asked = 0, qn[2] = {0, 0};
            if (lane == 0) {
                for (const CUtensorMap *m : {&mq, &mk, &mv})
                    asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
            }
            Piece p = piece_of(a, l, log_p, blockIdx.x);
            for (;;) {
                // the others' copy (len 0: nothing is left)
                {
                    const int x = wi & 1;
                    if (wi >= 2) ok = wait_w(&bar_wfree[x], (wi >> 1) - 1);
                    if (ok && lane == 0) {
                        pieces_s[x][0] = make_int4(p.len, p.row0, p.q0, p.h0);
                        pieces_s[x][1] = make_int4(p.kvh, p.n0, p.n1, p.look0);
                        mbar_arrive(smem_u32(&bar_work[x]));
                    }
                    __syncwarp();
                    ++wi;
                }
                if (!ok || p.len == 0) break;
                for (int i = 0; i < 2 * p.n_max() && ok; ++i, ++it) {
                    const int sl = slot(it);
                    if (it >= NS) ok = wait_w(&bar_free[sl], rph(it) - 1);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_expect_tx(smem_u32(&bar_full[sl]), C::kTile);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load3(smem_u32(ring + sl * C::kTile + x * C::kBlock), (i & 1) ? &mv : &mk, 64 * x, p.kvh,
                                      p.row0 + (i >> 1) * kKeys, smem_u32(&bar_full[sl]));
                        if ((i & 1) && (i >> 1) >= p.look0) {
                            mbar_arrive(smem_u32(&bar_go[lk & 3]));
                            ++lk;
                        }
                    }
                    __syncwarp();
                    if (i == 0) {
                        for (int c = 0; c < (p.n1 > 0 ? 2 : 1) && ok; ++c) {
                            if (qn[c] > 0) ok = wait_w(&bar_qfree[c], qn[c] - 1);
                            if (!ok) break;
                            if (lane == 0) {
                                mbar_expect_tx(smem_u32(&bar_q[c]), C::kTile);
#pragma unroll
                                for (int x = 0; x < D / 64; ++x)
                                    tma_load3(smem_u32(sm + c * C::kTile + x * C::kBlock), &mq, 64 * x, p.h0,
                                              p.row0 + p.q0 + c * (128 >> log_p), smem_u32(&bar_q[c]));
                            }
                            ++qn[c];
                            __syncwarp();
                        }
                    }
                }
                // With its last load on the way the piece has a few tiles left to go:
                // time to ask for the next, late enough that short pieces take the most.
                if (!ok) break;
                if (lane == 0) {
                    fence_proxy_async();  // the answer before this one has been read
                    mbar_expect_tx(smem_u32(&bar_answer), 16);
                    ask_work(smem_u32(&answer), smem_u32(&bar_answer));
                }
                __syncwarp();
                ok = wait_w(&bar_answer, asked++);
                if (!ok) break;
                const int w = __shfl_sync(0xffffffffu, work_of(smem_u32(&answer)), 0);
                __syncwarp();
                if (w >= 0) p = piece_of(a, l, log_p, w);
                else p.len = 0;
            }
            // the last copies land before the CTA's shared memory is given up (bounded)
            for (int c = 0; c < 2; ++c)
                if (qn[c] > 0) wait_w(&bar_q[c], qn[c] - 1);
            for (uint32_t i = it > NS ? it - NS : 0; i < it; ++i) wait_w(&bar_full[slot(i)], rph(i));
            if (!ok && lane == 0 && a.err) atomicOr(a.err, 2);
        } else {
            // ---------------- MMA issue: chain c (one lane) ----------------
            const int c = warp == kWarpMma0 ? 0 : 1;
            const uint32_t tS = tbase + 256 + 128 * c, tO = tbase + 128 * c;
            const uint64_t dQ = desc_sw128(smem_u32(sm + c * C::kTile));
            // S_c = Q_c K^T (ring item i), then the barriers; on the way the turn
            // passes to the other chain, whose issuing warp needs a while to see it
            auto qk = [&](uint32_t i, bool pass, bool last) {
                const int sl = slot(i);
                const uint64_t dK = desc_sw128(smem_u32(ring + sl * C::kTile));
                if (elect_lane()) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t o = ((k >> 2) * C::kBlock + (k & 3) * 32u) >> 4;
                        mma_f16(tS, dQ + o, dK + o, idesc16<T>(kKeys, false), k > 0);
                        if (k == D / 16 - kPassLeft && pass) mbar_arrive(smem_u32(&bar_p[c ^ 1]));
                    }
                    mma_commit(smem_u32(&bar_s[c]));
                    mma_commit(smem_u32(&bar_free[sl]));
                    if (last) mma_commit(smem_u32(&bar_qfree[c]));
                }
                __syncwarp();
            };
            uint32_t it = 0, lk = 0, tiles = 0, pieces = 0;  // of the ring, looked over, of the chain
            bool owed = false;  // chain 0: the piece before ends with a turn from chain 1
            Piece p;
            while (next_piece(p)) {
                const int n = c ? p.n1 : p.n0, n_max = p.n_max();
                if (n > 0) {
                    ok = wait_w(&bar_q[c], pieces) && wait_w(&bar_full[slot(it)], rph(it));
                    if (!ok) break;
                    fence_after_sync();
                    qk(it, false, n == 1);
                }
                for (int j = 0; j < n && ok; ++j, ++tiles) {
                    const uint32_t iv = it + 2 * j + 1;
                    const int sv = slot(iv);
                    ok = wait_w(&bar_full[sv], rph(iv));
                    if (ok && j + 1 < n) ok = wait_w(&bar_full[slot(iv + 1)], rph(iv + 1));
                    if (ok && j == 0 && pieces > 0) ok = wait_w(&bar_ofree[c], pieces - 1);
                    if (ok && j >= p.look0) {
                        const uint32_t x = lk + j - p.look0;
                        ok = wait_w(&bar_look[x & 3], x >> 2);
                    }
                    // P, and this chain's turn: the other chain's products before these
                    // (chain 0's of tile j, chain 1's of tile j - 1 or of the piece
                    // before), or the most of them, have been issued; where there are
                    // none the chain takes its turn itself
                    const bool given = c ? j < p.n0 : j > 0 ? j - 1 < p.n1 : owed;
                    if (ok && !given && elect_lane()) mbar_arrive(smem_u32(&bar_p[c]));
                    if (ok) ok = wait_w(&bar_p[c], tiles);
                    if (!ok) break;
                    fence_after_sync();
                    const uint64_t dV = desc_mn(smem_u32(ring + sv * C::kTile), C::kBlock);
                    uint32_t acc = 1u;
                    if (j == 0) {
                        acc = *static_cast<volatile uint32_t *>(&held[c]);
                        __syncwarp();
                        if (elect_lane()) *static_cast<volatile uint32_t *>(&held[c]) = 0;
                    }
                    if (elect_lane()) {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            mma_f16_ts(tO, tS + 8 * k, dV + ((k * 2048u) >> 4), idesc16<T>(D, true), k > 0 ? 1u : acc);
                        mma_commit(smem_u32(&bar_free[sv]));
                        if (j + 1 == n) mma_commit(smem_u32(&bar_o[c]));
                    }
                    __syncwarp();
                    // the other chain's products follow (chain 1's last are followed
                    // by chain 0's first of the next piece)
                    const bool pass = c ? j + 1 < p.n0 || j + 1 == n : j < p.n1;
                    if (j + 1 < n) qk(iv + 1, pass, j + 2 == n);
                    else if (pass && elect_lane()) mbar_arrive(smem_u32(&bar_p[c ^ 1]));
                    __syncwarp();
                }
                // items past the chain's last tile are free as far as this chain goes
                // (counted once they have landed, so that each counts for its own phase)
                for (uint32_t i = it + 2 * n; i < it + 2 * n_max && ok; ++i) {
                    ok = wait_w(&bar_full[slot(i)], rph(i));
                    if (ok && elect_lane()) mbar_arrive(smem_u32(&bar_free[slot(i)]));
                }
                it += 2 * n_max;
                lk += p.looks();
                if (n > 0) ++pieces;
                owed = p.n1 > 0;
            }
            if (!ok && lane == 0 && a.err) atomicOr(a.err, 2);
        }
    } else {
        // -------------- compute warps: one thread per row and chain --------------
        setmaxnreg_inc<kTcComputeRegs>();
        const int c = warp >> 2, m = tid & 127, P = 1 << log_p, TQ = 128 >> log_p;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tbase + lanes + 256 + 128 * c, tO = tbase + lanes + 128 * c;
        const float cs = a.scale_log2;  // > 0
        uint32_t it = 0, lk = 0, tiles = 0, pieces = 0;
        Piece p;
        while (next_piece(p)) {
            const int n = c ? p.n1 : p.n0;
            const int tok = p.q0 + c * TQ + (m >> log_p);
            const bool valid = tok < p.len;
            const int lim = a.causal ? min(tok + 1, p.len) : p.len;  // keys this row sees
            float m_ref = -INFINITY, l_run = 0.f, unit = 0.f;
            uint32_t hold[kLong ? D / 4 : 1];  // with it the output's sum is O + h * unit
            if constexpr (kLong) {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) hold[i] = 0x80808080u;
            }
            const int step = kLong && p.len > kLongKeys ? kHold : n;
            for (int j0 = 0; j0 < n && ok; j0 += step) {
                if constexpr (kLong) {
                    if (j0 > 0) {
                        ok = wait_w(&bar_s[c], tiles);
                        if (!ok) break;
                        fence_after_sync();
                        uint32_t x[D];
#pragma unroll
                        for (int i = 0; i < D; i += 32) tmem_ld32_issue(tO + i, x + i);
                        tmem_ld_done(x);
                        unit = set_aside(x, hold, unit, j0 > kHold, D);
#pragma unroll
                        for (int i = 0; i < D; i += 16) {
                            float v[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(x[i + k]);
                            tmem_st16(tO + i, v);
                        }
                        tmem_st_wait();  // (O may be rescaled next)
                    }
                }
                for (int j = j0; j < min(n, j0 + step); ++j, ++tiles) {
                    const uint32_t look = lk + j - p.look0;
                    if (j >= p.look0 && (c == 1 || j >= p.n1)) {
                        // this chain looks over V_j: keys up to key0 are seen by every row; a
                        // key's 128 bytes of each 64 columns are 8 chunks.  (The loading warp
                        // tells when the slot is at V_j: these warps follow no earlier item.)
                        const uint32_t i = it + 2 * j + 1;
                        ok = wait_w(&bar_go[look & 3], look >> 2) && wait_w(&bar_full[slot(i)], rph(i));
                        if (!ok) break;
                        uint4 *v = reinterpret_cast<uint4 *>(ring + slot(i) * C::kTile);
                        const int key0 = max(0, (a.causal ? p.q0 + 1 : p.len) - j * kKeys);
                        constexpr uint32_t kE = std::is_same<T, bf16>::value ? 0x7f807f80u : 0x7c007c00u;
                        constexpr uint32_t kOne = std::is_same<T, bf16>::value ? 0x00800080u : 0x04000400u;
                        uint32_t seen = 0;  // a half's exponent is all ones where adding one to it reaches the sign bit
#pragma unroll
                        for (int x0 = 0; x0 < static_cast<int>(C::kTile / 16); x0 += 128) {
                            const int x = x0 + m;
                            if ((x & 1023) >= key0 * 8) {
                                const uint4 y = v[x];
                                seen |= ((y.x & kE) + kOne) | ((y.y & kE) + kOne) | ((y.z & kE) + kOne) | ((y.w & kE) + kOne);
                            }
                        }
                        if (seen & 0x80008000u) {
                            for (int x = m; x < static_cast<int>(C::kTile / 16); x += 128) {
                                if ((x & 1023) < key0 * 8) continue;
                                const uint4 y = v[x];
                                uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if (not_finite<T>(u[k])) u[k] &= 0xffff0000u;
                                    if (not_finite<T>(u[k] >> 16)) u[k] &= 0xffffu;
                                }
                                v[x] = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                            // the flag holds the count of the look it belongs to (+ 1)
                            *static_cast<volatile uint32_t *>(&dirty[look & 3]) = look + 1;
                        }
                        fence_proxy_async();  // before the MMAs read the tile
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bar_look[look & 3]));
                    }
                    ok = wait_w(&bar_s[c], tiles);
                    if (!ok) break;
                    fence_after_sync();
                    uint32_t x[kKeys];  // the row's scores (f32 bits)
#pragma unroll
                    for (int i = 0; i < kKeys; i += 32) tmem_ld32_issue(tS + i, x + i);
                    tmem_ld_done(x);
                    auto xf = [&](int i) { return __uint_as_float(x[i]); };
                    const int base = j * kKeys;
                    if (base + kKeys > lim) {
#pragma unroll
                        for (int i = 0; i < kKeys; ++i) x[i] = base + i < lim ? x[i] : 0xff800000u;
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[i] = fmaxf(xf(2 * i), xf(2 * i + 1));
#pragma unroll
                    for (int i = 8; i < kKeys; i += 2) mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], xf(i), xf(i + 1));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs;
                    const bool move = top > m_ref + kGrow || m_ref == -INFINITY;
                    const float m_use = move ? top : m_ref;
                    const float nm = m_use == -INFINITY ? 0.f : -m_use;
                    // O moves with the reference (QK(j), already done, followed PV(j - 1))
                    const float f = move && m_ref != -INFINITY ? ex2(m_ref - m_use) : 1.f;
                    if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            float o[16];
                            tmem_ld16(tO + 16 * i, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] *= f;
                            tmem_st16(tO + 16 * i, o);
                        }
                        unit *= f;
                    }
                    m_ref = m_use;
                    // P over S
                    uint64_t sum[2] = {0, 0};
                    const uint64_t cs2 = pair(cs, cs), nm2 = pair(nm, nm);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t pr[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float2 e = unpair(fma2(pair(xf(64 * i + 2 * k), xf(64 * i + 2 * k + 1)), cs2, nm2));
                            const float p0 = ex2(e.x), p1 = ex2(e.y);
                            sum[k & 1] = add2(sum[k & 1], pair(p0, p1));
                            pr[k] = pack2(T{}, p0, p1);
                        }
                        tmem_st32u(tS + 32 * i, pr);
                    }
                    const float2 s2 = unpair(add2(sum[0], sum[1]));
                    l_run = fmaf(l_run, f, s2.x + s2.y);
                    tmem_st_wait();
                    if (j >= p.look0) {
                        ok = wait_w(&bar_look[look & 3], look >> 2);
                        if (!ok) break;
                        if (*static_cast<volatile uint32_t *>(&dirty[look & 3]) == look + 1) {
                            // this tile's V values that are not finite, key by key (PV(0) of
                            // the piece writes over O, unless told that O holds something;
                            // O is this piece's from then on: its reader is this thread)
                            const T *v = static_cast<const T *>(a.V) + static_cast<int64_t>(p.row0 + base) * a.v_stride +
                                         static_cast<int64_t>(p.kvh) * a.hd;
                            const int see = valid ? min(kKeys, lim - base) : 0;
#pragma unroll 1
                            for (int i = 0; i < D / 16; ++i) {
                                float o[16];
                                if (j > 0) {
                                    tmem_ld16(tO + 16 * i, o);
                                } else {
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] = 0.f;
                                }
#pragma unroll 1
                                for (int kk = 0; kk < kKeys / 2; ++kk) {
                                    const uint32_t pw = tmem_ld1(tS + kk);
#pragma unroll
                                    for (int e = 0; e < 2; ++e) {
                                        if (2 * kk + e >= see) continue;
                                        const unsigned short *vr = reinterpret_cast<const unsigned short *>(
                                            v + static_cast<int64_t>(2 * kk + e) * a.v_stride) + 16 * i;
                                        const float pe = half_of(T{}, pw, e);
#pragma unroll
                                        for (int k = 0; k < 16; ++k) {
                                            if (16 * i + k >= a.hd) continue;
                                            const uint32_t b = __ldg(vr + k);
                                            if (not_finite<T>(b)) o[k] = fmaf(pe, half_of(T{}, b, 0), o[k]);
                                        }
                                    }
                                    __syncwarp();
                                }
                                tmem_st16(tO + 16 * i, o);
                            }
                            if (j == 0 && m == 0) *static_cast<volatile uint32_t *>(&held[c]) = 1;
                            tmem_st_wait();
                        }
                    }
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar_p[c]));
                }
            }
            if (n > 0 && ok) {
                ok = wait_w(&bar_o[c], pieces);
                if (!ok) break;
                fence_after_sync();
                uint32_t o[D];
#pragma unroll
                for (int i = 0; i < D; i += 32) tmem_ld32_issue(tO + i, o + i);
                tmem_ld_done(o);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_ofree[c]));
                if constexpr (kLong) {
                    if (n > step) {
#pragma unroll
                        for (int i = 0; i < D; ++i)
                            o[i] = __float_as_uint(fmaf(aside(hold[i / 4], i & 3), unit, __uint_as_float(o[i])));
                    }
                }
                const float inv = 1.f / l_run;
                T *dst = static_cast<T *>(a.out) + static_cast<int64_t>(p.row0 + (valid ? tok : 0)) * a.o_stride +
                         static_cast<int64_t>(p.h0 + (m & (P - 1))) * a.hd;
                auto two = [&](int i) { return pack2(T{}, __uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv); };
                if (a.out32) {  // whole 32-byte sectors
#pragma unroll
                    for (int i = 0; i < D; i += 16)
                        if (valid && i < a.hd)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + i),
                                         "r"(two(i)), "r"(two(i + 2)), "r"(two(i + 4)), "r"(two(i + 6)), "r"(two(i + 8)),
                                         "r"(two(i + 10)), "r"(two(i + 12)), "r"(two(i + 14))
                                         : "memory");
                } else {
#pragma unroll
                    for (int i = 0; i < D; i += 8)
                        if (valid && i < a.hd)
                            *reinterpret_cast<uint4 *>(dst + i) = make_uint4(two(i), two(i + 2), two(i + 4), two(i + 6));
                }
                ++pieces;
            }
            it += 2 * p.n_max();
            lk += p.looks();
        }
        if (!ok && lane == 0 && a.err) atomicOr(a.err, 2);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, kTcCols);
}

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
    const uint32_t a = smem_u32(p);
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

// Rows [tokens][heads][hd] with a token stride, in boxes of 64 columns x
// box_heads x box_tokens; columns past hd and tokens past the last read as 0.
cudaError_t rows_map(CUtensorMap *m, EncodeTiled f, const PackedArgs &a, const void *base, int64_t stride, int heads,
                     int box_heads, int box_tokens) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.hd), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(a.n_tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.hd) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = f(m, a.type == Elem::bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
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
    if (e == cudaSuccess) e = rows_map(&mq, f, a, a.Q, a.q_stride, a.n_heads, 1 << log_p, 128 >> log_p);
    if (e == cudaSuccess) e = rows_map(&mk, f, a, a.K, a.k_stride, a.n_kv, 1, kKeys);
    if (e == cudaSuccess) e = rows_map(&mv, f, a, a.V, a.v_stride, a.n_kv, 1, kKeys);
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

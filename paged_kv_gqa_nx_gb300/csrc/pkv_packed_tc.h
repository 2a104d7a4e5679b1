// pkv_packed_tc.h -- the tensor-core kernel of packed 16-bit rows: whole prompts
// (pkv_packed.cu) and runs of queries over keys of other lengths, behind a
// shared prefix or not (pkv_ragged_tc.h).
#pragma once

#include "pkv_half.h"
#include "pkv_ragged.h"
#include "pkv_softmax_tc.h"
#include "pkv_tcgen05.h"
#include "pkv_tma.h"

namespace pkv {
namespace {

using namespace tc;

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
    // Heads wider than 128: one chain, whose O takes the columns of both
    static constexpr int kChains = D > 128 ? 1 : 2;
    static constexpr int kSlots = D == 64 ? 8 : D == 128 ? 5 : D == 192 ? 3 : 2;
    static constexpr size_t kSmem = (kChains + kSlots) * kTile + 1024;  // + alignment slack
};

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
        : "memory");
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

// Whole prompts: every sequence's queries attend its own keys.
template <int N>
struct WholePrompts {
    static constexpr bool kRuns = false, kStacks = false, kAlt = false;
    // Tokens of a tile, token and head of its row m; `tile` is log2 of its heads.
    __device__ __forceinline__ static int tokens(int tile) { return 128 >> tile; }
    __device__ __forceinline__ static int token(int m, int tile) { return m >> tile; }
    __device__ __forceinline__ static int head(int m, int tile) { return m & ((1 << tile) - 1); }
    __device__ __forceinline__ static int rows(int) { return 128; }
    using Args = PackedArgs;
    using List = PackedSeqs<N>;
    // What block index w of the grid stands for.
    struct Piece {
        static constexpr int kWords = 2;  // int4s
        int len, row0, q0, h0, kvh;  // sequence, first token of chain 0's tile, heads
        int n0, n1, look0;           // key tiles of each chain; tiles from look0 on hold a key that some row does not see
        __device__ __forceinline__ int n_max() const { return max(n0, n1); }
        __device__ __forceinline__ int looks() const { return max(0, n_max() - look0); }
    };
    __device__ __forceinline__ static Piece piece(const Args &a, const List &l, int log_p, int w) {
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
    __device__ __forceinline__ static bool is_long(const Piece &p) { return p.len > kLongKeys; }
    // Key tile j of the piece: its keys that a row sees (row limits counted from
    // the tile's first key), and of those the ones that all rows see.
    __device__ __forceinline__ static int key0(const Args &a, const Piece &p, int j) {
        return max(0, (a.causal ? p.q0 + 1 : p.len) - j * kKeys);
    }
};

// Runs of queries over keys of their own, behind a shared prefix or not, the
// key tiles (the prefix's, then the run's) split or not.  A piece has at least one key tile a
// chain, seen or not, so that every row's record is written.
//
// With kTurns a piece of one query tile takes its key tiles on both chains in
// turn, the even ones on chain 0, and the chains' parts are joined at the end: one chain
// by itself waits for its own softmax.
template <int N, int kChains, bool kTurns>
struct Runs {
    static constexpr bool kRuns = true, kStacks = false, kAlt = kTurns;
    // `tile` is the number of its heads; rows past the last whole token are not used.
    __device__ __forceinline__ static int tokens(int tile) { return 128 / tile; }
    __device__ __forceinline__ static int token(int m, int tile) { return m / tile; }
    __device__ __forceinline__ static int head(int m, int tile) { return m % tile; }
    __device__ __forceinline__ static int rows(int tile) { return 128 / tile * tile; }
    using Args = RaggedArgs;
    using List = RunList<RaggedRun, N>;
    struct Piece {
        static constexpr int kWords = 4;
        int len, row0, q0, h0, kvh;  // queries of the run, its first row, first query of chain 0's tile, heads
        int n0, n1, look0;           // counted from tile j0 on
        int j0, k0, nk, off;         // first tile of the split; key rows
        int rec, ns, alt, pad;       // record of query 0 (-1: none), records a query; the chains take key tiles in turn
        __device__ __forceinline__ int n_max() const { return alt ? n0 + n1 : max(n0, n1); }
        __device__ __forceinline__ void turns() {
            alt = kTurns && n1 == 0 && n0 > 1;
            if (alt) {
                n1 = n0 / 2;
                n0 -= n1;
            }
        }
        __device__ __forceinline__ int looks() const { return max(0, n_max() - look0); }
    };
    __device__ __forceinline__ static Piece piece(const Args &a, const List &l, int tile, int w) {
        Piece p;
        const int TQ = 128 / tile, n_ht = a.n_heads / tile;
        const int t = w / n_ht, ht = w - t * n_ht;
        int lo = 0, hi = l.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (l.unit0[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        const RaggedRun r = l.run[lo];
        const int pairs = (r.nq + kChains * TQ - 1) / (kChains * TQ), u = t - l.unit0[lo], split = u / pairs;
        p.len = r.nq;
        p.row0 = r.q0;
        p.q0 = (pairs - 1 - (u - split * pairs)) * kChains * TQ;
        p.h0 = ht * tile;
        p.kvh = p.h0 / (a.n_heads / a.n_kv);
        p.k0 = r.k0;
        p.nk = r.nk;
        p.off = r.off;
        p.rec = r.rec0 < 0 ? -1 : r.rec0 + split;
        p.ns = r.ns;
        p.pad = 0;
        const int pre = (a.n_pre + kKeys - 1) / kKeys, all = pre + (r.nk + kKeys - 1) / kKeys, per = (all + r.ns - 1) / r.ns;
        p.j0 = split * per;
        auto tiles = [&](int q) {  // up to the last key that query q sees
            return min(pre + (min(r.nk, r.off + q + 1) + kKeys - 1) / kKeys - p.j0, per);
        };
        p.n0 = max(1, tiles(min(p.q0 + TQ, r.nq) - 1));
        p.n1 = kChains == 1 || p.q0 + TQ >= r.nq ? 0 : max(1, tiles(min(p.q0 + 2 * TQ, r.nq) - 1));
        p.look0 = max(0, pre + min(r.nk, r.off + p.q0 + 1) / kKeys - p.j0);
        p.turns();
        return p;
    }
    __device__ __forceinline__ static bool is_long(const Piece &p) { return p.n_max() * kKeys > kLongKeys; }
    __device__ __forceinline__ static int key0(const Args &a, const Piece &p, int j) {
        return max(0, min(p.nk, p.off + p.q0 + 1) - (p.j0 + j - (a.n_pre + kKeys - 1) / kKeys) * kKeys);
    }
};

// The queries of neighbouring sequences as stretches of rows behind the shared
// prefix, own key rows in the same order: a tile may hold rows of several
// sequences, and its own keys are those of all of them, of which a row sees some.
// A list's runs are in the order of their queries.
template <int N, int kChains, bool kTurns>
struct Stacks : Runs<N, kChains, kTurns> {
    static constexpr bool kStacks = true;
    using typename Runs<N, kChains, kTurns>::Args;
    using typename Runs<N, kChains, kTurns>::List;
    using typename Runs<N, kChains, kTurns>::Piece;
    // The sequence of query row q.
    __device__ __forceinline__ static int seq(const List &l, int q) {
        int lo = 0, hi = l.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (l.run[mid].q0 <= q) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
    // Key row behind the last one that query row q, of run r, sees.
    __device__ __forceinline__ static int end(const RaggedRun &r, int q) { return r.k0 + r.off + (q - r.q0) + 1; }
    __device__ __forceinline__ static Piece piece(const Args &a, const List &l, int tile, int w) {
        Piece p;
        const int TQ = 128 / tile, n_ht = a.n_heads / tile;
        const int t = w / n_ht, ht = w - t * n_ht;
        int x = 0, hi = a.n_stretches - 1;
        while (x < hi) {
            const int mid = (x + hi + 1) >> 1;
            if (l.unit0[mid] <= t) x = mid;
            else hi = mid - 1;
        }
        const int u = t - l.unit0[x];
        const RaggedRun &f = l.run[l.run[x].kind], &e = l.run[(x + 1 < a.n_stretches ? l.run[x + 1].kind : l.n) - 1];
        p.row0 = f.q0;
        p.len = e.q0 + e.nq - p.row0;
        p.ns = f.ns;
        const int pairs = (p.len + kChains * TQ - 1) / (kChains * TQ), split = u / pairs;
        p.q0 = (pairs - 1 - (u - split * pairs)) * kChains * TQ;
        p.h0 = ht * tile;
        p.kvh = p.h0 / (a.n_heads / a.n_kv);
        p.rec = f.rec0 < 0 ? -1 : f.rec0 + split;
        p.off = p.pad = 0;
        const int last0 = min(p.q0 + TQ, p.len) - 1, last = min(p.q0 + kChains * TQ, p.len) - 1;
        p.k0 = l.run[seq(l, p.row0 + p.q0)].k0;
        p.nk = end(l.run[seq(l, p.row0 + last)], p.row0 + last) - p.k0;
        const int pre = (a.n_pre + kKeys - 1) / kKeys, all = pre + (p.nk + kKeys - 1) / kKeys, per = (all + p.ns - 1) / p.ns;
        p.j0 = split * per;
        const int keys0 = end(l.run[seq(l, p.row0 + last0)], p.row0 + last0) - p.k0;
        p.n0 = max(1, min(pre + (keys0 + kKeys - 1) / kKeys - p.j0, per));
        p.n1 = last == last0 ? 0 : max(1, min(all - p.j0, per));
        p.look0 = max(0, pre - p.j0);
        p.turns();
        return p;
    }
    __device__ __forceinline__ static int key0(const Args &, const Piece &, int) { return 0; }
};

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
//   part[x]                  chain 1's part of a piece taken in turn written (four warps)
// mkp, mvp: of the shared prefix (Runs).
template <int D, class T, bool kLong, class F>
__device__ __forceinline__ void packed_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                                          const CUtensorMap &mkp, const CUtensorMap &mvp, const typename F::Args &a,
                                          const typename F::List &l, int tile) {
    using C = TcCfg<D>;
    using Piece = typename F::Piece;
    static_assert(!kLong || D <= 128, "sums are set aside in registers");
    constexpr int NS = C::kSlots;
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smraw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char *ring = sm + C::kChains * C::kTile;  // Q_c at c * kTile
    __shared__ uint64_t bar_full[NS], bar_free[NS], bar_q[2], bar_qfree[2], bar_s[2], bar_p[2], bar_o[2], bar_ofree[2];
    __shared__ uint64_t bar_go[4], bar_look[4], bar_answer, bar_work[2], bar_wfree[2];
    __shared__ __align__(16) uint4 answer;
    __shared__ int4 pieces_s[2][Piece::kWords];  // decoded by the loading warp for the others
    __shared__ uint32_t tslot, dirty[4], held[2];  // held[c]: O_c already holds something before PV(0)
    // Chain 1's maxima and sums of a piece taken in turn; two, as it may end the next
    // such piece before chain 0 has read them (not the one after: its product waits for O_1).
    __shared__ uint64_t bar_part[2];
    __shared__ float2 part_s[2][F::kAlt ? 128 : 1];

    // (values that the compiler knows to be the same in a warp stay in uniform
    // registers, where the MMA instructions want their operands)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    auto wait_w = [&](uint64_t *bar, uint32_t parity) {  // bounded; the warp agrees on the outcome
        return __all_sync(0xffffffffu, wait_phase(smem_u32(bar), parity & 1u)) != 0;
    };
    auto in_turn = [](const Piece &p) {
        if constexpr (F::kAlt) return p.alt != 0;
        else return false;
    };
    auto slot = [](uint32_t i) { return static_cast<int>(i % NS); };
    auto rph = [](uint32_t i) { return i / NS; };

    if (warp == 0) {
        tmem_alloc(smem_u32(&tslot), kTcCols);
        tmem_relinquish();
    }
    if constexpr (F::kRuns) {  // rows of Q that no load writes
        const int at = F::rows(tile) * 128, n = (static_cast<int>(C::kBlock) - at) / 16;
        for (int i = tid; i < C::kChains * (D / 64) * n; i += kTcThreads)
            *reinterpret_cast<uint4 *>(sm + i / n * C::kBlock + at + i % n * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
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
        for (int x = 0; x < 2; ++x) mbar_init(smem_u32(&bar_part[x]), 4);
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
        int4 u[Piece::kWords];
#pragma unroll
        for (int i = 0; i < Piece::kWords; ++i) u[i] = pieces_s[x][i];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_wfree[x]));
        ++wi;
        auto same = [](int y) { return __shfl_sync(0xffffffffu, y, 0); };
        if constexpr (F::kRuns)
            p = Piece{same(u[0].x), same(u[0].y), same(u[0].z), same(u[0].w), same(u[1].x), same(u[1].y), same(u[1].z), same(u[1].w),
                      same(u[2].x), same(u[2].y), same(u[2].z), same(u[2].w), same(u[3].x), same(u[3].y), F::kAlt ? same(u[3].z) : 0, 0};
        else
            p = Piece{same(u[0].x), same(u[0].y), same(u[0].z), same(u[0].w), same(u[1].x), same(u[1].y), same(u[1].z), same(u[1].w)};
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
                if constexpr (F::kRuns) {
                    for (const CUtensorMap *m : {&mkp, &mvp})
                        asm volatile("prefetch.tensormap [%0];\n" ::"l"(m) : "memory");
                }
            }
            Piece p = F::piece(a, l, tile, blockIdx.x);
            for (;;) {
                // the others' copy (len 0: nothing is left)
                {
                    const int x = wi & 1;
                    if (wi >= 2) ok = wait_w(&bar_wfree[x], (wi >> 1) - 1);
                    if (ok && lane == 0) {
                        pieces_s[x][0] = make_int4(p.len, p.row0, p.q0, p.h0);
                        pieces_s[x][1] = make_int4(p.kvh, p.n0, p.n1, p.look0);
                        if constexpr (F::kRuns) {
                            pieces_s[x][2] = make_int4(p.j0, p.k0, p.nk, p.off);
                            pieces_s[x][3] = make_int4(p.rec, p.ns, p.alt, 0);
                        }
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
                        const CUtensorMap *map = (i & 1) ? &mv : &mk;
                        int row = p.row0 + (i >> 1) * kKeys;
                        if constexpr (F::kRuns) {
                            const int t = p.j0 + (i >> 1), pre = (a.n_pre + kKeys - 1) / kKeys;
                            if (t < pre) map = (i & 1) ? &mvp : &mkp;
                            row = t < pre ? t * kKeys : p.k0 + (t - pre) * kKeys;
                        }
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load3(smem_u32(ring + sl * C::kTile + x * C::kBlock), map, 64 * x, p.kvh, row, smem_u32(&bar_full[sl]));
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
                                mbar_expect_tx(smem_u32(&bar_q[c]), F::rows(tile) * (D * 2));
#pragma unroll
                                for (int x = 0; x < D / 64; ++x)
                                    tma_load3(smem_u32(sm + c * C::kTile + x * C::kBlock), &mq, 64 * x, p.h0,
                                              p.row0 + p.q0 + (in_turn(p) ? 0 : c * F::tokens(tile)), smem_u32(&bar_q[c]));
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
                if (w >= 0) p = F::piece(a, l, tile, w);
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
                const bool alt = in_turn(p);
                // Items of the other chain's tiles, as far as `end`: free as far as this
                // chain goes.  (All items are waited for in order: a wait for a later use of
                // a slot would take the phase before an unfinished one for its own.)
                uint32_t seen = it;
                auto pass_over = [&](uint32_t end) {
                    for (; seen < end && ok; ++seen) {
                        if (((seen - it) >> 1 & 1) == static_cast<uint32_t>(c)) continue;
                        ok = wait_w(&bar_full[slot(seen)], rph(seen));
                        if (ok && elect_lane()) mbar_arrive(smem_u32(&bar_free[slot(seen)]));
                    }
                };
                auto tile_of = [&](int j) { return alt ? 2 * j + c : j; };  // of the piece
                if (n > 0) {
                    const uint32_t ik = it + 2 * tile_of(0);
                    if (alt) pass_over(ik);
                    ok = ok && wait_w(&bar_q[c], pieces) && wait_w(&bar_full[slot(ik)], rph(ik));
                    if (!ok) break;
                    fence_after_sync();
                    qk(ik, false, n == 1);
                }
                for (int j = 0; j < n && ok; ++j, ++tiles) {
                    const int jt = tile_of(j);
                    const uint32_t iv = it + 2 * jt + 1, ik = it + 2 * tile_of(j + 1);
                    const int sv = slot(iv);
                    ok = wait_w(&bar_full[sv], rph(iv));
                    if (alt) pass_over(min(ik, it + 2 * n_max));
                    if (ok && j + 1 < n) ok = wait_w(&bar_full[slot(ik)], rph(ik));
                    if (ok && j == 0 && pieces > 0) ok = wait_w(&bar_ofree[c], pieces - 1);
                    if (ok && jt >= p.look0) {
                        const uint32_t x = lk + jt - p.look0;
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
                    if (j + 1 < n) qk(ik, pass, j + 2 == n);
                    else if (pass && elect_lane()) mbar_arrive(smem_u32(&bar_p[c ^ 1]));
                    __syncwarp();
                }
                // items past the chain's last tile are free as far as this chain goes
                // (counted once they have landed, so that each counts for its own phase)
                if (alt) pass_over(it + 2 * n_max);
                for (uint32_t i = it + 2 * n; i < it + 2 * n_max && ok && !alt; ++i) {
                    ok = wait_w(&bar_full[slot(i)], rph(i));
                    if (ok && elect_lane()) mbar_arrive(smem_u32(&bar_free[slot(i)]));
                }
                it += 2 * n_max;
                lk += p.looks();
                if (n > 0) ++pieces;
                owed = p.n1 > 0 && p.n0 <= p.n1;
            }
            if (!ok && lane == 0 && a.err) atomicOr(a.err, 2);
        }
    } else {
        // -------------- compute warps: one thread per row and chain --------------
        setmaxnreg_inc<kTcComputeRegs>();
        const int c = warp >> 2, m = tid & 127, TQ = F::tokens(tile), head = F::head(m, tile);
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tbase + lanes + 256 + 128 * c, tO = tbase + lanes + 128 * c;
        const float cs = a.scale_log2;  // > 0
        uint32_t it = 0, lk = 0, tiles = 0, pieces = 0, pieces1 = 0, parts = 0;  // pieces of chain 1, taken in turn
        Piece p;
        while (next_piece(p)) {
            const int n = c ? p.n1 : p.n0;
            const bool alt = in_turn(p);
            const int tok = p.q0 + (alt ? 0 : c * TQ) + F::token(m, tile);
            const bool valid = tok < p.len && m < F::rows(tile);
            int lim, from = 0;  // keys this row sees (Runs: of the run's own)
            if constexpr (F::kStacks) {
                const int q = p.row0 + (valid ? tok : p.q0);
                const RaggedRun &r = l.run[F::seq(l, q)];
                from = r.k0 - p.k0;
                lim = F::end(r, q) - p.k0;
            } else if constexpr (F::kRuns) lim = min(p.nk, p.off + tok + 1);
            else lim = a.causal ? min(tok + 1, p.len) : p.len;
            float m_ref = -INFINITY, l_run = 0.f, unit = 0.f;
            uint32_t hold[kLong ? D / 4 : 1];  // with it the output's sum is O + h * unit
            if constexpr (kLong) {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) hold[i] = 0x80808080u;
            }
            const int step = kLong && F::is_long(p) ? kHold : n;
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
                    const int jt = alt ? 2 * j + c : j;  // of the piece
                    const uint32_t look = lk + jt - p.look0;
                    if (jt >= p.look0 && (c == 1 || alt || j >= p.n1)) {
                        // this chain looks over V_j: keys up to key0 are seen by every row; a
                        // key's 128 bytes of each 64 columns are 8 chunks.  (The loading warp
                        // tells when the slot is at V_j: these warps follow no earlier item.)
                        const uint32_t i = it + 2 * jt + 1;
                        ok = wait_w(&bar_go[look & 3], look >> 2) && wait_w(&bar_full[slot(i)], rph(i));
                        if (!ok) break;
                        uint4 *v = reinterpret_cast<uint4 *>(ring + slot(i) * C::kTile);
                        const int key0 = F::key0(a, p, jt);
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
                    int base = jt * kKeys, end = lim;  // the tile's first key, and the first that this row does not see
                    if constexpr (F::kRuns) {
                        const int t = p.j0 + jt, pre = (a.n_pre + kKeys - 1) / kKeys;
                        base = (t < pre ? t : t - pre) * kKeys;
                        end = t < pre ? a.n_pre : lim;
                        if constexpr (F::kStacks) {
                            if (t >= pre && base < from) {
#pragma unroll
                                for (int i = 0; i < kKeys; ++i) x[i] = base + i >= from ? x[i] : 0xff800000u;
                            }
                        }
                    }
                    if (base + kKeys > end) {
#pragma unroll
                        for (int i = 0; i < kKeys; ++i) x[i] = base + i < end ? x[i] : 0xff800000u;
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
                    if (jt >= p.look0) {
                        ok = wait_w(&bar_look[look & 3], look >> 2);
                        if (!ok) break;
                        if (*static_cast<volatile uint32_t *>(&dirty[look & 3]) == look + 1) {
                            // this tile's V values that are not finite, key by key (PV(0) of
                            // the piece writes over O, unless told that O holds something;
                            // O is this piece's from then on: its reader is this thread,
                            // but for an O_1 of tiles taken in turn, which chain 0 reads)
                            if (F::kAlt && c == 1 && j == 0 && pieces > 0) {
                                ok = wait_w(&bar_ofree[1], pieces - 1);
                                if (!ok) break;
                                fence_after_sync();
                            }
                            int64_t row = p.row0 + base;
                            if constexpr (F::kRuns) row = p.k0 + base;  // (a tile of the run's own)
                            const T *v = static_cast<const T *>(a.V) + row * a.v_stride + static_cast<int64_t>(p.kvh) * a.hd;
                            const int see = valid ? min(kKeys, end - base) : 0;
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
                                        if constexpr (F::kStacks) {
                                            if (base + 2 * kk + e < from) continue;
                                        }
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
            if (F::kAlt && alt && c == 1) {
                if (!ok) break;
                part_s[parts & 1][F::kAlt ? m : 0] = make_float2(m_ref, l_run);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_part[parts & 1]));
            } else if (n > 0 && ok) {
                ok = wait_w(&bar_o[c], pieces);
                // (chain 1's part first: with it the piece before is surely behind its O_1)
                if (F::kAlt && alt) ok = ok && wait_w(&bar_part[parts & 1], parts >> 1) && wait_w(&bar_o[1], pieces1);
                if (!ok) break;
                fence_after_sync();
                if (F::kAlt && alt) {  // chain 1's part of these rows (of the same lanes) into chain 0's
                    const float2 other = part_s[parts & 1][F::kAlt ? m : 0];
                    const float top = fmaxf(m_ref, other.x), ref = top == -INFINITY ? 0.f : top;
                    const float f0 = ex2(m_ref - ref), f1 = ex2(other.x - ref);
                    m_ref = top;
                    l_run = l_run * f0 + other.y * f1;
#pragma unroll 1
                    for (int i = 0; i < D; i += 16) {
                        float x0[16], x1[16];
                        tmem_ld16(tO + i, x0);
                        tmem_ld16(tO + 128 + i, x1);
#pragma unroll
                        for (int k = 0; k < 16; ++k) x0[k] = fmaf(x1[k], f1, x0[k] * f0);
                        tmem_st16(tO + i, x0);
                    }
                    tmem_st_wait();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar_ofree[1]));
                }
                constexpr int kPart = D > 128 ? 64 : D;  // columns at a time
#pragma unroll 1
                for (int i0 = 0; i0 < D; i0 += kPart) {
                    uint32_t o[kPart];
#pragma unroll
                    for (int i = 0; i < kPart; i += 32) tmem_ld32_issue(tO + i0 + i, o + i);
                    tmem_ld_done(o);
                    if (i0 + kPart == D) {
                        fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bar_ofree[c]));
                    }
                    if constexpr (kLong) {
                        if (n > step) {
#pragma unroll
                            for (int i = 0; i < D; ++i)
                                o[i] = __float_as_uint(fmaf(aside(hold[i / 4], i & 3), unit, __uint_as_float(o[i])));
                        }
                    }
                    if constexpr (F::kRuns) {
                        if (p.rec >= 0) {
                            const int64_t r = (p.rec + static_cast<int64_t>(tok) * p.ns) * a.n_heads + p.h0 + head;
                            float *dst = a.pacc + r * a.hd + i0;
                            if (valid && i0 == 0) {
                                a.pm[r] = m_ref;
                                a.pl[r] = l_run;
                            }
                            if (valid && l_run != 0.f) {
#pragma unroll
                                for (int i = 0; i < kPart; i += 8)  // whole sectors
                                    if (i0 + i < a.hd)
                                        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + i),
                                                     "r"(o[i]), "r"(o[i + 1]), "r"(o[i + 2]), "r"(o[i + 3]), "r"(o[i + 4]),
                                                     "r"(o[i + 5]), "r"(o[i + 6]), "r"(o[i + 7])
                                                     : "memory");
                            }
                            continue;
                        }
                    }
                    const float inv = 1.f / l_run;
                    T *dst = static_cast<T *>(a.out) + static_cast<int64_t>(p.row0 + (valid ? tok : 0)) * a.o_stride +
                             static_cast<int64_t>(p.h0 + head) * a.hd + i0;
                    auto two = [&](int i) { return pack2(T{}, __uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv); };
                    if (a.out32) {  // whole 32-byte sectors
#pragma unroll
                        for (int i = 0; i < kPart; i += 16)
                            if (valid && i0 + i < a.hd)
                                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + i),
                                             "r"(two(i)), "r"(two(i + 2)), "r"(two(i + 4)), "r"(two(i + 6)), "r"(two(i + 8)),
                                             "r"(two(i + 10)), "r"(two(i + 12)), "r"(two(i + 14))
                                             : "memory");
                    } else {
#pragma unroll
                        for (int i = 0; i < kPart; i += 8)
                            if (valid && i0 + i < a.hd)
                                *reinterpret_cast<uint4 *>(dst + i) = make_uint4(two(i), two(i + 2), two(i + 4), two(i + 6));
                    }
                }
            }
            if (n > 0) ++pieces;
            if (p.n1 > 0) ++pieces1;
            if (alt) ++parts;
            it += 2 * p.n_max();
            lk += p.looks();
        }
        if (!ok && lane == 0 && a.err) atomicOr(a.err, 2);
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, kTcCols);
}

// Rows [tokens][heads][hd] with a token stride, in boxes of 64 columns x
// box_heads x box_tokens; columns past hd and tokens past the last read as 0.
inline cudaError_t rows_map(CUtensorMap *m, EncodeTiled f, Elem type, int hd, int64_t rows, const void *base, int64_t stride, int heads,
                            int box_heads, int box_tokens) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = f(m, type == Elem::bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                         const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace pkv

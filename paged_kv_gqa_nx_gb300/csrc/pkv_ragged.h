// pkv_ragged.h -- attention of packed 16-bit query rows over keys of other
// lengths (cross attention, a shared prefix): what the host plan
// (pkv_ragged_host.cpp) hands to the kernels.
//
// A call's sequences become runs: consecutive query rows that attend the same
// stretch of key rows, with the shared prefix before it where a launch has one.
// A run's keys may be split; each (query, split) then leaves a partial record
// (maximum, sum, unnormalised output of every head) in the caller's workspace
// and the join launch combines them.
#pragma once

#include "pkv_internal.h"

namespace pkv {

constexpr int32_t kSMs = 152;  // of the GPU that the plans and grids are made for

constexpr int32_t kSees = 0x3fffffff;  // `off` of a run whose queries see every key

// What a run of the row kernel is: its own keys (behind the prefix, where the
// launch has one), or the prefix's rows themselves (k0 0, nk all of them).
constexpr int32_t kOwnKeys = 0, kOnPrefix = 1;

struct RaggedRun {
    int32_t q0, nq;    // first row of Q and out, queries
    int32_t k0, nk;    // first key row, keys
    int32_t off;       // query i sees the run's keys j <= off + i
    int32_t ns;        // splits of the prefix and the run's keys together
    int32_t rec0;      // record of (query i, split x): rec0 + i * ns + x; -1: one split, written to out
    int32_t kind;
};

// A query's records: ns of its own keys and pns of the shared prefix.
struct JoinRun {
    int32_t q0, nq, rec0, ns, pre0, pns;
};

// Lists travel in the launch's parameters (no upload), in two sizes as a
// launch takes longer with more of them.
constexpr int32_t kRaggedSmall = 64, kRaggedLarge = 850;
template <class R, int N>
struct RunList {
    int32_t n;
    int32_t unit0[N + 1];  // units of the runs before it
    R run[N];
};

struct RaggedArgs {
    const void *Q, *K, *V;
    void *out;
    int64_t q_stride, k_stride, v_stride, o_stride;  // elements per row
    const void *Kp, *Vp;                              // the shared prefix
    int64_t kp_stride, vp_stride;
    int32_t n_pre;                                    // its rows (0: none)
    int32_t n_heads, n_kv, hd;
    float scale_log2;
    Elem type;
    float *pm, *pl, *pacc;                            // records: [rec][head], [rec][head], [rec][head][hd]
    int32_t *err;
    int32_t cluster;  // blocks of a cluster (1: none), which split a unit's keys in place of ns
    int32_t n_stretches;  // of the tiles' list (set by the launcher); run[x].kind is the first run of stretch x
    int32_t out32;  // out's rows and heads start on 32-byte boundaries (set by the launcher)
    bool vec;       // rows on 16-byte boundaries, heads of whole 16 bytes
    bool overlap;   // the launch may start before the one in front of it on the stream has ended
};

// Tensor-core tiles (pkv_ragged_tc.h): 128 / P consecutive queries x P heads of
// a kv head, P the largest divisor of the group up to 16 (117 rows of 128 at worst);
// a piece is two of them, one of heads wider than 128, and a split of the 128-key
// tiles, the prefix's and then the run's.
constexpr int32_t kRaggedKeyTile = 128;
inline int ragged_tile_heads(int group) {
    int p = group < 16 ? group : 16;
    while (group % p != 0) --p;
    return p;
}
constexpr int32_t ragged_piece_tokens(int heads, int hd) { return (hd > 128 ? 1 : 2) * (128 / heads); }
constexpr int32_t ragged_pieces(int32_t nq, int tokens) { return (nq + tokens - 1) / tokens; }
constexpr int32_t ragged_key_tiles(int32_t n_pre, int32_t nk) {
    return (n_pre + kRaggedKeyTile - 1) / kRaggedKeyTile + (nk + kRaggedKeyTile - 1) / kRaggedKeyTile;
}
constexpr int32_t ragged_split_tiles(int32_t n_pre, const RaggedRun &r) { return (ragged_key_tiles(n_pre, r.nk) + r.ns - 1) / r.ns; }
// TMA's alignment rules, and a positive finite scale (the kernel masks with
// -inf before it scales).
inline bool ragged_tc_takes(const RaggedArgs &a) { return a.vec && a.scale_log2 > 0.f && a.scale_log2 <= 3e38f; }
// Keys that a piece of heads wider than 128, or of sequences that share tiles,
// may add up (the tensor core rounds sums toward zero; other pieces set longer
// ones aside).
constexpr int32_t kRaggedSumKeys = 16384 - 2 * kRaggedKeyTile;
// With n_stretches, run[first[x]] .. are sequences whose queries and own key rows
// follow one another; their tiles are those of the whole stretch (ns and rec0 of its first
// run count).  Stretches in the order of their queries.
cudaError_t launch_ragged_tc(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches,
                             cudaStream_t s);
cudaError_t launch_ragged_tc_bf16(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches,
                                  cudaStream_t s);
cudaError_t launch_ragged_tc_f16(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches,
                                 cudaStream_t s);

// Few query rows by warp-level MMAs (pkv_ragged_rows.cu): units of 8 * wide
// rows ((query, head of the group) pairs) of one kv head; wide 1, 2 or, for heads up to 128, 4
// (2 where rows are not vec).
cudaError_t launch_ragged_rows(const RaggedArgs &a, const RaggedRun *runs, int32_t n, int wide, cudaStream_t s);
__host__ __device__ constexpr int32_t ragged_row_units(int32_t rows, int wide) { return (rows + 8 * wide - 1) / (8 * wide); }
cudaError_t launch_ragged_join(const RaggedArgs &a, const JoinRun *runs, int32_t n, cudaStream_t s);

// Rotary positions with several axes (pkv_rope.cu).
constexpr int32_t kRopeAxes = 4, kRopePairs = 128;
struct RopePacked {
    const void *src[2];        // Q, K
    void *dst[2];
    int64_t src_stride[2], dst_stride[2];
    int32_t heads[2];          // 0: left out
    const int32_t *pos;        // [axis][row]
    int64_t pos_stride;
    int32_t n_rows, hd, n_pairs, inverse;
    Elem type;
    bool vec;
    uint64_t step[kRopePairs]; // turns a position, as a fraction of 2^64
    uint8_t axis[kRopePairs];
};
cudaError_t launch_rope_packed(const RopePacked &a, cudaStream_t s);

// pkv_host.cpp: the current device's error word of calls without a pool (its
// set-up, at the first use, cannot be captured).
int contiguous_error_word(cudaStream_t s, int32_t **out);

}  // namespace pkv

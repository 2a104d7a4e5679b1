// pkv_ragged_host.cpp -- entry points of cross attention, shared-prefix
// attention and multi-axis rotary positions: argument checks, the plan of a
// call (which sequences run on which kernel, how their keys are split, where
// partial records go) and its launches.
#include "../../include/pkv.h"
#include "pkv_ragged.h"

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <vector>

using namespace pkv;

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 30;   // query rows, and key rows, of a call

int refuse(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return report_error(code, buf);
}

template <class F>
int guarded(F &&f) {
    try {
        return f();
    } catch (const std::exception &) {
        return report_error(PKV_ERR_ARG, "out of host memory");
    }
}

template <class F>
int counted(int kind, cudaStream_t s, const char *what, F &&f) {
    const cudaError_t e = launch_counted(kind, s, [](void *ctx) { return (*static_cast<std::remove_reference_t<F> *>(ctx))(); }, &f);
    return e == cudaSuccess ? PKV_OK : refuse(PKV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// ------------------------------------------------------------------ plan ----

struct Shape {
    int32_t n_heads, n_kv, hd;
    int32_t group() const { return n_heads / n_kv; }
};

// One sequence of a call, or several in a row that see the same keys.
struct Seq {
    int32_t q0, nq, k0, nk, off;
};

struct Plan {
    std::vector<RaggedRun> tiles_pre;    // the prefix, for the stacked rows of sequences with few
    std::vector<RaggedRun> tiles, rows;  // own keys (behind the prefix, unless stacked); rows: of the prefix too
    std::vector<RaggedRun> shared;       // sequences that share tiles, behind the prefix, in stretches
    std::vector<int32_t> first;          // of the stretches
    std::vector<JoinRun> joins;
    int64_t n_rec = 0;
    bool stacked = false;
    int wide = 1, cluster = 1;
};

// What a call's kernels go by besides its lengths.
struct Kernels {
    bool vec, tc;  // rows on 16-byte boundaries; the tensor-core tiles take them
};

// Maxima, sums and outputs of records start on 32-byte boundaries, as the
// tensor-core kernel stores whole sectors; the workspace itself on 16.
int64_t record_stats(int64_t n_rec, const Shape &sh) { return (n_rec * sh.n_heads + 7) & ~int64_t{7}; }
int64_t record_bytes(int64_t n_rec, const Shape &sh) {
    return n_rec == 0 ? 0 : 16 + 4 * (2 * record_stats(n_rec, sh) + n_rec * sh.n_heads * sh.hd);
}

// Keys of a cluster's block up to which a cluster is worth it: with more, more
// blocks than a cluster has are.
constexpr int64_t kClusterKeys = 512;

// Query rows a unit of the row kernel takes, in eights: a unit reads its keys
// once, which costs about as much as the arithmetic of two eights.
int pick_wide(const std::vector<RaggedRun> &runs, const Shape &sh, const Kernels &k) {
    if (!k.vec) return 2;
    int best = 1;
    int64_t least = -1;
    for (int wide = 1; wide <= (sh.hd > 128 ? 2 : 4); wide *= 2) {
        int64_t cost = 0;
        for (const RaggedRun &r : runs) cost += static_cast<int64_t>(ragged_row_units(r.nq * sh.group(), wide)) * (2 + wide) * (r.nk + 1);
        if (least < 0 || cost < least) least = cost, best = wide;
    }
    return best;
}

// Units of the row kernel that the GPU holds at once: four blocks a SM, two of wide heads.
int64_t row_slots(const Shape &sh) { return static_cast<int64_t>(kSMs) * (sh.hd > 128 ? 2 : 4); }

// The least number of keys (or key tiles) a split, from `least` to `most`, with which
// no more than `room` units come out; total(per) counts them.
template <class F>
int64_t least_split(int64_t least, int64_t most, int64_t room, F &&total) {
    while (least < most) {
        const int64_t mid = least + (most - least) / 2;
        if (total(mid) <= room) most = mid;
        else least = mid + 1;
    }
    return least;
}

// Splits of the row kernel.  Where there are few units, three quarters of what the
// GPU holds at once (three documents of 50,000 to 120,000 keys: 208 us, with all of
// it 218, with twice as many 216); where whole runs nearly fill it, runs longer than
// a slot's share are split (200 runs of 100 to 2,000 keys: 84 us, with half the
// share 92).  `coarse` times as many keys a split where the workspace is
// short.  A split below 256 keys is mostly latency.
void split_rows(std::vector<RaggedRun> &runs, const Shape &sh, int wide, int64_t n_pre, int64_t coarse) {
    int64_t work = 0, units = 0, most = 256;
    auto keys = [&](const RaggedRun &r) { return (r.kind == kOnPrefix ? 0 : n_pre) + r.nk; };
    auto blocks = [&](const RaggedRun &r) { return static_cast<int64_t>(ragged_row_units(r.nq * sh.group(), wide)) * sh.n_kv; };
    for (const RaggedRun &r : runs) {
        units += blocks(r);
        work += blocks(r) * keys(r);
        most = std::max(most, keys(r));
    }
    const int64_t slots = row_slots(sh), few = slots * 3 / 4;
    int64_t per = (work + slots - 1) / slots;
    if (2 * units <= slots)
        per = least_split(256, most, few, [&](int64_t x) {
            int64_t n = 0;
            for (const RaggedRun &r : runs) n += blocks(r) * ((keys(r) + x - 1) / x);
            return n;
        });
    per = std::max<int64_t>(256, per) * coarse;
    for (RaggedRun &r : runs) r.ns = static_cast<int32_t>(std::clamp<int64_t>((keys(r) + per - 1) / per, 1, 128));
}

// Blocks of a cluster that share a unit's keys, for launches so small that
// every block of every cluster runs at once and a join launch behind would
// take as long as they do; 1: not such a launch.
int pick_cluster(const std::vector<RaggedRun> &runs, const Shape &sh, const Kernels &k, int32_t n_pre) {
    const int wide = pick_wide(runs, sh, k);
    int64_t units = 0, most = 0;
    for (const RaggedRun &r : runs) {
        units += static_cast<int64_t>(ragged_row_units(r.nq * sh.group(), wide)) * sh.n_kv;
        most = std::max<int64_t>(most, n_pre + r.nk);
    }
    const int64_t room = row_slots(sh);
    int n = 1;
    while (n < 8 && units * 2 * n <= room && most > 64 * n) n *= 2;
    return most <= kClusterKeys * n ? n : 1;
}

// Splits of the tensor-core kernel, which runs a block a SM: the least key tiles a
// split with which there is one round of blocks, where that is sooner done by
// the times measured, in hundredths of a us: a piece takes 4 and 1.3 a key
// tile, 3 more with records to write, the join of n rows and heads 3 and 1 a thousand (64 queries
// over 1,024 keys, 8 tiles: 17 us in one piece a kv head, 21 split; over 2,048:
// 28 and 20).  `joined`: the records are joined with others anyway, and other rows
// are attended at the same time, which a quarter of the SMs is left to.
void split_tiles(std::vector<RaggedRun> &runs, const Shape &sh, int32_t n_pre, int64_t coarse, bool joined = false) {
    const int heads = ragged_tile_heads(sh.group());  // of a tile
    int64_t pieces = 0, most = 0, rows = 0;
    auto blocks = [&](const RaggedRun &r) { return static_cast<int64_t>(ragged_pieces(r.nq, ragged_piece_tokens(heads, sh.hd))) * (sh.n_heads / heads); };
    for (RaggedRun &r : runs) {
        r.ns = 1;
        pieces += blocks(r);
        most = std::max<int64_t>(most, ragged_key_tiles(n_pre, r.nk));
        rows += static_cast<int64_t>(r.nq) * sh.n_heads;
    }
    const int64_t room = joined ? kSMs * 3 / 4 : kSMs;
    if (pieces > room || most < 4) return;
    const int64_t per = coarse * least_split(2, most, room, [&](int64_t x) {
        int64_t n = 0;
        for (const RaggedRun &r : runs) n += blocks(r) * ((ragged_key_tiles(n_pre, r.nk) + x - 1) / x);
        return n;
    });
    if (!joined && 400 + 130 * most <= 700 + 130 * per + 300 + rows / 10) return;
    for (RaggedRun &r : runs) r.ns = static_cast<int32_t>((ragged_key_tiles(n_pre, r.nk) + per - 1) / per);
}

// Query rows of a tensor-core tile (queries x heads of the group) from which a
// sequence takes it: 24 sequences over 700 to 1,500 keys take 38 us there and 54 on the row kernel at 6
// queries of 4 heads a kv head, 43 to 48 and 42 to 43 at 12 of one.
constexpr int64_t kTileRows = 24;

// Stretches of neighbouring sequences that share tiles.  A tile's rows
// multiply the own keys of all its sequences, so a sequence takes part where that is
// no more than two tiles of keys, or half of the prefix, on top: a few tokens behind a long history of
// their own do not, nor do sequences in slots far apart.  (64-wide heads have less to
// gain, as a tile by itself takes both chains: 121 sequences of 84 to 110 queries in slots of 400
// rows behind 1,493, 20 heads of 64: 222 us by themselves, 239 together; 39 of 25 to 209 in
// slots of 216, 12 heads of 80: 91 and 79.)
std::vector<std::vector<Seq>> find_stretches(std::vector<Seq> &seqs, const Shape &sh, int32_t n_pre) {
    const int heads = ragged_tile_heads(sh.group());  // of a tile
    const int64_t pair = ragged_piece_tokens(heads, sh.hd), most = std::max<int64_t>(2, ragged_key_tiles(n_pre, 0) / 2);
    std::vector<std::vector<Seq>> found;
    std::vector<Seq> alone, run;
    int64_t rows = 0;
    auto close = [&] {
        // (half a piece at least: the prefix costs a piece the same for fewer rows)
        const bool take = run.size() > 1 && rows * heads >= kTileRows && 2 * rows >= pair;
        if (take) found.push_back(run);
        else alone.insert(alone.end(), run.begin(), run.end());
        run.clear();
        rows = 0;
    };
    for (const Seq &s : seqs) {
        const bool fits = s.off != kSees && s.off * pair <= 128 * most * s.nq && n_pre + s.nk <= kRaggedSumKeys;
        const int64_t gap = run.empty() ? 0 : int64_t{s.k0} - run.back().k0 - run.back().nk;  // key rows between that nobody sees
        const bool follows = !run.empty() && s.q0 == run.back().q0 + run.back().nq && gap >= 0 && (s.off + gap) * pair <= 128 * most * s.nq &&
                             (sh.hd > 64 || gap <= 32);
        if (!fits || (!run.empty() && !follows)) close();
        if (!fits) {
            alone.push_back(s);
            continue;
        }
        run.push_back(s);
        rows += s.nq;
    }
    close();
    seqs = alone;
    return found;
}

// Whether sequences with few queries attend the prefix together: reading it once a
// unit (at 6 TB/s from L2) against a further launch and a join, by the times measured
// (143 sequences of 4 queries behind 181 keys, 32 heads over 8: 58 us stacked, 34 not).
bool worth_stacking(const std::vector<RaggedRun> &runs, const Shape &sh, const Kernels &k, int32_t n_pre) {
    const int wide = pick_wide(runs, sh, k);
    int64_t units = 0, rows = 0;
    for (const RaggedRun &r : runs) {
        units += static_cast<int64_t>(ragged_row_units(r.nq * sh.group(), wide)) * sh.n_kv;
        rows += static_cast<int64_t>(r.nq) * sh.n_heads;
    }
    return units * n_pre * sh.hd * 4 / 6000 > 15000 + rows;  // ns
}

// Whether sequences with few queries go with the others' tiles, which saves a launch of
// their own: where they add no more than twice the others' key tiles.  24 prompts of
// 4 to 448 queries, 7 of them with few, over 700 to 1,500 keys, 20 heads of 64: 58 us in
// two launches, 49 in one; with one of few, 32 heads over 8 of 128: 58 and 42; one prompt and one
// token: 10 and 7 to 9; but 200 tokens and one prompt, over 1,000 keys each: 165 and 201.
template <class Can, class Takes>
bool goes_along(const std::vector<Seq> &seqs, const Shape &sh, Can &&can, Takes &&takes) {
    const int32_t tokens = ragged_piece_tokens(ragged_tile_heads(sh.group()), sh.hd);
    int64_t few = 0, many = 0;
    for (const Seq &s : seqs) {
        if (!can(s.nk)) continue;
        (takes(s.nq, s.nk) ? many : few) += static_cast<int64_t>(ragged_pieces(s.nq, tokens)) * ragged_key_tiles(0, s.nk);
    }
    return few > 0 && few <= 2 * many;
}

// The plan of up to kRaggedLarge sequences; with less workspace than it would
// like, keys are split less, or not at all.
Plan make_plan(std::vector<Seq> seqs, const Shape &sh, int32_t n_pre, const Kernels &kernels, int64_t workspace) {
    constexpr int64_t kCoarsest = int64_t{1} << 24;
    const int heads = ragged_tile_heads(sh.group());  // of a tile
    auto can_take_tiles = [&](int32_t keys) { return kernels.tc && keys > 0 && (sh.hd <= 128 || keys <= kRaggedSumKeys); };
    auto takes_tiles = [&](int64_t nq, int32_t keys) { return can_take_tiles(keys) && nq * heads >= kTileRows; };
    std::vector<RaggedRun> own;
    Plan p;
    if (kernels.tc)
        for (const std::vector<Seq> &part : find_stretches(seqs, sh, n_pre)) {
            p.first.push_back(static_cast<int32_t>(p.shared.size()));
            for (const Seq &s : part) p.shared.push_back(RaggedRun{s.q0, s.nq, s.k0, s.nk, s.off, 1, -1, kOwnKeys});
        }
    // a stretch as one run, with the own keys of an average piece
    std::vector<RaggedRun> whole;
    for (size_t x = 0; x < p.first.size(); ++x) {
        const RaggedRun &f = p.shared[p.first[x]], &e = p.shared[(x + 1 < p.first.size() ? p.first[x + 1] : p.shared.size()) - 1];
        const int32_t nq = e.q0 + e.nq - f.q0, pieces = ragged_pieces(nq, ragged_piece_tokens(heads, sh.hd));
        whole.push_back(RaggedRun{f.q0, nq, f.k0, std::max(std::max(f.nk, e.nk), (e.k0 + e.nk - f.k0 + pieces - 1) / pieces), 0, 1, -1, kOwnKeys});
    }
    const bool along = n_pre == 0 && goes_along(seqs, sh, can_take_tiles, takes_tiles);
    for (const Seq &s : seqs)
        ((along && can_take_tiles(s.nk)) || takes_tiles(s.nq, n_pre + s.nk) ? p.tiles : own).push_back(RaggedRun{s.q0, s.nq, s.k0, s.nk, s.off, 1, -1, kOwnKeys});
    for (int64_t coarse = workspace < record_bytes(1, sh) ? 2 * kCoarsest : 1;; coarse *= 2) {
        const bool last = coarse > kCoarsest;
        p.cluster = pick_cluster(own, sh, kernels, n_pre);
        p.stacked = !last && p.cluster == 1 && n_pre >= 128 && own.size() > 1 && worth_stacking(own, sh, kernels, n_pre);
        p.rows.clear();
        p.tiles_pre.clear();
        p.joins.clear();
        std::vector<RaggedRun> stacks;  // neighbours together, over the prefix
        if (p.stacked) {
            for (const RaggedRun &r : own) {
                if (!stacks.empty() && stacks.back().q0 + stacks.back().nq == r.q0) stacks.back().nq += r.nq;
                else stacks.push_back(RaggedRun{r.q0, r.nq, 0, n_pre, kSees, 1, -1, kOnPrefix});
            }
            for (RaggedRun &r : stacks) {
                const bool tiles = takes_tiles(r.nq, n_pre);
                r.kind = tiles ? kOwnKeys : kOnPrefix;
                (tiles ? p.tiles_pre : p.rows).push_back(r);
            }
        }
        const size_t n_stacks = p.rows.size();
        p.rows.insert(p.rows.end(), own.begin(), own.end());
        p.wide = pick_wide(p.rows, sh, kernels);
        if (last) {
            for (RaggedRun &r : p.tiles) r.ns = 1;
            for (RaggedRun &r : whole) r.ns = 1;
        } else {
            split_tiles(whole, sh, n_pre, coarse);
            if (p.cluster == 1) split_rows(p.rows, sh, p.wide, p.stacked ? 0 : n_pre, coarse);
            split_tiles(p.tiles, sh, n_pre, coarse);
            split_tiles(p.tiles_pre, sh, 0, coarse, true);
        }
        // records, run by run
        int64_t at = 0;
        auto records = [&](RaggedRun &r) {
            r.rec0 = static_cast<int32_t>(std::min<int64_t>(at, 0x7fffffff));
            at += static_cast<int64_t>(r.nq) * r.ns;
        };
        for (RaggedRun &r : p.tiles_pre) records(r);
        size_t rows_at = 0, tiles_at = 0;  // the next stacks (both lists are in the order of the queries)
        const RaggedRun *stack = nullptr;
        for (size_t i = 0; i < p.rows.size(); ++i) {
            RaggedRun &r = p.rows[i];
            r.rec0 = -1;
            if (i < n_stacks) {
                records(r);
                continue;
            }
            if (!p.stacked) {
                if (r.ns == 1) continue;
                records(r);
                p.joins.push_back(JoinRun{r.q0, r.nq, r.rec0, r.ns, 0, 0});
                continue;
            }
            if (!stack || r.q0 >= stack->q0 + stack->nq)
                stack = rows_at < n_stacks && r.q0 >= p.rows[rows_at].q0 && r.q0 < p.rows[rows_at].q0 + p.rows[rows_at].nq
                            ? &p.rows[rows_at++]
                            : &p.tiles_pre[tiles_at++];
            records(r);
            const int64_t pre0 = stack->rec0 + static_cast<int64_t>(r.q0 - stack->q0) * stack->ns;
            p.joins.push_back(JoinRun{r.q0, r.nq, r.rec0, r.ns, static_cast<int32_t>(std::min<int64_t>(pre0, 0x7fffffff)), stack->ns});
        }
        for (RaggedRun &r : p.tiles) {
            r.rec0 = -1;
            if (r.ns == 1) continue;
            records(r);
            p.joins.push_back(JoinRun{r.q0, r.nq, r.rec0, r.ns, 0, 0});
        }
        for (size_t x = 0; x < whole.size(); ++x) {
            RaggedRun &r = whole[x], &f = p.shared[p.first[x]];
            r.rec0 = -1;
            if (r.ns > 1) {
                records(r);
                p.joins.push_back(JoinRun{r.q0, r.nq, r.rec0, r.ns, 0, 0});
            }
            f.ns = r.ns;
            f.rec0 = r.rec0;
        }
        p.n_rec = at;
        if (at > 0 && (at > 0x7fffffff || record_bytes(at, sh) > workspace)) continue;
        // the longest pieces and splits first: the launches then end on their shortest
        std::stable_sort(p.rows.begin(), p.rows.end(), [&](const RaggedRun &x, const RaggedRun &y) { return x.nk / x.ns > y.nk / y.ns; });
        auto length = [&](const RaggedRun &r) { return ragged_split_tiles(n_pre, r) * (r.nq * heads > 128 ? 2 : 1); };
        std::stable_sort(p.tiles.begin(), p.tiles.end(), [&](const RaggedRun &x, const RaggedRun &y) { return length(x) > length(y); });
        return p;
    }
}

// ------------------------------------------------------------------ calls ----

struct Call {
    const void *Q, *K, *V, *Kp, *Vp;
    void *out;
    int64_t q_stride, k_stride, v_stride, kp_stride, vp_stride, o_stride;
    int64_t q_rows, k_rows;  // that Q and out, and K and V, have
    int32_t dtype, n_pre;
    bool causal;  // own keys j <= k_len - q_len + i; otherwise all
    const int32_t *q_lens, *k_lens, *k_start;
    int32_t n_seqs;
    Shape sh;
    float scale;
    void *workspace;
    int64_t workspace_bytes;
};

// Sizes and grouping of a call, and its sequences with queries.
int sequences(const Call &c, std::vector<Seq> &seqs, int64_t *q_reach, int64_t *k_reach) {
    if (c.n_seqs <= 0 || !c.q_lens || !c.k_lens)
        return refuse(PKV_ERR_BAD_DIM, "n_seqs must be positive and the lengths non-NULL");
    if (c.sh.n_heads <= 0 || c.sh.n_kv <= 0 || c.sh.hd <= 0)
        return refuse(PKV_ERR_BAD_DIM, "n_heads, n_kv_heads and head_dim must be positive");
    if (c.sh.hd > kMaxHeadDim) return refuse(PKV_ERR_BAD_DIM, "head_dim %d > %d is not supported", c.sh.hd, kMaxHeadDim);
    if (c.n_pre < 0 || c.n_pre > kMaxRows - 256) return refuse(PKV_ERR_BAD_DIM, "a prefix of %d rows", c.n_pre);
    int64_t q = 0, k = 0;
    *k_reach = 0;
    for (int32_t s = 0; s < c.n_seqs; ++s) {
        const int32_t nq = c.q_lens[s], nk = c.k_lens[s];
        if (nq < 0 || nk < 0) return refuse(PKV_ERR_BAD_DIM, "sequence %d has a negative length", s);
        if (c.causal && nq > nk)
            return refuse(PKV_ERR_BAD_DIM, "sequence %d has %d queries and %d keys of its own: its queries' keys come last among them", s, nq, nk);
        const int64_t k0 = c.k_start ? c.k_start[s] : k;
        if (k0 < 0 || k0 + nk > kMaxRows - 256) return refuse(PKV_ERR_BAD_DIM, "sequence %d: key rows %lld and on", s, static_cast<long long>(k0));
        if (q + nq > kMaxRows) return refuse(PKV_ERR_BAD_DIM, "too many query rows");
        if (nq > 0) {
            const Seq x{static_cast<int32_t>(q), nq, static_cast<int32_t>(k0), nk, c.causal ? nk - nq : kSees};
            // neighbours that see the same keys (beams of one request) are one
            if (!c.causal && !seqs.empty() && seqs.back().k0 == x.k0 && seqs.back().nk == nk) seqs.back().nq += nq;
            else seqs.push_back(x);
        }
        if (nk > 0) *k_reach = std::max(*k_reach, k0 + nk);
        q += nq;
        k += nk;
    }
    *q_reach = q;
    if (q * c.sh.n_heads > 0x7fff0000LL) return refuse(PKV_ERR_BAD_DIM, "%lld query rows of %d heads are too many", static_cast<long long>(q), c.sh.n_heads);
    if (static_cast<int64_t>(c.sh.n_heads) * c.sh.hd > 0x7fffffffLL) return refuse(PKV_ERR_BAD_DIM, "n_heads * head_dim too large");
    if (c.sh.n_heads % c.sh.n_kv != 0)
        return refuse(PKV_ERR_BAD_GQA, "n_heads (%d) is not a multiple of n_kv_heads (%d)", c.sh.n_heads, c.sh.n_kv);
    return PKV_OK;
}

template <class F>
int each_chunk(const std::vector<Seq> &seqs, F &&f) {
    for (size_t i = 0; i < seqs.size(); i += kRaggedLarge) {
        const size_t n = std::min<size_t>(kRaggedLarge, seqs.size() - i);
        const int rc = f(std::vector<Seq>(seqs.begin() + i, seqs.begin() + i + n));
        if (rc) return rc;
    }
    return PKV_OK;
}

int64_t workspace_of(const Call &c) {
    std::vector<Seq> seqs;
    int64_t q, k;
    if (sequences(c, seqs, &q, &k)) return -1;
    int64_t most = 0;
    each_chunk(seqs, [&](const std::vector<Seq> &part) {
        // (alignment and scale, which a call's kernels go by too, are not known here)
        const bool vec = c.sh.hd % 8 == 0, tc = vec;
        for (const Kernels k : {Kernels{false, false}, Kernels{vec, false}, Kernels{vec, tc}})
            most = std::max(most, record_bytes(make_plan(part, c.sh, c.n_pre, k, int64_t{1} << 62).n_rec, c.sh));
        return PKV_OK;
    });
    return most;
}

int attend(const Call &c, cudaStream_t st) {
    std::vector<Seq> seqs;
    int64_t q, k;
    int rc = sequences(c, seqs, &q, &k);
    if (rc) return rc;
    if (c.dtype != PKV_BF16 && c.dtype != PKV_F16) return refuse(PKV_ERR_ARG, "packed attention takes PKV_BF16 or PKV_F16 rows");
    const int64_t q_dim = static_cast<int64_t>(c.sh.n_heads) * c.sh.hd, kv_dim = static_cast<int64_t>(c.sh.n_kv) * c.sh.hd;
    if (c.q_stride < q_dim || c.o_stride < q_dim || c.k_stride < kv_dim || c.v_stride < kv_dim ||
        (c.n_pre > 0 && (c.kp_stride < kv_dim || c.vp_stride < kv_dim)))
        return refuse(PKV_ERR_ARG, "a row stride below the row's width makes rows overlap");
    if (std::max({c.q_stride, c.o_stride, c.k_stride, c.v_stride, c.kp_stride, c.vp_stride}) > (int64_t{1} << 32))
        return refuse(PKV_ERR_BAD_DIM, "row stride too large");
    if (c.workspace_bytes < 0 || (c.workspace_bytes > 0 && !c.workspace)) return refuse(PKV_ERR_ARG, "workspace");
    if (reinterpret_cast<uintptr_t>(c.workspace) % 16 != 0) return refuse(PKV_ERR_ARG, "the workspace must be aligned to 16 bytes");
    if (q > c.q_rows || k > c.k_rows)
        return refuse(PKV_ERR_ARG, "the sequences reach over %lld query and %lld key rows, there are %lld and %lld", static_cast<long long>(q),
                      static_cast<long long>(k), static_cast<long long>(c.q_rows), static_cast<long long>(c.k_rows));
    if (seqs.empty()) return PKV_OK;
    if (!c.Q || !c.out || (k > 0 && (!c.K || !c.V)) || (c.n_pre > 0 && (!c.Kp || !c.Vp)))
        return refuse(PKV_ERR_ARG, "NULL data pointer");
    for (const void *p : {c.Q, c.K, c.V, c.Kp, c.Vp, static_cast<const void *>(c.out)})
        if (reinterpret_cast<uintptr_t>(p) % 2 != 0) return refuse(PKV_ERR_ARG, "rows must be aligned to their element");

    RaggedArgs a{};
    a.Q = c.Q;
    a.K = c.K;
    a.V = c.V;
    a.out = c.out;
    a.q_stride = c.q_stride;
    a.k_stride = c.k_stride;
    a.v_stride = c.v_stride;
    a.o_stride = c.o_stride;
    a.Kp = c.Kp;
    a.Vp = c.Vp;
    a.kp_stride = c.kp_stride;
    a.vp_stride = c.vp_stride;
    a.n_pre = c.n_pre;
    a.cluster = 1;
    a.n_heads = c.sh.n_heads;
    a.n_kv = c.sh.n_kv;
    a.hd = c.sh.hd;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    a.type = c.dtype == PKV_BF16 ? Elem::bf16 : Elem::f16;
    auto whole = [](const void *p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; };
    a.vec = c.sh.hd % 8 == 0 && whole(c.Q, c.q_stride) && whole(c.K, c.k_stride) && whole(c.V, c.v_stride) &&
            whole(c.out, c.o_stride) && (c.n_pre == 0 || (whole(c.Kp, c.kp_stride) && whole(c.Vp, c.vp_stride)));
    const Kernels kernels{a.vec, ragged_tc_takes(a)};
    return each_chunk(seqs, [&](const std::vector<Seq> &part) {
        const Plan p = make_plan(part, c.sh, c.n_pre, kernels, c.workspace_bytes);
        if (!a.err && !(p.tiles.empty() && p.tiles_pre.empty() && p.shared.empty())) {
            const int r = contiguous_error_word(st, &a.err);
            if (r) return r;
        }
        a.pm = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(c.workspace) + 31) & ~uintptr_t{31});
        a.pl = a.pm + record_stats(p.n_rec, c.sh);
        a.pacc = a.pl + record_stats(p.n_rec, c.sh);
        bool first = true;
        enum { kRows, kTiles, kShared };
        auto run = [&](RaggedArgs b, const std::vector<RaggedRun> &runs, int how) {
            for (size_t i = 0; i < runs.size(); i += kRaggedLarge) {
                const int32_t n = static_cast<int32_t>(std::min<size_t>(kRaggedLarge, runs.size() - i));
                b.overlap = !first;
                first = false;
                const int r = how == kRows ? counted(PKV_KERNEL_DECODE, st, "ragged attention rows",
                                                     [&] { return launch_ragged_rows(b, &runs[i], n, p.wide, st); })
                                           : counted(PKV_KERNEL_PREFILL, st, "ragged attention tiles",
                                                     [&] {
                                                         return launch_ragged_tc(b, &runs[i], n, p.first.data(),
                                                                                 how == kShared ? static_cast<int32_t>(p.first.size()) : 0, st);
                                                     });
                if (r) return r;
            }
            return static_cast<int>(PKV_OK);
        };
        RaggedArgs pre = a, own = a;  // the prefix as a run's keys; own keys of sequences whose rows are stacked over it
        pre.K = c.Kp;
        pre.V = c.Vp;
        pre.k_stride = c.kp_stride;
        pre.v_stride = c.vp_stride;
        pre.n_pre = 0;
        own.n_pre = p.stacked ? 0 : c.n_pre;
        own.cluster = p.cluster;
        int r = run(a, p.shared, kShared);
        if (!r) r = run(a, p.tiles, kTiles);
        if (!r) r = run(pre, p.tiles_pre, kTiles);
        if (!r) r = run(own, p.rows, kRows);
        if (r || p.joins.empty()) return r;
        return counted(PKV_KERNEL_MERGE, st, "ragged join kernel",
                       [&] { return launch_ragged_join(a, p.joins.data(), static_cast<int32_t>(p.joins.size()), st); });
    });
}

// ------------------------------------------------------------------- rope ----

int rope(const void *Q, int64_t q_stride, const void *K, int64_t k_stride, int32_t dtype, const int32_t *pos,
         int64_t pos_stride, int32_t n_axes, const int32_t *pairs, int32_t order, int32_t n_rows, int32_t n_heads,
         int32_t n_kv_heads, int32_t head_dim, double base, int32_t inverse, void *Q_out, int64_t qo_stride, void *K_out,
         int64_t ko_stride, cudaStream_t st) {
    if (n_rows < 0 || n_rows > kMaxRows) return refuse(PKV_ERR_BAD_DIM, "%d rows", n_rows);
    if (n_axes <= 0 || n_axes > kRopeAxes || !pairs) return refuse(PKV_ERR_BAD_DIM, "one to %d axes, with their pairs", kRopeAxes);
    if ((Q && n_heads <= 0) || (K && n_kv_heads <= 0) || head_dim <= 0)
        return refuse(PKV_ERR_BAD_DIM, "n_heads, n_kv_heads and head_dim must be positive");
    if (head_dim > kMaxHeadDim) return refuse(PKV_ERR_BAD_DIM, "head_dim %d > %d is not supported", head_dim, kMaxHeadDim);
    int64_t total = 0;
    for (int32_t a = 0; a < n_axes; ++a) {
        if (pairs[a] < 0) return refuse(PKV_ERR_BAD_DIM, "axis %d has %d pairs", a, pairs[a]);
        total += pairs[a];
    }
    if (total <= 0 || 2 * total > head_dim)
        return refuse(PKV_ERR_BAD_DIM, "%lld pairs in heads of %d", static_cast<long long>(total), head_dim);
    const int64_t q_dim = Q ? static_cast<int64_t>(n_heads) * head_dim : 0, k_dim = K ? static_cast<int64_t>(n_kv_heads) * head_dim : 0;
    if (q_dim + k_dim > (1 << 26)) return refuse(PKV_ERR_BAD_DIM, "heads * head_dim too large");
    if (dtype != PKV_F32 && dtype != PKV_BF16 && dtype != PKV_F16) return refuse(PKV_ERR_ARG, "unknown dtype %d", dtype);
    if (order != PKV_ROPE_BLOCKS && order != PKV_ROPE_TURNS && order != PKV_ROPE_AXIAL) return refuse(PKV_ERR_ARG, "unknown order %d", order);
    if (!(base >= 1.0) || !std::isfinite(base)) return refuse(PKV_ERR_ARG, "rope_base must be finite and at least 1");
    const int32_t n = static_cast<int32_t>(total);

    RopePacked a{};
    int32_t count[kRopeAxes] = {};
    double turns = 0.0, fall = 1.0;
    for (int32_t i = 0, axis = 0, first = 0; i < n; ++i) {
        while (i >= first + pairs[axis]) first += pairs[axis++];
        int32_t mine = axis, number = i, ramp = n;
        if (order == PKV_ROPE_TURNS) {
            mine = i % n_axes;
            if (i >= static_cast<int64_t>(n_axes) * pairs[mine]) mine = 0;
        } else if (order == PKV_ROPE_AXIAL) {
            number = i - first;
            ramp = pairs[axis];
        }
        ++count[mine];
        a.axis[i] = static_cast<uint8_t>(mine);
        // turns a position; a ramp falls by one factor a pair, with a power every
        // fourth (64 powers take 1 us; three products between cost 2^-50 at most); the
        // step is cut to whole 2^-64 turns
        if (number % 4 == 0) {
            turns = std::pow(base, -static_cast<double>(number) / ramp) / 6.283185307179586477;
            if (number == 0) fall = std::pow(base, -1.0 / ramp);
        } else {
            turns *= fall;
        }
        a.step[i] = static_cast<uint64_t>(std::ldexp(turns, 64));
    }
    for (int32_t x = 0; x < n_axes; ++x)
        if (count[x] != pairs[x])
            return refuse(PKV_ERR_BAD_DIM, "pairs dealt in turn give axis %d %d of them, not %d", x, count[x], pairs[x]);

    if ((Q && (q_stride < q_dim || qo_stride < q_dim)) || (K && (k_stride < k_dim || ko_stride < k_dim)))
        return refuse(PKV_ERR_ARG, "a row stride below the row's width makes rows overlap");
    if (std::max({q_stride, k_stride, qo_stride, ko_stride, pos_stride}) > (int64_t{1} << 32)) return refuse(PKV_ERR_BAD_DIM, "row stride too large");
    if (n_axes > 1 && pos_stride != 0 && pos_stride < n_rows) return refuse(PKV_ERR_ARG, "the axes' positions overlap");
    if (n_rows == 0) return PKV_OK;
    if ((!Q && !K) || !pos || (Q && !Q_out) || (K && !K_out) || (!Q && Q_out) || (!K && K_out))
        return refuse(PKV_ERR_ARG, "NULL data pointer (a left out part has neither rows nor a place for them)");
    const uintptr_t size = dtype == PKV_F32 ? 4 : 2;
    for (const void *p : {Q, K, static_cast<const void *>(Q_out), static_cast<const void *>(K_out)})
        if (reinterpret_cast<uintptr_t>(p) % size != 0) return refuse(PKV_ERR_ARG, "rows must be aligned to their element");
    if (reinterpret_cast<uintptr_t>(pos) % 4 != 0) return refuse(PKV_ERR_ARG, "positions must be aligned to 4 bytes");
    if ((Q && Q == Q_out && q_stride != qo_stride) || (K && K == K_out && k_stride != ko_stride))
        return refuse(PKV_ERR_ARG, "rows turned in place keep their stride");
    a.src[0] = Q;
    a.src[1] = K;
    a.dst[0] = Q_out;
    a.dst[1] = K_out;
    a.src_stride[0] = q_stride;
    a.src_stride[1] = k_stride;
    a.dst_stride[0] = qo_stride;
    a.dst_stride[1] = ko_stride;
    a.heads[0] = Q ? n_heads : 0;
    a.heads[1] = K ? n_kv_heads : 0;
    a.pos = pos;
    a.pos_stride = n_axes > 1 ? pos_stride : 0;
    a.n_rows = n_rows;
    a.hd = head_dim;
    a.n_pairs = n;
    a.inverse = inverse ? 1 : 0;
    a.type = dtype == PKV_F32 ? Elem::f32 : dtype == PKV_BF16 ? Elem::bf16 : Elem::f16;
    return counted(PKV_KERNEL_APPEND, st, "rotary kernel", [&] { return launch_rope_packed(a, st); });
}

}  // namespace

extern "C" {

int64_t pkv_attn_cross_workspace(const int32_t *q_lens, const int32_t *k_lens, const int32_t *k_start, int32_t n_seqs,
                                 int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    int64_t n = -1;
    const int rc = guarded([&] {
        Call c{};
        c.q_lens = q_lens;
        c.k_lens = k_lens;
        c.k_start = k_start;
        c.n_seqs = n_seqs;
        c.sh = Shape{n_heads, n_kv_heads, head_dim};
        n = workspace_of(c);
        return static_cast<int>(PKV_OK);
    });
    return rc ? -1 : n;
}

int64_t pkv_attn_prefix_workspace_at(int32_t prefix_len, const int32_t *q_lens, const int32_t *k_lens, const int32_t *k_start,
                                     int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    int64_t n = -1;
    const int rc = guarded([&] {
        Call c{};
        c.n_pre = prefix_len;
        c.causal = true;
        c.q_lens = q_lens;
        c.k_lens = k_lens;
        c.k_start = k_start;
        c.n_seqs = n_seqs;
        c.sh = Shape{n_heads, n_kv_heads, head_dim};
        n = workspace_of(c);
        return static_cast<int>(PKV_OK);
    });
    return rc ? -1 : n;
}

int64_t pkv_attn_prefix_workspace(int32_t prefix_len, const int32_t *q_lens, const int32_t *k_lens, int32_t n_seqs,
                                  int32_t n_heads, int32_t n_kv_heads, int32_t head_dim) {
    return pkv_attn_prefix_workspace_at(prefix_len, q_lens, k_lens, nullptr, n_seqs, n_heads, n_kv_heads, head_dim);
}

int pkv_attn_cross(const void *Q, int64_t q_stride, int64_t q_rows, const int32_t *q_lens, const void *K, int64_t k_stride,
                   const void *V, int64_t v_stride, int64_t k_rows, const int32_t *k_lens, const int32_t *k_start,
                   int32_t dtype, int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale, void *out,
                   int64_t out_stride, void *workspace, int64_t workspace_bytes, pkv_stream_t stream) {
    return guarded([&] {
        Call c{};
        c.Q = Q, c.K = K, c.V = V, c.out = out;
        c.q_stride = q_stride, c.k_stride = k_stride, c.v_stride = v_stride, c.o_stride = out_stride;
        c.q_rows = q_rows, c.k_rows = k_rows;
        c.dtype = dtype;
        c.q_lens = q_lens, c.k_lens = k_lens, c.k_start = k_start, c.n_seqs = n_seqs;
        c.sh = Shape{n_heads, n_kv_heads, head_dim};
        c.scale = scale;
        c.workspace = workspace, c.workspace_bytes = workspace_bytes;
        return attend(c, static_cast<cudaStream_t>(stream));
    });
}

int pkv_attn_prefix(const void *Q, int64_t q_stride, int64_t q_rows, const int32_t *q_lens, const void *K_prefix,
                    int64_t kp_stride, const void *V_prefix, int64_t vp_stride, int32_t prefix_len, const void *K,
                    int64_t k_stride, const void *V, int64_t v_stride, int64_t k_rows, const int32_t *k_lens,
                    const int32_t *k_start, int32_t dtype, int32_t n_seqs, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale, void *out,
                    int64_t out_stride, void *workspace, int64_t workspace_bytes, pkv_stream_t stream) {
    return guarded([&] {
        Call c{};
        c.Q = Q, c.K = K, c.V = V, c.Kp = K_prefix, c.Vp = V_prefix, c.out = out;
        c.q_stride = q_stride, c.k_stride = k_stride, c.v_stride = v_stride, c.o_stride = out_stride;
        c.kp_stride = kp_stride, c.vp_stride = vp_stride;
        c.q_rows = q_rows, c.k_rows = k_rows;
        c.dtype = dtype;
        c.n_pre = prefix_len;
        c.causal = true;
        c.q_lens = q_lens, c.k_lens = k_lens, c.k_start = k_start, c.n_seqs = n_seqs;
        c.sh = Shape{n_heads, n_kv_heads, head_dim};
        c.scale = scale;
        c.workspace = workspace, c.workspace_bytes = workspace_bytes;
        return attend(c, static_cast<cudaStream_t>(stream));
    });
}

int pkv_rope_packed(const void *Q, int64_t q_stride, const void *K, int64_t k_stride, int32_t dtype,
                    const int32_t *positions, int64_t pos_stride, int32_t n_axes, const int32_t *pairs, int32_t order,
                    int32_t n_rows, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, double rope_base,
                    int32_t inverse, void *Q_out, int64_t qo_stride, void *K_out, int64_t ko_stride, pkv_stream_t stream) {
    return guarded([&] {
        return rope(Q, q_stride, K, k_stride, dtype, positions, pos_stride, n_axes, pairs, order, n_rows, n_heads, n_kv_heads,
                    head_dim, rope_base, inverse, Q_out, qo_stride, K_out, ko_stride, static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"

// pkv_internal.h -- descriptors and kernel launchers shared by the host core
// (pkv_host.cpp) and the kernels (pkv_kernels.cu).  Not part of the C ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <vector>

#include <cuda_runtime.h>

namespace pkv {

// One batch row: a sequence appending and attending n_q consecutive rows.
struct RowDesc {
    int32_t slot;      // page-table row of the sequence on the device
    int32_t past_len;  // tokens committed before this call (seq_len)
    int32_t n_q;       // rows appended and attended by this call
    int32_t q_row0;    // first of this row's rows in Q / K_new / V_new / out
    // Shared-prefix (cascade) rows: keys [0, k0) were attended by a prefix
    // pass whose partials are the first s0 records of the query's merge item;
    // the row's decode unit of split s covers k0 + (s - s0) * S .. (S keys).
    // 0, 0 for every other row.
    int32_t k0 = 0, s0 = 0;
};

// One split-K work unit: query qi of row `row`, keys [split*S, (split+1)*S)
// clipped to the visible range.  item >= 0: the query has several splits and
// MergeDesc `item` describes them (this unit's partial record is
// part0 + split); item < 0: the unit writes out directly.
struct UnitDesc {
    int32_t row, qi, split, item;
};

// One query whose splits are combined by the merge kernel.
struct MergeDesc {
    int32_t row, qi, part0, n_split;
};

// One appended token row: position `pos` (in block `blk` of the host page
// table) receives row `src_row` of K_new / V_new.
struct AppendDesc {
    int32_t slot, pos, src_row, blk;
};

// A run of page-table entries to upload: pt[slot][start .. start+count) =
// vals[voff .. voff+count).
struct PtRun {
    int32_t slot, start, count, voff;
};

// One copy-on-append block copy (every layer, K and V).
struct CopyDesc {
    int32_t src, dst;
};

// Address of a key/value row in the paged pool:
//   pool[pt[slot][pos / bs]][layer][pos % bs][kv_head*hd ...]
struct PagedAddr {
    void *k, *v;           // pool storage: f32 elements, or bf16 when bf16 != 0
    int32_t *pt;           // written only by the fused append, for pages no reader of that launch uses
    int64_t block_stride;  // elements per block: n_layers * bs * kv_dim
    int64_t layer_off;     // elements to the layer: layer * bs * kv_dim
    int32_t kv_dim, bs, bs_shift, max_blocks, n_blocks;
    int32_t bf16 = 0;      // storage element: 0 f32, 1 bf16 (rounded to nearest even on write)
    int32_t fp8 = 0;       // 1: fp8 e4m3 elements holding x / kv_scale (saturating)
    float kv_scale = 1.f;  // power of two; 1 unless fp8
};

// An 8-bit pool with block scales: the element u (1 .. 255) of a row of kv head
// h in block b stands for (u - 128) * s, s the scale of (b, layer, h), a power
// of two (NaN: the block took a value that is not finite).
struct Q8Addr {
    PagedAddr a;               // k, v: one byte per element
    float *ks, *vs;            // scales of the layer's first head: block b, head h at b * scale_stride + h
    int64_t scale_stride;      // floats per block: n_layers * n_kv
    int32_t n_kv, hd;
    const void *maps = nullptr;  // host: the pool's Q8Maps where its pages can be loaded by TMA
};

// The rows of one page that a packed append writes, or a packed read returns:
// offsets off .. off + n - 1 of block blk <-> packed rows row0 ..
struct PageItem {
    int32_t blk, off, n, row0;
};

// A block of queries over an 8-bit pool, and one decode unit of it (two lists,
// as the host lays them out).  Queries q_row .. q_row + nq - 1 (rows of Q and
// out), of which query t sees the keys below see0 + t (causal) or kend; the unit
// takes keys [kbeg, kend).  part0 < 0: the unit is the block's only one and
// writes out; else its partial of query t is record part0 + t * n_rec + rec, and
// the last of the block's n_dec units to finish (by the counters cnt ..) joins
// all n_rec records of each query.
struct Q8Block {
    int32_t slot, q_row, nq, see0;
    int32_t part0, n_rec, n_dec, cnt;
};
struct Q8Part {
    int32_t block, kbeg, kend, rec;
};
struct Q8Unit : Q8Block {
    int32_t kbeg, kend, rec;
};

// A call's descriptors where they are few: they travel in the launch's
// parameters instead of through an upload, which the launch waits 7 us for
// (prompts of 9,000 rows: 37.7 -> 22.6 us for their append and read; decode
// of 64 sequences 54.9 -> 47.2 us).  A launch takes longer with more of them
// (one token of 64 sequences: 16.3 us with the small blob, 19.3 with the
// large), so there are two sizes; a launch's parameters end at 32,764 bytes.
constexpr int32_t kInlineSmall = 3840, kInlineLarge = 31744;
template <int N>
struct alignas(16) InlineBlob {
    unsigned char b[N];
};
struct NoBlob {};  // descriptors in device memory
// An address in device memory, or a byte offset into the inline blob held in
// the pointer.
template <class T>
__host__ __device__ __forceinline__ const T *blob_at(const T *p, const NoBlob &) {
    return p;
}
template <class T, int N>
__host__ __device__ __forceinline__ const T *blob_at(const T *p, const InlineBlob<N> &blob) {
    return reinterpret_cast<const T *>(blob.b + reinterpret_cast<uintptr_t>(p));
}
// Calls f with the blob of n bytes at p (room for the large one), or with none.
template <class F>
auto with_blob(const InlineBlob<kInlineLarge> *p, size_t n, F &&f) {
    if (!p) return f(NoBlob{});
    if (n <= kInlineSmall) return f(*reinterpret_cast<const InlineBlob<kInlineSmall> *>(p));
    return f(*p);
}

// Element types of packed rows (pkv_dtype) and of pool storage.
enum class Elem : int32_t { f32 = 0, bf16 = 1, f16 = 2, fp8 = 3, q8 = 4 };

// Packed rows <-> pages.  Append: also uploads n_runs page-table runs (as the
// prep launch does).  Row r of K starts k_stride elements after row r - 1.
struct PagesArgs {
    const PageItem *items;
    int32_t n_items;
    void *K, *V;               // packed rows (the read writes them, the append reads them)
    int64_t k_stride, v_stride;
    Elem type;                 // of the packed rows
    const PtRun *runs = nullptr;
    const int32_t *vals = nullptr;
    int32_t n_runs = 0;
    int32_t *err = nullptr;
    // With an inline blob (of blob_n bytes), items, runs and vals are byte
    // offsets into it, which the kernels turn into addresses.
    const InlineBlob<kInlineLarge> *blob = nullptr;
    size_t blob_n = 0;
    // With blob_dst the append also stores the blob there, for launches behind it.
    void *blob_dst = nullptr;
    int32_t n_pre = 0;  // leading blocks that upload runs or the blob (set by the launch)
};

// The decode launch over an 8-bit pool.
struct Q8Args {
    const float *Q;
    float *out;
    const Q8Block *blocks;  // these two: or byte offsets into the inline blob
    const Q8Part *units;
    int32_t n_units, max_q;
    float *pm, *pl, *pacc;
    uint32_t *cnt;        // zero between launches: the joining unit clears its own
    int32_t n_heads, n_kv, hd, group, causal;
    float scale_log2;
    int32_t *err;
    const InlineBlob<kInlineLarge> *blob = nullptr;
    size_t blob_n = 0;
};

// Rotated copies of the new rows (RoPE on append over an 8-bit pool, whose
// append needs the rotated keys of a whole block before it can scale them).
struct RopeArgs {
    const float *Q, *K;
    float *Q_rot, *K_rot;
    const RowDesc *rows;       // past_len, n_q, q_row0
    int32_t n_rows, n_tok, q_dim, kv_dim, hd;
    double base;
    const InlineBlob<kInlineLarge> *blob = nullptr;  // rows: an offset into it
    size_t blob_n = 0;
};

// Packed prompt attention: sequence s holds tokens start[s] .. start[s + 1) of
// the packed rows.  The list travels in the launch's parameters (no upload, no
// scratch), so a launch takes at most kPackedSeqs sequences.
constexpr int32_t kPackedSeqs = 2000;
template <int N>
struct PackedSeqs {
    int32_t n;
    int32_t start[N];          // first token
    int32_t len[N];            // tokens (> 0), longest sequence first
    int32_t tile0[N + 1];      // query tiles of the sequences before s
};
struct PackedArgs {
    const void *Q, *K, *V;
    void *out;
    int64_t q_stride, k_stride, v_stride, o_stride;  // elements per token
    int32_t n_heads, n_kv, hd, causal;
    float scale_log2;
    int64_t n_tokens;          // rows of Q, K, V and out that belong to some sequence (from row 0)
    Elem type;
    int32_t *err;
    int32_t out32 = 0;         // out's rows and heads start on 32-byte boundaries (set by the launcher)
};

// Address of a key/value row in a contiguous history: base[pos][kv_head*hd ...]
struct ContigAddr {
    const float *k, *v;
    int32_t kv_dim;
};

struct AttnArgs {
    const float *Q;
    float *out;
    const RowDesc *rows;
    const UnitDesc *units;
    const MergeDesc *merges;  // merge items of the units with several splits
    int32_t n_units;
    float *pm, *pl, *pacc;  // partials: [n_part][n_heads], [n_part][n_heads], [n_part][n_heads][hd]
    int32_t n_heads, n_kv, hd, group, causal, split_keys;
    float scale_log2;       // scale * log2(e): scores are kept in base-2 units
    int32_t *err;
    // Fused append (paged decode, K_new != nullptr): a row's positions
    // past_len .. past_len + n_q - 1 are read from K_new / V_new row
    // q_row0 + (pos - past_len) instead of the pool, and the unit of query
    // n_q - 1 whose split holds them also stores them into the pool (block id
    // app[q_row0 + t].blk) and, when pt_write is set, enters each new block
    // (a position at a block boundary) into the device page table.
    const float *K_new = nullptr, *V_new = nullptr;
    const AppendDesc *app = nullptr;
    int32_t pt_write = 0;
};

// One tensor-core prefill tile: queries q0 .. q0 + 128/G - 1 of row `row`
// (clipped to n_q), key split `split` of size PrefillArgs::split_keys.
// part0 < 0: the tile's queries have one split and write out directly;
// otherwise query q0 + t's partial for split s is record
// part0 + t*stride + s, stride = n_split unless the tile sets it (a prefix
// pass leaves room for the decode splits that follow each query's prefix).
// The kernel takes tiles in pairs, one pair per CTA: tiles 2i and 2i + 1 share
// the row and the split; row < 0 marks an absent second tile.
struct PrefillTile {
    int32_t row, q0, split, part0;
    int32_t stride = 0;
};

struct PrefillArgs {
    const float *Q;
    float *out;
    const RowDesc *rows;
    const PrefillTile *tiles;
    int32_t n_tiles;  // even: two per CTA
    float *pm, *pl, *pacc;  // same partial layout as AttnArgs
    int32_t n_heads, n_kv, group, causal, split_keys;
    float scale_log2;
    int32_t *err;
    // Paged launches: the K/V operand images made by the split pass (or kept
    // from earlier calls); row r's key tile kt for kv head h is image
    // img_slot[img_tile0[r] + kt] * n_kv + h.
    const unsigned char *img = nullptr;
    const int32_t *img_tile0 = nullptr;
    const int32_t *img_slot = nullptr;
    // the images' piece-1 planes are left out (a bf16 or fp8 pool: every K/V
    // value times the tile's power of two is an f16 value), so the products
    // with them and their copies are skipped
    int32_t lo_zero = 0;
};

// The tensor-core kernel's operands for one (row, 64-key tile, kv head), as
// they sit in its shared memory: K0, K1 (K-major, 128-byte swizzle, two
// k-blocks of 64 dims x 64 keys) and V0^T, V1^T (one k-block of 64 keys x
// 128 dims), f16; then the tile's two exponents (int32 K, V).  Each f32
// value x of the tile is x * 2^e = x0 + x1, x0 = f16(x * 2^e), x1 = f16 of the
// exact rest, e the tile's exponent (its largest magnitude into [2^14, 2^15)).
constexpr int32_t kKeyTile = 64;  // keys per tensor-core tile (and per image)
constexpr uint32_t kImagePlane = 16 * 1024;
constexpr uint32_t kImageExpOff = 4 * kImagePlane;
constexpr uint32_t kImageBytes = 4 * kImagePlane + 128;  // a multiple of 128 bytes

// One image to make: key tile kt of row `row` (all kv heads), into image
// slot `slot` (images slot * n_kv + h).
struct SplitItem {
    int32_t row, kt, slot;
};

struct SplitArgs {
    const RowDesc *rows;
    const SplitItem *items;
    int32_t n_items, n_kv;
    unsigned char *img;
    int32_t *err;
};

// Floats of the maxima, and of the sums, of n_part partial records of every
// head: a multiple of four, so that the sums of V behind both start on a 16-byte
// boundary (the tensor-core kernels store them sixteen bytes at a time).
inline size_t record_floats(int64_t n_part, int32_t n_heads) {
    return (static_cast<size_t>(n_part) * static_cast<size_t>(n_heads) + 3) & ~static_cast<size_t>(3);
}

struct MergeArgs {
    const float *pm, *pl, *pacc;
    float *out;
    const RowDesc *rows;
    const MergeDesc *items;
    int32_t n_items, n_heads, hd;
};

// One launch before attention: upload page-table runs, append the new rows.
struct PrepArgs {
    int32_t *pt;
    int32_t max_blocks;
    const PtRun *runs;
    const int32_t *vals;
    int32_t n_runs;
    const AppendDesc *app;
    int32_t n_app;
    const float *K_new, *V_new;
    bool vec4;
    int32_t *err;
    // RoPE on append (rope_base > 0): K rows are rotated on their way into
    // the pool and Q rows into Q_rot, at position AppendDesc::pos; pairs
    // (i, i + hd/2) turn by pos * rope_base^(-2i/hd).
    double rope_base = 0.0;
    const float *Q = nullptr;
    float *Q_rot = nullptr;
    int32_t q_dim = 0, hd = 0;
};

// Set-up done once per device: a kernel's function attributes (its dynamic
// shared-memory opt-in) belong to the current device's context, so a process
// that drives several GPUs sets them on each.  Setting an attribute is
// idempotent, so threads that race here all set the same value.
struct PerDeviceOnce {
    std::atomic<uint64_t> done{0};  // bit d: device d is set up
    template <class F>
    cudaError_t run(F &&f) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t{1} << dev) : 0;
        if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
        e = f();
        if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Kernel launchers (pkv_kernels.cu).  Each enqueues exactly one kernel.
cudaError_t launch_prep(const PrepArgs &a, const PagedAddr &addr, cudaStream_t s);
cudaError_t launch_pt_apply(int32_t *pt_dev, int32_t max_blocks, const PtRun *runs, int32_t n_runs,
                            const int32_t *vals, cudaStream_t s);
// block_words: one block's K (or V) storage in 4-byte words
cudaError_t launch_copy_blocks(void *k, void *v, const CopyDesc *items, int32_t n_items,
                               int64_t block_words, int32_t n_blocks, int32_t *err,
                               cudaStream_t s);
cudaError_t launch_decode_paged(const AttnArgs &a, const PagedAddr &addr, cudaStream_t s);
cudaError_t launch_decode_contig(const AttnArgs &a, const ContigAddr &addr, cudaStream_t s);
// Decode over a bf16 or fp8 pool on the tensor cores (pkv_decode_mma.cu), for
// the shapes decode_mma_shape accepts; with AttnArgs::K_new it also takes the
// fused append (the new rows rounded to the pool element as the append does).
cudaError_t launch_decode_mma_paged(const AttnArgs &a, const PagedAddr &addr, cudaStream_t s);
__host__ __device__ constexpr bool decode_mma_shape(int head_dim, int group, bool bf16, bool fp8) {
    return head_dim == 128 &&
           ((fp8 && (group == 1 || group == 2 || group == 4 || group == 8)) ||
            (!fp8 && bf16 && (group == 1 || group == 2 || group == 4)));
}
cudaError_t launch_merge(const MergeArgs &a, cudaStream_t s);
// Tensor-core prefill (pkv_prefill.cu): head_dim 128, group 1, 2, 4 or 8; its
// K/V operands are the images in PrefillArgs::img (made by the split pass).
cudaError_t launch_prefill_paged(const PrefillArgs &a, const PagedAddr &addr, cudaStream_t s);
cudaError_t launch_prefill_contig(const PrefillArgs &a, const ContigAddr &addr, cudaStream_t s);
// The split pass of the tensor-core launches: one image per item and kv head,
// from the pool's rows or from a contiguous K/V pair.
cudaError_t launch_split_paged(const SplitArgs &a, const PagedAddr &addr, cudaStream_t s);
cudaError_t launch_split_contig(const SplitArgs &a, const ContigAddr &addr, cudaStream_t s);

// Packed rows into and out of the pages (pkv_pages.cu).
cudaError_t launch_append_pages(const PagesArgs &a, const PagedAddr &addr, cudaStream_t s);
cudaError_t launch_append_pages_q8(const PagesArgs &a, const Q8Addr &addr, cudaStream_t s);
cudaError_t launch_read_pages(const PagesArgs &a, const PagedAddr &addr, cudaStream_t s);
cudaError_t launch_read_pages_q8(const PagesArgs &a, const Q8Addr &addr, cudaStream_t s);
cudaError_t launch_rope_rows(const RopeArgs &a, cudaStream_t s);
// Attention over an 8-bit pool with block scales (pkv_q8.cu): split-K decode
// units of up to q8_query_block consecutive queries each, and the split pass of
// the tensor-core launches.  The decode launch may start while the launch
// before it on the stream (the append) still runs; q8_counters: the counters a
// block of units needs.
cudaError_t launch_decode_q8(const Q8Args &a, const Q8Addr &addr, cudaStream_t s);
int q8_counters(int head_dim, int group, int n_kv);
struct Q8Maps;
cudaError_t make_q8_maps(Q8Maps *m, const Q8Addr &addr, int n_layers, bool *usable);
cudaError_t launch_split_q8(const SplitArgs &a, const Q8Addr &addr, cudaStream_t s);
// Tensor-core attention over an 8-bit pool's images (pkv_prefill_q8.cu): the
// contract of launch_prefill_paged with one-piece images.
cudaError_t launch_prefill_q8(const PrefillArgs &a, int hd, cudaStream_t s);
int q8_query_block(int head_dim, int group);
// Packed prompt attention (pkv_packed.cu); sequences sorted longest first.
cudaError_t launch_packed(const PackedArgs &a, const int32_t *start, const int32_t *len, int32_t n_seqs,
                          cudaStream_t s);

// Rows with at least this many queries take the tensor-core prefill kernel
// (when head_dim is 128 and the group is 1, 2, 4 or 8); its key split is
// kPrefillSplitFactor times the decode split.  Both depend only on the row.
constexpr int kPrefillMinQueries = 32;
constexpr int kPrefillSplitFactor = 16;
__host__ __device__ constexpr bool prefill_shape(int head_dim, int group) {
    return head_dim == 128 && (group == 1 || group == 2 || group == 4 || group == 8);
}

// Likewise over an 8-bit pool: any group whose heads fit a tile several tokens
// deep, any head width of whole 16s.
__host__ __device__ constexpr bool prefill_shape_q8(int head_dim, int group) {
    return head_dim % 16 == 0 && head_dim <= 128 && group <= 64;
}

// Host-core helpers for entry points defined in other translation units
// (pkv_host.cpp).  build_contig_work: the split-K work list of one contiguous
// row, as pkv_attn_contiguous builds it (allow_tc false: no tensor-core
// tiles, every query to the split-K decode kernels).  launch_counted: enqueue fn(ctx) with
// the library's launch accounting and optional event timing.  report_error:
// record the calling thread's last error message and return code.
void build_contig_work(int32_t n_q, int32_t total_k, int32_t causal, int32_t split_keys,
                       int32_t head_dim, int32_t group, std::vector<UnitDesc> &units,
                       std::vector<PrefillTile> &tiles, std::vector<MergeDesc> &merges,
                       int64_t *n_part, bool allow_tc = true);
cudaError_t launch_counted(int kind, cudaStream_t s, cudaError_t (*fn)(void *), void *ctx);
int32_t current_split_keys();
int report_error(int code, const char *msg);
// The error word of pkv_attn_contiguous_noalloc on device `dev` (current): its
// device address, or nullptr when no call has set it up yet and `setup` is
// false; with `setup`, the first use on the device sets it up (*e reports a
// failure).  Defined in pkv_noalloc.cu.
int32_t *noalloc_error_word(int dev, bool setup, cudaError_t *e);

// Largest head_dim the decode kernels accept.
constexpr int kMaxHeadDim = 256;

}  // namespace pkv

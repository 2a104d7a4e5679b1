// pkv_pages.cu -- packed rows into and out of the pages of a pool.
//
//   append_pages   K / V rows (f32, bf16 or f16, packed with a row stride) into
//                  the pages of their sequences, converted to the pool's
//                  element; on an 8-bit pool with block scales also the scales
//   read_pages     the reverse: rows as the values they stand for
//   rope_rows      rotated copies of new Q and K rows (RoPE on append over an
//                  8-bit pool)
//
// One warp per (page item, group of columns, K or V); a group is one kv head
// on an 8-bit pool and kColGroup columns elsewhere.  Both directions are pure
// copies with a conversion, bound by HBM: every element is read and written
// once, in 16-byte accesses of the packed side where its alignment allows.
// Measured on an 8-bit pool (bf16 rows, 8 heads of 128): 130,000 rows appended
// in 142 us and read back in 137 (5.7 TB/s; 0.84 of the copy peak), 9,000 rows in 10 each.
//
// Quantisation (8-bit pool).  With m the largest magnitude of the page's new
// rows of a head, need(m) is the least e >= -126 with m <= 127 * 2^e; a page
// whose rows start here (offset 0) takes e = need(m), any other page the
// larger of need(m) and its present exponent, and rows it already holds are
// rounded to the new step.  Steps are powers of two, so every stored value is
// exact in f32 and a growth of the step by 2^k moves a kept element by at most
// half the new step; as steps at least double, those halves add up to less
// than one step however often the page grows.
#include "pkv_elem.h"
#include "pkv_internal.h"

#include <algorithm>
#include <type_traits>

namespace pkv {
namespace {

constexpr int kColGroup = 128;

using f16 = __half;

// eight consecutive packed elements as f32 (16-byte aligned)
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16 *p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const f16 *p, float (&x)[8]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
// The same in two steps, so that many chunks can be on their way before one is used.
template <class S>
struct Raw8 {
    uint4 a, b;  // b: f32 only
};
template <class S>
__device__ __forceinline__ Raw8<S> fetch8(const S *p) {
    Raw8<S> r;
    r.a = __ldg(reinterpret_cast<const uint4 *>(p));
    if constexpr (sizeof(S) == 4) r.b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    return r;
}
__device__ __forceinline__ void widen8(const Raw8<float> &r, float (&x)[8]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void widen8(const Raw8<bf16> &r, float (&x)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen8(const Raw8<f16> &r, float (&x)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
// The largest magnitude so far, as bits: of f32 a word, of 16-bit types two
// halves (a magnitude's bits are ordered as the magnitude is, infinities and
// NaN above every finite one); max_bits: of everything, as the bits of an f32.
__device__ __forceinline__ uint32_t max_raw(uint32_t m, const Raw8<float> &r) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
}
template <class S>
__device__ __forceinline__ uint32_t max_raw(uint32_t m, const Raw8<S> &r) {
    m = __vmaxu2(m, r.a.x & 0x7fff7fffu);
    m = __vmaxu2(m, r.a.y & 0x7fff7fffu);
    m = __vmaxu2(m, r.a.z & 0x7fff7fffu);
    return __vmaxu2(m, r.a.w & 0x7fff7fffu);
}
template <class S>
__device__ __forceinline__ uint32_t max_bits(uint32_t m) {
    if constexpr (sizeof(S) == 4) return m;
    const uint32_t h = max(m & 0xffffu, m >> 16);
    if constexpr (std::is_same<S, bf16>::value) return h << 16;
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
}
__device__ __forceinline__ float load1(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load1(const bf16 *p) { return to_f32(*p); }
__device__ __forceinline__ float load1(const f16 *p) { return __half2float(*p); }

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// eight consecutive elements, rounded once to nearest even
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                                               pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(f16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]),
                                               pack_f16(x[6], x[7]));
}
__device__ __forceinline__ void store8(fp8 *p, const float (&x)[8]) {
    store4(p, make_float4(x[0], x[1], x[2], x[3]));
    store4(p + 4, make_float4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ void put1(float *p, float x) { *p = x; }
__device__ __forceinline__ void put1(bf16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put1(f16 *p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void put1(fp8 *p, float x) { store1(p, x); }

// eight pool elements as f32
__device__ __forceinline__ void pool8(const float *p, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void pool8(const bf16 *p, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void pool8(const fp8 *p, float (&x)[8]) {
    const float4 a = ldg4(p), b = ldg4(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ float pool1(const float *p) { return ldg1(p); }
__device__ __forceinline__ float pool1(const bf16 *p) { return ldg1(p); }
__device__ __forceinline__ float pool1(const fp8 *p) { return ldg1(p); }

__device__ __forceinline__ float pow2f(int e) {  // 2^e, e in [-126, 127]
    return __int_as_float((e + 127) << 23);
}

// ---------------------------------------------------------- quantisation ----

// The least e >= -126 with m <= 127 * 2^e, from the bits of a finite m >= 0:
// m = 1.f * 2^k and 127 * 2^e = 1.984375 * 2^(e+6), so e = k - 6, or k - 5
// where 1.f > 1.984375 (fraction bits above 0x7e0000).
__device__ __forceinline__ int need_exp(uint32_t m_bits) {
    const int k = static_cast<int>(m_bits >> 23) - 127;
    return max(-126, k - 6 + ((m_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0));
}
constexpr uint32_t kInfBits = 0x7f800000u;
// The exponent of a stored scale (a power of two; 0 reads as the least one).
__device__ __forceinline__ int scale_exp(float s) {
    return max(-126, static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127);
}
// the element of the value x at step 1 / inv: |x * inv| <= 127, the product exact
__device__ __forceinline__ uint32_t q8_elem(float x, float inv) {
    return static_cast<uint32_t>(__float2int_rn(x * inv) + 128) & 255u;
}
// Four elements in a word.  Adding 1.5 * 2^23 leaves the sum's integer part in
// the low mantissa bits, rounded to nearest even as the sum is (the 128 that
// comes along is even, so ties fall as they would without it): one FFMA a
// value where a conversion instruction would run at a quarter of its rate.
__device__ __forceinline__ uint32_t q8_word(float a, float b, float c, float d, float inv) {
    constexpr float kMagic = 12582912.f + 128.f;
    const uint32_t ta = __float_as_uint(fmaf(a, inv, kMagic)), tb = __float_as_uint(fmaf(b, inv, kMagic));
    const uint32_t tc = __float_as_uint(fmaf(c, inv, kMagic)), td = __float_as_uint(fmaf(d, inv, kMagic));
    return __byte_perm(__byte_perm(ta, tb, 0x0040), __byte_perm(tc, td, 0x0040), 0x5410);
}
// Element j of a word as u - 128, exact: 2^23 + u is the float of bits 0x4b000000
// | u (conversion instructions run at a quarter of the rate).
__device__ __forceinline__ float q8_value(uint32_t w, int j) {
    return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | j)) - (8388608.f + 128.f);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// ----------------------------------------------------------------- append ----

// A lane's chunks of eight, 32 apart: row and column without a division each.
struct ChunkWalk {
    int row, c, dr, dc, cpr;  // c in chunks
    __device__ __forceinline__ ChunkWalk(int lane, int cpr_) : cpr(cpr_) {
        dr = 32 / cpr;
        dc = 32 - dr * cpr;
        row = lane / cpr;
        c = lane - row * cpr;
    }
    __device__ __forceinline__ void next() {
        row += dr;
        c += dc;
        if (c >= cpr) c -= cpr, ++row;
    }
};

struct RowSpan {  // what one warp works on
    PageItem it;
    int32_t c0, cw;  // columns c0 .. c0 + cw - 1
    bool is_v, ok;
};

__device__ __forceinline__ RowSpan row_span(const PagesArgs &p, const PagedAddr &a, int group, int n_groups, int w) {
    RowSpan r;
    const int per_item = 2 * n_groups;
    r.it = p.items[w / per_item];
    int x = w % per_item;
    r.is_v = x >= n_groups;
    x -= r.is_v ? n_groups : 0;
    r.c0 = x * group;
    r.cw = min(group, a.kv_dim - r.c0);
    r.ok = static_cast<unsigned>(r.it.blk) < static_cast<unsigned>(a.n_blocks) && r.it.off >= 0 && r.it.n > 0 &&
           r.it.off + r.it.n <= a.bs;
    return r;
}

// Descriptors in device memory (NoBlob) or in the launch's parameters.
template <class B>
__device__ __forceinline__ void place(PagesArgs &p, const B &blob) {
    p.items = blob_at(p.items, blob);
    p.runs = blob_at(p.runs, blob);
    p.vals = blob_at(p.vals, blob);
}
// A launch that may start while this one runs waits for its end before it
// reads what this one writes; it may set itself up from now on.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

__device__ __forceinline__ bool upload_runs(const PagesArgs &p, const PagedAddr &a) {
    if (static_cast<int>(blockIdx.x) >= p.n_runs) return false;
    const PtRun r = p.runs[blockIdx.x];
    int32_t *dst = a.pt + static_cast<size_t>(r.slot) * a.max_blocks + r.start;
    for (int i = threadIdx.x; i < r.count; i += blockDim.x) dst[i] = p.vals[r.voff + i];
    return true;
}
template <class B>
__device__ __forceinline__ bool before_items(const PagesArgs &p, const PagedAddr &a, const B &blob) {
    if constexpr (!std::is_same<B, NoBlob>::value) {
        if (p.n_pre > p.n_runs && static_cast<int>(blockIdx.x) == p.n_runs) {
            const uint4 *src = reinterpret_cast<const uint4 *>(blob.b);
            for (int i = threadIdx.x; i < static_cast<int>((p.blob_n + 15) / 16); i += blockDim.x)
                static_cast<uint4 *>(p.blob_dst)[i] = src[i];
            return true;
        }
    }
    return upload_runs(p, a);
}

// The step of a page's head after rows of largest magnitude m (f32 bits) come
// to offset off: stores the scale, brings the rows before them into a step that
// grew, and returns 1 / step -- or 0 where there is none: a value that is not
// finite has no element, so the scale becomes NaN, which every read of the
// block and head returns until its first row is written again.
__device__ __forceinline__ float new_step(uint32_t m, float old, int off, int cw, float *scale, uint8_t *page,
                                          int kv_dim, int lane) {
    if (m >= kInfBits || abs_bits(old) >= kInfBits) {
        if (lane == 0) *scale = __uint_as_float(0x7fc00000u);
        return 0.f;
    }
    const int e_old = scale_exp(old), e = off > 0 ? max(e_old, need_exp(m)) : need_exp(m);
    if (lane == 0) *scale = pow2f(e);
    if (off > 0 && e > e_old) {
        const float f = pow2f(max(-126, e_old - e));
        for (int i = lane; i < off * cw; i += 32) {
            const int row = i / cw, c = i - row * cw;
            uint8_t *u = page + static_cast<size_t>(row) * kv_dim + c;
            *u = static_cast<uint8_t>(q8_elem(static_cast<float>(static_cast<int>(*u) - 128), f));
        }
    }
    return pow2f(-e);
}

template <class B, class S, class E, bool kVec>
__global__ void __launch_bounds__(256) append_pages_kernel(PagesArgs p, PagedAddr a, int n_groups, const __grid_constant__ B blob) {
    place(p, blob);
    let_next_start();
    if (upload_runs(p, a)) return;
    const int w = (static_cast<int>(blockIdx.x) - p.n_runs) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= p.n_items * 2 * n_groups) return;
    const RowSpan r = row_span(p, a, kColGroup, n_groups, w);
    if (!r.ok) {
        if (lane == 0 && p.err) atomicOr(p.err, 1);
        return;
    }
    const int64_t stride = r.is_v ? p.v_stride : p.k_stride;
    const S *src = static_cast<const S *>(r.is_v ? p.V : p.K) + static_cast<int64_t>(r.it.row0) * stride + r.c0;
    E *dst = static_cast<E *>(r.is_v ? a.v : a.k) + static_cast<size_t>(r.it.blk) * a.block_stride + a.layer_off +
             static_cast<size_t>(r.it.off) * a.kv_dim + r.c0;
    const float inv = 1.f / a.kv_scale;  // a power of two (1 except on fp8 pools)
    if constexpr (kVec) {
        const int cpr = r.cw >> 3;
        ChunkWalk w8(lane, cpr);
#pragma unroll 4
        for (int i = lane; i < r.it.n * cpr; i += 32, w8.next()) {
            const int row = w8.row, c = w8.c * 8;
            float x[8];
            load8(src + row * stride + c, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= inv;
            store8(dst + static_cast<size_t>(row) * a.kv_dim + c, x);
        }
    } else {
        for (int i = lane; i < r.it.n * r.cw; i += 32) {
            const int row = i / r.cw, c = i - row * r.cw;
            put1(dst + static_cast<size_t>(row) * a.kv_dim + c, load1(src + row * stride + c) * inv);
        }
    }
}

template <class B, class S, bool kVec>
__global__ void __launch_bounds__(256) append_pages_q8_kernel(PagesArgs p, Q8Addr q, const __grid_constant__ B blob) {
    place(p, blob);
    let_next_start();
    const PagedAddr &a = q.a;
    if (before_items(p, a, blob)) return;
    const int w = (static_cast<int>(blockIdx.x) - p.n_pre) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= p.n_items * 2 * q.n_kv) return;
    const RowSpan r = row_span(p, a, q.hd, q.n_kv, w);
    if (!r.ok) {
        if (lane == 0 && p.err) atomicOr(p.err, 1);
        return;
    }
    const int64_t stride = r.is_v ? p.v_stride : p.k_stride;
    const S *src = static_cast<const S *>(r.is_v ? p.V : p.K) + static_cast<int64_t>(r.it.row0) * stride + r.c0;
    uint8_t *page = static_cast<uint8_t *>(r.is_v ? a.v : a.k) + static_cast<size_t>(r.it.blk) * a.block_stride +
                    a.layer_off + r.c0;
    uint8_t *dst = page + static_cast<size_t>(r.it.off) * a.kv_dim;
    float *scale = (r.is_v ? q.vs : q.ks) + static_cast<int64_t>(r.it.blk) * q.scale_stride + r.c0 / q.hd;
    const float old = r.it.off > 0 ? *scale : 0.f;

    // the rows are read twice, for their largest magnitude and to store them
    const int cpr = kVec ? r.cw >> 3 : 1, n_ch = r.it.n * cpr;
    uint32_t m = 0;
    if constexpr (kVec) {
        ChunkWalk w8(lane, cpr);
#pragma unroll 4
        for (int i = lane; i < n_ch; i += 32, w8.next()) m = max_raw(m, fetch8(src + w8.row * stride + w8.c * 8));
        m = max_bits<S>(m);
    } else {
        for (int i = lane; i < r.it.n * r.cw; i += 32) {
            const int row = i / r.cw, c = i - row * r.cw;
            m = max(m, abs_bits(load1(src + row * stride + c)));
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const float inv = new_step(m, old, r.it.off, r.cw, scale, page, a.kv_dim, lane);
    const bool bad = inv == 0.f;
    if constexpr (kVec) {
        ChunkWalk w8(lane, cpr);
#pragma unroll 4
        for (int i = lane; i < n_ch; i += 32, w8.next()) {
            float x[8];
            widen8(fetch8(src + w8.row * stride + w8.c * 8), x);
            uint2 u = make_uint2(q8_word(x[0], x[1], x[2], x[3], inv), q8_word(x[4], x[5], x[6], x[7], inv));
            if (bad) u = make_uint2(0x80808080u, 0x80808080u);
            *reinterpret_cast<uint2 *>(dst + static_cast<size_t>(w8.row) * a.kv_dim + w8.c * 8) = u;
        }
    } else {
        for (int i = lane; i < r.it.n * r.cw; i += 32) {
            const int row = i / r.cw, c = i - row * r.cw;
            dst[static_cast<size_t>(row) * a.kv_dim + c] =
                bad ? 128 : static_cast<uint8_t>(q8_elem(load1(src + row * stride + c), inv));
        }
    }
}

// The same where a head's chunks of eight divide a warp and a page's fit in
// kHold a lane (16 rows of 128): a warp keeps its (head, K or V) and walks the
// items with a stride, holding one item's rows in registers while the next
// one's are on their way, so that every warp has a page in flight all the time.
// (With one item a warp, loads in flight only part of its life, an append of
// 130,000 rows took 183 us; held in registers without the walk 188-218.)
template <class B, class S, int kHold, bool kAhead>
__global__ void __launch_bounds__(256, 2) append_stream_q8_kernel(PagesArgs p, Q8Addr q, int n_warps, const __grid_constant__ B blob) {
    place(p, blob);
    let_next_start();
    const PagedAddr &a = q.a;
    if (before_items(p, a, blob)) return;
    const int w = (static_cast<int>(blockIdx.x) - p.n_pre) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int per_item = 2 * q.n_kv, step = n_warps / per_item;  // n_warps: a multiple of per_item
    int it = w / per_item;
    const int sub = w - it * per_item;
    if (it >= p.n_items) return;
    const bool is_v = sub >= q.n_kv;
    const int head = is_v ? sub - q.n_kv : sub;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int cpr = q.hd >> 3, dr = 32 / cpr, row0 = lane / cpr, c0 = (lane - row0 * cpr) * 8;
    const S *const src = static_cast<const S *>(is_v ? p.V : p.K) + head * q.hd + row0 * stride + c0;
    uint8_t *const pool = static_cast<uint8_t *>(is_v ? a.v : a.k) + a.layer_off + head * q.hd;
    float *const scales = (is_v ? q.vs : q.ks) + head;
    auto item = [&](int i) {
        const int4 x = *reinterpret_cast<const int4 *>(p.items + i);
        PageItem t{x.x, x.y, x.z, x.w};
        if (static_cast<unsigned>(t.blk) >= static_cast<unsigned>(a.n_blocks) || t.off < 0 || t.n <= 0 ||
            t.off + t.n > a.bs) {
            if (lane == 0 && p.err) atomicOr(p.err, 1);
            t.n = 0;
        }
        return t;
    };
    auto fetch = [&](const PageItem &t, Raw8<S> (&h)[kHold]) {
        const S *at = src + static_cast<int64_t>(t.row0) * stride;
#pragma unroll
        for (int k = 0; k < kHold; ++k)
            if (row0 + k * dr < t.n) h[k] = fetch8(at + k * dr * stride);
    };
    auto put = [&](const PageItem &t, const Raw8<S> (&h)[kHold]) {
        if (t.n == 0) return;
        float *scale = scales + static_cast<int64_t>(t.blk) * q.scale_stride;
        uint8_t *page = pool + static_cast<size_t>(t.blk) * a.block_stride;
        const float old = t.off > 0 ? *scale : 0.f;
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kHold; ++k)
            if (row0 + k * dr < t.n) m = max_raw(m, h[k]);
        m = __reduce_max_sync(0xffffffffu, max_bits<S>(m));
        const float inv = new_step(m, old, t.off, q.hd, scale, page, a.kv_dim, lane);
        uint8_t *dst = page + static_cast<size_t>(t.off + row0) * a.kv_dim + c0;
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
            if (row0 + k * dr >= t.n) continue;
            float x[8];
            widen8(h[k], x);
            uint2 u = make_uint2(q8_word(x[0], x[1], x[2], x[3], inv), q8_word(x[4], x[5], x[6], x[7], inv));
            if (inv == 0.f) u = make_uint2(0x80808080u, 0x80808080u);
            *reinterpret_cast<uint2 *>(dst + static_cast<size_t>(k * dr) * a.kv_dim) = u;
        }
    };
    Raw8<S> h0[kHold];
    if constexpr (!kAhead) {
        for (; it < p.n_items; it += step) {
            const PageItem t = item(it);
            fetch(t, h0);
            put(t, h0);
        }
        return;
    } else {
        Raw8<S> h1[kHold];
        PageItem t0 = item(it), t1;
        fetch(t0, h0);
        while (true) {  // two items a turn, each buffer's registers its own
            const bool more1 = it + step < p.n_items;
            if (more1) {
                t1 = item(it + step);
                fetch(t1, h1);
            }
            put(t0, h0);
            if (!more1) return;
            it += 2 * step;
            const bool more0 = it < p.n_items;
            if (more0) {
                t0 = item(it);
                fetch(t0, h0);
            }
            put(t1, h1);
            if (!more0) return;
        }
    }
}

// ------------------------------------------------------------------- read ----

template <class B, class D, class E, bool kVec>
__global__ void __launch_bounds__(256) read_pages_kernel(PagesArgs p, PagedAddr a, int n_groups, const __grid_constant__ B blob) {
    place(p, blob);
    const int w = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= p.n_items * 2 * n_groups) return;
    const RowSpan r = row_span(p, a, kColGroup, n_groups, w);
    if (!r.ok) {
        if (lane == 0 && p.err) atomicOr(p.err, 1);
        return;
    }
    const int64_t stride = r.is_v ? p.v_stride : p.k_stride;
    D *dst = static_cast<D *>(r.is_v ? p.V : p.K) + static_cast<int64_t>(r.it.row0) * stride + r.c0;
    const E *src = static_cast<const E *>(r.is_v ? a.v : a.k) + static_cast<size_t>(r.it.blk) * a.block_stride +
                   a.layer_off + static_cast<size_t>(r.it.off) * a.kv_dim + r.c0;
    if constexpr (kVec) {
        const int cpr = r.cw >> 3;
        ChunkWalk w8(lane, cpr);
#pragma unroll 4
        for (int i = lane; i < r.it.n * cpr; i += 32, w8.next()) {
            const int row = w8.row, c = w8.c * 8;
            float x[8];
            pool8(src + static_cast<size_t>(row) * a.kv_dim + c, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= a.kv_scale;
            store8(dst + row * stride + c, x);
        }
    } else {
        for (int i = lane; i < r.it.n * r.cw; i += 32) {
            const int row = i / r.cw, c = i - row * r.cw;
            put1(dst + row * stride + c, pool1(src + static_cast<size_t>(row) * a.kv_dim + c) * a.kv_scale);
        }
    }
}

template <class B, class D, bool kVec>
__global__ void __launch_bounds__(256) read_pages_q8_kernel(PagesArgs p, Q8Addr q, const __grid_constant__ B blob) {
    place(p, blob);
    const PagedAddr &a = q.a;
    const int w = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= p.n_items * 2 * q.n_kv) return;
    const RowSpan r = row_span(p, a, q.hd, q.n_kv, w);
    if (!r.ok) {
        if (lane == 0 && p.err) atomicOr(p.err, 1);
        return;
    }
    const int64_t stride = r.is_v ? p.v_stride : p.k_stride;
    D *dst = static_cast<D *>(r.is_v ? p.V : p.K) + static_cast<int64_t>(r.it.row0) * stride + r.c0;
    const uint8_t *src = static_cast<const uint8_t *>(r.is_v ? a.v : a.k) +
                         static_cast<size_t>(r.it.blk) * a.block_stride + a.layer_off +
                         static_cast<size_t>(r.it.off) * a.kv_dim + r.c0;
    const float sc = __ldg((r.is_v ? q.vs : q.ks) + static_cast<int64_t>(r.it.blk) * q.scale_stride + r.c0 / q.hd);
    if constexpr (kVec) {
        constexpr int kFly = 8;  // chunks on the way at once
        const int cpr = r.cw >> 3, n_ch = r.it.n * cpr;
        ChunkWalk wl(lane, cpr), ws = wl;
        for (int i0 = lane; i0 < n_ch; i0 += 32 * kFly) {
            uint2 u[kFly];
#pragma unroll
            for (int k = 0; k < kFly; ++k, wl.next())
                if (i0 + 32 * k < n_ch)
                    u[k] = __ldg(reinterpret_cast<const uint2 *>(src + static_cast<size_t>(wl.row) * a.kv_dim + wl.c * 8));
#pragma unroll
            for (int k = 0; k < kFly; ++k, ws.next()) {
                if (i0 + 32 * k >= n_ch) continue;
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = q8_value(j < 4 ? u[k].x : u[k].y, j & 3) * sc;
                store8(dst + ws.row * stride + ws.c * 8, x);
            }
        }
    } else {
        for (int i = lane; i < r.it.n * r.cw; i += 32) {
            const int row = i / r.cw, c = i - row * r.cw;
            put1(dst + row * stride + c,
                 static_cast<float>(static_cast<int>(src[static_cast<size_t>(row) * a.kv_dim + c]) - 128) * sc);
        }
    }
}

// ------------------------------------------------------------------- rope ----

// The pairs (i, i + hd/2) of every query and key head of a token turned by pos *
// base^(-2i/hd), with the arithmetic of the append kernel's rotation (angle,
// cosine and sine in double precision, the products and sums each rounded to
// f32).  A CTA takes tokens blockIdx.x, + gridDim.x, ...: thread i < hd/2 keeps
// its frequency and makes the token's i'th cosine and sine, then all turn the
// heads' pairs.  Bound by the double-precision cosines where tokens are many
// (hd/2 a token), by latency where they are few.
constexpr int kRopeThreads = 256;
template <class B>
__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(RopeArgs p, const __grid_constant__ B blob) {
    __shared__ float2 turn[kMaxHeadDim / 2];
    const RowDesc *rows = blob_at(p.rows, blob);
    const int half = p.hd >> 1, tid = threadIdx.x;
    const int n_pairs = (p.q_dim + p.kv_dim) / p.hd * half, nq = p.q_dim / p.hd * half;
    const double freq = tid < half ? exp(-2.0 * tid / p.hd * log(p.base)) : 0.0;
    for (int t = blockIdx.x; t < p.n_tok; t += gridDim.x) {
        int lo = 0, hi = p.n_rows - 1;  // the batch row of token t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (rows[mid].q_row0 <= t) lo = mid;
            else hi = mid - 1;
        }
        const int pos = rows[lo].past_len + (t - rows[lo].q_row0);
        __syncthreads();  // the token before this one is done with its turns
        if (tid < half) {
            double sd, cd;
            sincos(static_cast<double>(pos) * freq, &sd, &cd);
            turn[tid] = make_float2(static_cast<float>(cd), static_cast<float>(sd));
        }
        __syncthreads();
        const float *Q = p.Q + static_cast<size_t>(t) * p.q_dim, *K = p.K + static_cast<size_t>(t) * p.kv_dim;
        float *Qr = p.Q_rot + static_cast<size_t>(t) * p.q_dim, *Kr = p.K_rot + static_cast<size_t>(t) * p.kv_dim;
#pragma unroll 4
        for (int x = tid; x < n_pairs; x += kRopeThreads) {
            const bool is_k = x >= nq;
            const int y = is_k ? x - nq : x, h = y / half, i = y - h * half, o = h * p.hd + i;
            const float *src = is_k ? K : Q;
            float *dst = is_k ? Kr : Qr;
            const float x0 = __ldg(src + o), x1 = __ldg(src + o + half);
            const float2 r = turn[i];
            dst[o] = __fsub_rn(__fmul_rn(x0, r.x), __fmul_rn(x1, r.y));
            dst[o + half] = __fadd_rn(__fmul_rn(x0, r.y), __fmul_rn(x1, r.x));
        }
    }
}

// ---------------------------------------------------------------- dispatch ----

size_t type_bytes(Elem t) { return t == Elem::f32 ? 4 : t == Elem::bf16 || t == Elem::f16 ? 2 : 1; }

// 16-byte accesses of eight packed elements, and of the pool's: the packed
// rows' bases and strides and the columns of a group all on such boundaries.
bool vec_ok(const PagesArgs &p, const PagedAddr &a, int group) {
    const size_t e = type_bytes(p.type);
    auto al = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    return al(p.K) && al(p.V) && (p.k_stride * e) % 16 == 0 && (p.v_stride * e) % 16 == 0 && a.kv_dim % 8 == 0 &&
           group % 8 == 0 && al(a.k) && al(a.v);
}

bool grid_of(long long warps, int n_runs, unsigned *grid) {
    const long long b = (warps + 7) / 8 + n_runs;
    if (b <= 0 || b > 0x7fffffffLL) return false;
    *grid = static_cast<unsigned>(b);
    return true;
}

template <class F>
cudaError_t launch_with(const PagesArgs &p, F &&f) {
    with_blob(p.blob, p.blob_n, f);
    return cudaGetLastError();
}

template <class S, class E>
cudaError_t append_as(const PagesArgs &p, const PagedAddr &a, cudaStream_t s) {
    const int n_groups = (a.kv_dim + kColGroup - 1) / kColGroup;
    unsigned grid;
    if (!grid_of(2LL * p.n_items * n_groups, p.n_runs, &grid)) return cudaErrorInvalidConfiguration;
    return launch_with(p, [&](const auto &b) {
        using B = std::decay_t<decltype(b)>;
        if (vec_ok(p, a, kColGroup)) append_pages_kernel<B, S, E, true><<<grid, 256, 0, s>>>(p, a, n_groups, b);
        else append_pages_kernel<B, S, E, false><<<grid, 256, 0, s>>>(p, a, n_groups, b);
    });
}
template <class S>
cudaError_t append_from(const PagesArgs &p, const PagedAddr &a, cudaStream_t s) {
    if (a.fp8) return append_as<S, fp8>(p, a, s);
    if (a.bf16) return append_as<S, bf16>(p, a, s);
    return append_as<S, float>(p, a, s);
}
template <class S>
cudaError_t append_q8_from(const PagesArgs &args, const Q8Addr &q, cudaStream_t s) {
    PagesArgs p = args;
    p.n_pre = p.n_runs + (p.blob && p.blob_dst ? 1 : 0);
    unsigned grid;
    constexpr int kHold = 8;
    const int cpr = q.hd / 8;
    // (fewer than four items a walking warp: one item a warp, more warps a SM)
    if (2LL * p.n_items * q.n_kv >= 4LL * 2 * 152 * 8 && vec_ok(p, q.a, q.hd) && cpr <= 32 && 32 % cpr == 0 && q.a.bs * cpr <= 32 * kHold) {
        // a whole number of items (and blocks) per round of warps, two blocks a SM
        const long long warps = 2LL * p.n_items * q.n_kv, round = 16LL * q.n_kv;  // 8 items, 2 n_kv blocks
        const long long want = std::min<long long>((warps + round - 1) / round, std::max<long long>(1, 2LL * 152 * 8 / round));
        const int n_warps = static_cast<int>(want * round);
        if (!grid_of(n_warps, p.n_pre, &grid)) return cudaErrorInvalidConfiguration;
        return launch_with(p, [&](const auto &b) {
            append_stream_q8_kernel<std::decay_t<decltype(b)>, S, kHold, sizeof(S) == 2>
                <<<grid, 256, 0, s>>>(p, q, n_warps, b);
        });
    }
    if (!grid_of(2LL * p.n_items * q.n_kv, p.n_pre, &grid)) return cudaErrorInvalidConfiguration;
    return launch_with(p, [&](const auto &b) {
        using B = std::decay_t<decltype(b)>;
        if (vec_ok(p, q.a, q.hd)) append_pages_q8_kernel<B, S, true><<<grid, 256, 0, s>>>(p, q, b);
        else append_pages_q8_kernel<B, S, false><<<grid, 256, 0, s>>>(p, q, b);
    });
}
template <class D, class E>
cudaError_t read_as(const PagesArgs &p, const PagedAddr &a, cudaStream_t s) {
    const int n_groups = (a.kv_dim + kColGroup - 1) / kColGroup;
    unsigned grid;
    if (!grid_of(2LL * p.n_items * n_groups, 0, &grid)) return cudaErrorInvalidConfiguration;
    return launch_with(p, [&](const auto &b) {
        using B = std::decay_t<decltype(b)>;
        if (vec_ok(p, a, kColGroup)) read_pages_kernel<B, D, E, true><<<grid, 256, 0, s>>>(p, a, n_groups, b);
        else read_pages_kernel<B, D, E, false><<<grid, 256, 0, s>>>(p, a, n_groups, b);
    });
}
template <class D>
cudaError_t read_to(const PagesArgs &p, const PagedAddr &a, cudaStream_t s) {
    if (a.fp8) return read_as<D, fp8>(p, a, s);
    if (a.bf16) return read_as<D, bf16>(p, a, s);
    return read_as<D, float>(p, a, s);
}
template <class D>
cudaError_t read_q8_to(const PagesArgs &p, const Q8Addr &q, cudaStream_t s) {
    unsigned grid;
    if (!grid_of(2LL * p.n_items * q.n_kv, 0, &grid)) return cudaErrorInvalidConfiguration;
    return launch_with(p, [&](const auto &b) {
        using B = std::decay_t<decltype(b)>;
        if (vec_ok(p, q.a, q.hd)) read_pages_q8_kernel<B, D, true><<<grid, 256, 0, s>>>(p, q, b);
        else read_pages_q8_kernel<B, D, false><<<grid, 256, 0, s>>>(p, q, b);
    });
}

}  // namespace

cudaError_t launch_append_pages(const PagesArgs &p, const PagedAddr &a, cudaStream_t s) {
    switch (p.type) {
        case Elem::f32: return append_from<float>(p, a, s);
        case Elem::bf16: return append_from<bf16>(p, a, s);
        case Elem::f16: return append_from<f16>(p, a, s);
        default: return cudaErrorInvalidValue;
    }
}
cudaError_t launch_append_pages_q8(const PagesArgs &p, const Q8Addr &q, cudaStream_t s) {
    switch (p.type) {
        case Elem::f32: return append_q8_from<float>(p, q, s);
        case Elem::bf16: return append_q8_from<bf16>(p, q, s);
        case Elem::f16: return append_q8_from<f16>(p, q, s);
        default: return cudaErrorInvalidValue;
    }
}
cudaError_t launch_read_pages(const PagesArgs &p, const PagedAddr &a, cudaStream_t s) {
    switch (p.type) {
        case Elem::f32: return read_to<float>(p, a, s);
        case Elem::bf16: return read_to<bf16>(p, a, s);
        case Elem::f16: return read_to<f16>(p, a, s);
        default: return cudaErrorInvalidValue;
    }
}
cudaError_t launch_read_pages_q8(const PagesArgs &p, const Q8Addr &q, cudaStream_t s) {
    switch (p.type) {
        case Elem::f32: return read_q8_to<float>(p, q, s);
        case Elem::bf16: return read_q8_to<bf16>(p, q, s);
        case Elem::f16: return read_q8_to<f16>(p, q, s);
        default: return cudaErrorInvalidValue;
    }
}
cudaError_t launch_rope_rows(const RopeArgs &p, cudaStream_t s) {
    if (p.n_tok <= 0 || p.hd > kMaxHeadDim) return cudaErrorInvalidValue;
    // eight blocks a SM, so that many tokens share a block's frequencies
    const unsigned grid = static_cast<unsigned>(std::min(p.n_tok, 8 * 152));
    with_blob(p.blob, p.blob_n, [&](const auto &b) { rope_rows_kernel<<<grid, kRopeThreads, 0, s>>>(p, b); });
    return cudaGetLastError();
}

}  // namespace pkv

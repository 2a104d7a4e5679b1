// pkv_prefill_q8.cu -- tensor-core attention of rows with many queries (and of
// shared prefixes) over an 8-bit pool.
//
// The contract, the operand images and the arithmetic are those of the prefill
// kernel on one-piece images: f32 queries and probabilities as two f16 pieces
// (x times a power of two = x0 + x1, 22 bits), K and V values exact in f16 times
// their tile's power of two, so a product is x0*y + x1*y; the largest-score
// reference moves, and the accumulator is rescaled, only where a tile's maximum
// passes it by 2^8; probabilities times 2^(C - c), c the exponent of their V
// tile and C one of the chain that only falls.
//
// A key tile is two images (128 keys), which keeps every MMA at N = 128:
//
//   S_c [128 x 128] = (Q0_c + Q1_c) K_j^T    16 MMAs, A and B from shared memory
//   D_c [128 x 128] += (P0_c + P1_c) V_j     16 MMAs, A from TMEM over S_c
//
// (at 64 keys the QK MMAs run at two thirds of their rate).  One CTA = two tiles
// of 128 query rows that share every K/V tile, one softmax chain each; row m of
// a tile is token m / G, head m % G, TMEM lane m, thread m of the chain's four
// warps.  Each chain has one S buffer and runs QK(j), softmax(j), PV(j), QK(j+1)
// in turn, its products issued by its own warp (8 and 10); the chains alternate
// by turns, so that one's softmax runs under the other's 2052 clocks of MMAs.
// Warp 9 copies the images (K_0, V_0, K_1, ... through three slots of 32 KiB).
// Shared memory: Q pieces 128 KiB, slots 96 KiB.  TMEM: D_c at 128c, S_c / P_c
// at 256 + 128c (P0 in its first 64 columns, P1 in the others).
//
// A CTA with one tile gives its chain both S buffers and the other's query
// pieces as two further slots, so that QK(j + 1) runs under softmax(j): 2,900
// clocks a key tile instead of 4,600.  The chain's arithmetic is the same.
//
// Measured (8 rows of 512 queries behind 2,048 keys, 32 heads over 8, 568 CTAs
// of 18.5 key tiles on average): 244 us, 1.25 PFLOP/s of f16 products.  With two
// tiles a key tile takes 5,200 clocks where its MMAs alone take 4,104: what is
// left is a chain's wait for its own softmax (2,100 to 2,400 clocks from S to
// P) and for the slots.  A CTA spends 12,000 clocks on its start, 5,000 on its
// output and 7,000 pass before the next one runs; the rest is the last round.
//
// The tensor core rounds its f32 sums toward zero, twice a 16 keys, which on
// values of one sign took 1.1e-5 of an output after 2,300 keys and 1e-4 after
// 16,000.  So after kHold key tiles the compute threads take the leading part of D
// into 32 registers, a byte a dim in units of the row's own power of two, and leave
// D the rest, below 1/64 of the row's largest; it comes back at the end.  With 12
// tiles (192 additions) the error is 6.2e-6 at most on values of one sign and 2.9e-6
// of the norm on random ones, whatever the length (10 tiles: 5.0e-6 and 2.4e-6, and
// 2% more time on long rows).  It takes 12 of the 244 us above, 7% behind 16,000
// keys and nothing up to 1,536 keys.  Sums set aside whole instead, in the result's
// place, took 13 to 40 us more: they leave L2 between two looks.
// Measured and not taken: six slots of 16 KiB (286 us against 257 at the time),
// PV begun at the first half of P (no gain), 8 or 32 query rows in flight a
// warp (258 and 259 us against 252).
#include "pkv_elem.h"
#include "pkv_internal.h"
#include "pkv_softmax_tc.h"
#include "pkv_tcgen05.h"

namespace pkv {
namespace {

using namespace tc;

constexpr int kMaxHD = 128, kKeys = 128;
constexpr int kThreads = 384;
constexpr int kWarpMma0 = 8, kWarpLoad = 9, kWarpSpare = 11;  // warp 10: chain 1's MMAs
// registers per thread: at launch, then of warps 8-11 and of the compute warps
constexpr int kLaunchRegs = 168, kOtherRegs = 88, kComputeRegs = 208;
static_assert(256 * kComputeRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kQPiece = 32 * 1024;         // two k-blocks of 128 rows x 64 f16
constexpr uint32_t kSlot = 32 * 1024;           // K: two k-blocks of 128 keys; V^T: two of 128 dims
constexpr uint32_t kBlock = 16 * 1024;          // one k-block
constexpr int kSlots = 3, kLoneSlots = kSlots + 2;  // a lone tile's has the other's query pieces' place too
constexpr size_t kSmem = 4 * kQPiece + kSlots * kSlot + 1024;  // + alignment slack
static_assert(2 * kQPiece == (kLoneSlots - kSlots) * kSlot, "the second tile's pieces are whole slots");
constexpr float kGrow = 8.f;                    // log2 headroom of the reference maximum
constexpr int kPExp = 7;                        // C <= kPExp + c: p * 2^(C - c) <= 2^15
constexpr int kHold = 12;                       // key tiles until D's leading part is set aside
static_assert(kKeyTile == 64, "a key tile is two images");

__device__ __forceinline__ float pow2f(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }
__device__ __forceinline__ float mul_pow2(float x, int n) {  // n in [-252, 254], two exact steps
    return x * pow2f(n / 2) * pow2f(n - n / 2);
}
__device__ __forceinline__ int f16_scale_exp(float m) {  // brings m into [2^14, 2^15)
    return max(-113, min(126, 14 - (static_cast<int>((__float_as_uint(m) >> 23) & 255u) - 127)));
}
// a pair of f32 as f16 pieces, each pair packed (a in the low half)
__device__ __forceinline__ void split2(float a, float b, uint32_t &p0, uint32_t &p1) {
    const __half2 h0 = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h0);
    const __half2 h1 = __floats2half2_rn(a - f.x, b - f.y);
    p0 = *reinterpret_cast<const uint32_t *>(&h0);
    p1 = *reinterpret_cast<const uint32_t *>(&h1);
}

// Gc, Hc: the group and the head width where compiled in (0: taken from g_arg, hd_arg)
template <int Gc, int Hc>
__global__ void __launch_bounds__(kThreads, 1) prefill_q8_kernel(PrefillArgs a, int g_arg, int hd_arg) {
    const int G = Gc ? Gc : g_arg, kHD = Hc ? Hc : hd_arg;
    const int TQ = 128 / G;  // tokens per tile; rows past TQ * G stay empty
    extern __shared__ __align__(1024) unsigned char smraw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smraw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t bar_full[kLoneSlots], bar_free[kLoneSlots], bar_q[2], bar_s[2], bar_p[2], bar_o[2], bar_v;
    __shared__ uint32_t tslot;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int pi = blockIdx.x / a.n_kv, kvh = blockIdx.x - pi * a.n_kv;
    // the pair's tiles: one row and one split; the second may be absent
    const PrefillTile t0 = a.tiles[2 * pi], t1 = a.tiles[2 * pi + 1];
    const RowDesc rd = a.rows[t0.row];
    const int total_k = rd.past_len + rd.n_q;
    const int kbeg = t0.split * a.split_keys, kt0 = kbeg / kKeyTile, n_img = (total_k + kKeyTile - 1) / kKeyTile;
    auto tile_end = [&](const PrefillTile &t) {  // past the tile's last visible key of the split
        const int nv = min(TQ, rd.n_q - t.q0);
        return min(kbeg + a.split_keys, a.causal ? min(total_k, total_k - rd.n_q + t.q0 + nv) : total_k);
    };
    const int kend0 = tile_end(t0);
    int kend1 = kbeg;
    if (t1.row >= 0) {
        if (t1.row == t0.row && t1.split == t0.split) kend1 = tile_end(t1);
        else if (tid == 0 && a.err) atomicOr(a.err, 1);  // not a pair: the second tile is dropped
    }
    const int n0 = max(0, (kend0 - kbeg + kKeys - 1) / kKeys), n1 = max(0, (kend1 - kbeg + kKeys - 1) / kKeys);
    const int n_max = max(n0, n1);
    const bool lone = n1 == 0;  // chain 0 alone, on both S buffers
    const int ns = lone ? kLoneSlots : kSlots;
    unsigned char *ring = sm + (lone ? 2 : 4) * kQPiece;  // chain c's Q0 at 2c pieces, Q1 one on
    auto wait_w = [&](uint64_t *bar, uint32_t parity) {  // bounded; the warp agrees on the outcome
        return __all_sync(0xffffffffu, wait_phase(smem_u32(bar), parity & 1u)) != 0;
    };
    auto there = [&](uint64_t *bar, uint32_t parity) {  // without waiting
        return __all_sync(0xffffffffu, test_phase(smem_u32(bar), parity & 1u)) != 0;
    };
    auto slot = [&](int i) { return lone ? i % kLoneSlots : i % kSlots; };
    auto rph = [&](int i) { return static_cast<uint32_t>(lone ? i / kLoneSlots : i / kSlots); };

    if (warp == 0) {
        tmem_alloc(smem_u32(&tslot), kTmemCols);
        tmem_relinquish();
    }
    if (tid == 32 * kWarpLoad) {
        for (int i = 0; i < ns; ++i) {
            mbar_init(smem_u32(&bar_full[i]), 1);
            mbar_init(smem_u32(&bar_free[i]), lone ? 1 : 2);  // the issuing warps
        }
        mbar_init(smem_u32(&bar_v), 1);
        for (int c = 0; c < 2; ++c) {
            mbar_init(smem_u32(&bar_q[c]), 4);
            mbar_init(smem_u32(&bar_s[c]), 1);
            mbar_init(smem_u32(&bar_p[c]), lone ? 4 : 5);  // four compute warps, and the chain's turn
            mbar_init(smem_u32(&bar_o[c]), 1);
        }
        fence_proxy_async();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = __shfl_sync(0xffffffffu, tslot, 0);
    bool ok = true;
    const int32_t *slots = a.img_slot + a.img_tile0[t0.row];
    auto image = [&](int kt) {
        return a.img + (static_cast<size_t>(__ldg(slots + kt)) * a.n_kv + kvh) * kImageBytes;
    };
    // a tile's second image: past the row's last one the first stands in (its
    // keys are masked; what counts is that the bytes are a tile's values)
    auto second = [&](int kt) { return kt + 1 < n_img ? kt + 1 : kt; };

    if (warp >= 8) {
        setmaxnreg_dec<kOtherRegs>();
        if (warp == kWarpSpare) {
            // nothing to do
        } else if (warp == kWarpLoad) {
            // ---------------- copies (one lane): K_0, V_0, K_1, ... ----------------
            int issued = 0;
            for (int i = 0; i < 2 * n_max; ++i) {
                const int sl = slot(i), kt = kt0 + 2 * (i >> 1);
                const unsigned char *ia = image(kt), *ib = image(second(kt));  // looked up before the slot is free
                if (i >= ns && !wait_w(&bar_free[sl], rph(i) - 1)) break;
                if (elect_lane()) {
                    const uint32_t dst = smem_u32(ring + sl * kSlot), bar = smem_u32(&bar_full[sl]);
                    const uint32_t n_kb = kHD > 64 ? 2 : 1, v_bytes = kHD * 128;
                    mbar_expect_tx(bar, (i & 1) ? 2 * v_bytes : n_kb * kBlock);
                    if (i & 1) {  // V^T: a k-block of 64 keys each
                        bulk_g2s(dst, ia + 2 * kImagePlane, v_bytes, bar);
                        bulk_g2s(dst + kBlock, ib + 2 * kImagePlane, v_bytes, bar);
                    } else {      // K: of each k-block of 64 dims, 64 keys each
                        for (uint32_t kb = 0; kb < n_kb; ++kb) {
                            bulk_g2s(dst + kb * kBlock, ia + kb * (kBlock / 2), kBlock / 2, bar);
                            bulk_g2s(dst + kb * kBlock + kBlock / 2, ib + kb * (kBlock / 2), kBlock / 2, bar);
                        }
                    }
                }
                __syncwarp();
                issued = i + 1;
            }
            // the last copies land before the CTA's shared memory is given up (bounded)
            for (int i = max(0, issued - ns); i < issued; ++i) wait_w(&bar_full[slot(i)], rph(i));
        } else {
            // ---------------- MMA issue: chain c (one lane) ----------------
            const int c = warp == kWarpMma0 ? 0 : 1, n = c ? n1 : n0;
            const uint32_t tO = tbase + 128 * c;
            constexpr uint32_t idesc = idesc_f16(128, 128);
            const uint32_t idesc_v = idesc_f16(128, kHD);
            const int nk = kHD / 16;
            const uint64_t dQ0 = desc_sw128(smem_u32(sm + 2 * c * kQPiece)), dQ1 = desc_sw128(smem_u32(sm + (2 * c + 1) * kQPiece));
            // S_c = Q_c K_j^T, then the barriers; on the way the turn passes
            // (b: the S buffer, a chain's own or a lone chain's of the tile)
            auto qk = [&](int j, int b, bool pass) {
                const uint32_t tS = tbase + 256 + 128 * b;
                const int sl = slot(2 * j);
                const uint64_t dK = desc_sw128(smem_u32(ring + sl * kSlot));
                if (elect_lane()) {
#pragma unroll
                    for (int k = 0; k < 2 * (kMaxHD / 16); ++k) {  // the small pieces first: fewer additions to a large sum
                        const int x = k & 7;
                        const uint64_t o = ((x >> 2) * kBlock + (x & 3) * 32u) >> 4;
                        if (x < nk) mma_f16(tS, (k < 8 ? dQ1 : dQ0) + o, dK + o, idesc, k > 0);
                        if (k == 8 + max(0, nk - 3) && pass) mbar_arrive(smem_u32(&bar_p[c ^ 1]));
                    }
                    mma_commit(smem_u32(&bar_s[b]));
                    mma_commit(smem_u32(&bar_free[sl]));
                }
                __syncwarp();
            };
            // D_c += P_c V_j
            auto pv = [&](int j, int b) {
                const uint32_t tS = tbase + 256 + 128 * b;
                const int sv = slot(2 * j + 1);
                const uint64_t dV = desc_sw128(smem_u32(ring + sv * kSlot));
                if (elect_lane()) {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k) {
                        const uint64_t o = ((k >> 2) * kBlock + (k & 3) * 32u) >> 4;
                        mma_f16_ts(tO, tS + 8 * k, dV + o, idesc_v, j > 0 || k > 0);
                        mma_f16_ts(tO, tS + 64 + 8 * k, dV + o, idesc_v, 1);
                    }
                    mma_commit(smem_u32(&bar_free[sv]));
                    if (lone) mma_commit(smem_u32(&bar_v));
                    if (j + 1 == n) mma_commit(smem_u32(&bar_o[c]));
                }
                __syncwarp();
            };
            if (n > 0) {
                ok = wait_w(&bar_q[c], 0) && wait_w(&bar_full[0], 0);
                if (ok) {
                    fence_after_sync();
                    qk(0, c, false);
                }
            }
            // a lone chain: QK(j + 1) runs under softmax(j).  A compute warp may be
            // a tile ahead of another, so S and P have a barrier a buffer.
            for (int j = 0; lone && j < n && ok; ++j) {
                const int iv = 2 * j + 1;
                if (j + 1 < n) {
                    ok = wait_w(&bar_full[slot(iv + 1)], rph(iv + 1));
                    if (!ok) break;
                    fence_after_sync();
                    qk(j + 1, (j + 1) & 1, false);
                }
                ok = wait_w(&bar_full[slot(iv)], rph(iv)) && wait_w(&bar_p[j & 1], j >> 1);
                if (!ok) break;
                fence_after_sync();
                pv(j, j & 1);
            }
            for (int j = 0; !lone && j < n && ok; ++j) {
                const int iv = 2 * j + 1, sv = slot(iv);
                ok = wait_w(&bar_full[sv], rph(iv));
                // (a K tile that is not there yet is waited for after PV)
                const bool k_there = ok && j + 1 < n && there(&bar_full[slot(iv + 1)], rph(iv + 1));
                // P, and the chain's turn: the other chain's products before these
                // (chain 0's of tile j, chain 1's of tile j - 1), or the most of
                // them, have been issued; a chain without such products takes it
                if (ok && !(c ? j < n0 : j > 0 && j - 1 < n1) && elect_lane()) mbar_arrive(smem_u32(&bar_p[c]));
                if (ok) ok = wait_w(&bar_p[c], j);
                if (!ok) break;
                fence_after_sync();
                pv(j, c);
                const bool pass = c ? j + 1 < n0 : j < n1;  // the other chain's products follow
                if (j + 1 < n && !k_there) ok = wait_w(&bar_full[slot(iv + 1)], rph(iv + 1));
                if (!ok) break;
                fence_after_sync();
                if (j + 1 < n) qk(j + 1, c, pass);
                else if (pass && elect_lane()) mbar_arrive(smem_u32(&bar_p[c ^ 1]));
                __syncwarp();
            }
            // items past the chain's last tile are free as far as this chain goes
            // (counted once they have landed, so that each counts for its own phase)
            for (int i = 2 * n; !lone && i < 2 * n_max && ok; ++i) {
                ok = wait_w(&bar_full[slot(i)], rph(i));
                if (ok && elect_lane()) mbar_arrive(smem_u32(&bar_free[slot(i)]));
            }
            if (!ok && lane == 0 && a.err) atomicOr(a.err, 2);
        }
    } else {
        // -------------- compute warps: one thread per tile row and chain --------------
        setmaxnreg_inc<kComputeRegs>();
        const int c = warp >> 2, n = c ? n1 : n0, m = tid & 127;
        const int tq = m / G, g = m - tq * G, qi = (c ? t1.q0 : t0.q0) + tq;
        const bool valid = tq < TQ && qi < rd.n_q;
        const int klim = min(valid ? (a.causal ? total_k - rd.n_q + qi + 1 : total_k) : 1, c ? kend1 : kend0);
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tO = tbase + lanes + 128 * c;
        if (n > 0) {
            // the query rows in base-2 units, times a power of two each, as two
            // pieces.  A warp reads its 32 rows one after another, 512 bytes at
            // once (a row a thread took ~16,000 clocks for a CTA); lane l
            // holds dims 4l .. 4l + 3 and keeps row l's exponent.
            int qexp = 0;
            {
                const int w0 = 32 * (warp & 3), q0 = c ? t1.q0 : t0.q0;
                const float *qb = a.Q + static_cast<size_t>(rd.q_row0) * (a.n_heads * kHD) + static_cast<size_t>(kvh * G) * kHD + 4 * lane;
                unsigned char *d = sm + 2 * c * kQPiece + (lane >> 4) * kBlock + (lane & 1) * 8;  // k-block lane / 16
                auto load = [&](int r0, float4 (&q)[8]) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const int row = w0 + r0 + r, t = q0 + row / G;
                        q[r] = row / G < TQ && t < rd.n_q && 4 * lane < kHD
                                   ? __ldg(reinterpret_cast<const float4 *>(
                                         qb + static_cast<size_t>(t) * (a.n_heads * kHD) + (row % G) * kHD))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                };
                auto store = [&](int r0, const float4 (&q)[8]) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        float4 x = q[r];
                        x.x *= a.scale_log2, x.y *= a.scale_log2, x.z *= a.scale_log2, x.w *= a.scale_log2;
                        // largest magnitude as bits; a NaN or an infinity counts as none (its products are not finite)
                        const float mx = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
                        const int e = f16_scale_exp(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx))));
                        if (lane == r0 + r) qexp = e;
                        const float up = pow2f(e);
                        uint2 c0, c1;
                        split2(x.x * up, x.y * up, c0.x, c1.x);
                        split2(x.z * up, x.w * up, c0.y, c1.y);
                        const uint32_t off = sw128_chunk(w0 + r0 + r, (lane >> 1) & 7);
                        if (4 * lane < kHD) {
                            *reinterpret_cast<uint2 *>(d + off) = c0;
                            *reinterpret_cast<uint2 *>(d + off + kQPiece) = c1;
                        }
                    }
                };
                float4 qa[8], qc[8];  // sixteen rows on the way
                load(0, qa);
                load(8, qc);
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 16) {
                    store(r0, qa);
                    if (r0 == 0) load(16, qa);
                    store(r0 + 8, qc);
                    if (r0 == 0) load(24, qc);
                }
            }
            fence_proxy_async();  // before the MMAs read them
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_q[c]));

            float m_ref = -INFINITY, l_run = 0.f;
            int cexp = 0;  // C: D + h * unit, h of hold's bytes, is 2^C x the output's sum
            uint32_t hold[kMaxHD / 4];
            float unit = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxHD / 4; ++i) hold[i] = 0x80808080u;
            auto exps = [&](int kt) { return __ldg(reinterpret_cast<const int2 *>(image(kt) + kImageExpOff)); };
            int2 ea = exps(kt0), eb = exps(second(kt0));  // the images' exponents (K, V), a tile ahead
            for (int j0 = 0; j0 < n && ok; j0 += kHold) {
                if (j0 > 0) {
                    ok = wait_w(&bar_s[lone ? j0 & 1 : c], lone ? j0 >> 1 : j0) && (!lone || wait_w(&bar_v, j0 - 1));
                    if (!ok) break;
                    fence_after_sync();
                    uint32_t x[kMaxHD];
#pragma unroll
                    for (int i = 0; i < kMaxHD; i += 32) tmem_ld32_issue(tO + i, x + i);
                    tmem_ld_done(x);
                    unit = set_aside(x, hold, unit, j0 > kHold, kHD);  // (columns past the width hold anything)
#pragma unroll
                    for (int i = 0; i < kMaxHD; i += 16) {
                        if (i >= kHD) continue;
                        float v[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(x[i + k]);
                        tmem_st16(tO + i, v);
                    }
                    tmem_st_wait();  // (D may be rescaled next)
                }
                for (int j = j0; j < min(n, j0 + kHold); ++j) {
                    const int base = kbeg + j * kKeys;
                    const int ke[2] = {ea.x, eb.x}, ve[2] = {ea.y, eb.y};
                    if (j + 1 < n) {
                        const int kt = kt0 + 2 * (j + 1);
                        ea = exps(kt);
                        eb = exps(second(kt));
                    }
                    const int b = lone ? j & 1 : c;
                    const uint32_t tS = tbase + lanes + 256 + 128 * b;
                    ok = wait_w(&bar_s[b], lone ? j >> 1 : j);
                    if (!ok) break;
                    fence_after_sync();
                    uint32_t x[kKeys];  // the row's scores (f32 bits)
#pragma unroll
                    for (int i = 0; i < kKeys; i += 32) tmem_ld32_issue(tS + i, x + i);
                    tmem_ld_done(x);
                    auto xf = [&](int i) { return __uint_as_float(x[i]); };
                    // scores to base-2 units: one exact factor 2^sn a half (two steps
                    // where 2^sn is not a normal f32)
                    float fsc[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int sn = -(qexp + ke[h]);
                        const bool one = sn >= -126 && sn <= 127;
                        fsc[h] = one ? pow2f(sn) : 1.f;
                        if (!one) {
#pragma unroll
                            for (int i = 0; i < 64; ++i) x[64 * h + i] = __float_as_uint(mul_pow2(xf(64 * h + i), sn));
                        }
                    }
                    if (base + kKeys > klim) {
#pragma unroll
                        for (int i = 0; i < kKeys; ++i) x[i] = base + i < klim ? x[i] : 0xff800000u;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float mx[2] = {fmaxf(xf(64 * h), xf(64 * h + 1)), fmaxf(xf(64 * h + 2), xf(64 * h + 3))};
#pragma unroll
                        for (int i = 4; i < 64; i += 2) mx[(i >> 1) & 1] = max3(mx[(i >> 1) & 1], xf(64 * h + i), xf(64 * h + i + 1));
                        top = fmaxf(top, fmaxf(mx[0], mx[1]) * fsc[h]);
                    }
                    const bool move = m_ref != -INFINITY && top > m_ref + kGrow;
                    const float m_use = m_ref == -INFINITY || move ? top : m_ref;
                    const float nm = m_use == -INFINITY ? 0.f : -m_use;
                    const int vmin = min(ve[0], ve[1]);
                    const int c_new = j == 0 ? kPExp + vmin : min(cexp, kPExp + vmin);
                    const float f = move ? ex2(m_ref - m_use) : 1.f;
                    // D moves with the reference or with C (after PV(j - 1): QK(j), done,
                    // followed it, but for a lone chain's); the whole warp takes the
                    // branch, as TMEM accesses are the warp's
                    if (j > 0 && (c_new != cexp || __any_sync(0xffffffffu, move))) {
                        if (lone) {
                            ok = wait_w(&bar_v, j - 1);
                            if (!ok) break;
                            fence_after_sync();
                        }
                        const int d = c_new - cexp;
                        unit = mul_pow2(unit * f, d);
#pragma unroll 1
                        for (int i = 0; i < kHD / 16; ++i) {
                            float v[16];
                            tmem_ld16(tO + 16 * i, v);
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = mul_pow2(v[k] * f, d);
                            tmem_st16(tO + 16 * i, v);
                        }
                    }
                    m_ref = m_use;
                    cexp = c_new;
                    // P over S, half by half: two pieces of p * 2^(C - c)
                    uint64_t sum[2] = {0, 0};
                    const uint64_t nm2 = pair(nm, nm);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int pe = cexp - ve[h];  // <= kPExp
                        const float pf = pe >= -126 ? pow2f(pe) : 0.f;
                        const uint64_t f2 = pair(fsc[h], fsc[h]), pf2 = pair(pf, pf);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {  // 32 keys
                            uint32_t p0[16], p1[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int i = 64 * h + 32 * r + 2 * k;
                                const float2 e = unpair(fma2(pair(xf(i), xf(i + 1)), f2, nm2));
                                const uint64_t p = pair(ex2(e.x), ex2(e.y));
                                sum[k & 1] = add2(sum[k & 1], p);
                                const float2 y = unpair(mul2(p, pf2));
                                split2(y.x, y.y, p0[k], p1[k]);
                            }
                            tmem_st16u(tS + 32 * h + 16 * r, p0);
                            tmem_st16u(tS + 64 + 32 * h + 16 * r, p1);
                        }
                    }
                    const float2 s2 = unpair(add2(sum[0], sum[1]));
                    l_run = fmaf(l_run, f, s2.x + s2.y);
                    tmem_st_wait();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar_p[b]));
                }
            }
            if (ok) ok = wait_w(&bar_o[c], 0);
            if (!ok) {
                if (lane == 0 && a.err) atomicOr(a.err, 2);
            } else {
                fence_after_sync();
                // the result: D / l, then 2^-C (exact; in this order it does not
                // overflow where D * 2^-C, up to l times it, would)
                const PrefillTile tile = c ? t1 : t0;
                const bool direct = tile.part0 < 0;
                const int h = kvh * G + g;
                float *dst;
                size_t pidx = 0;
                if (direct) {
                    dst = a.out + static_cast<size_t>(rd.q_row0 + (valid ? qi : 0)) * (a.n_heads * kHD) + static_cast<size_t>(h) * kHD;
                } else {
                    const int nv = min(TQ, rd.n_q - tile.q0);
                    const int kend_tile = a.causal ? min(total_k, total_k - rd.n_q + tile.q0 + nv) : total_k;
                    const int stride = tile.stride > 0 ? tile.stride : (kend_tile + a.split_keys - 1) / a.split_keys;
                    pidx = static_cast<size_t>(tile.part0 + (valid ? tq : 0) * stride + tile.split) * a.n_heads + h;
                    dst = a.pacc + pidx * kHD;
                }
                const float scl = direct ? 1.f / l_run : 1.f;
                const bool vec = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;  // whole 32-byte sectors
#pragma unroll
                for (int i = 0; i < kMaxHD / 32; ++i) {
                    if (32 * i >= kHD) continue;
                    const int nd = min(32, kHD - 32 * i);  // 16 or 32 dims
                    float v[32];
                    tmem_ld32(tO + 32 * i, v);
                    if (n > kHold) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = fmaf(aside(hold[8 * i + k / 4], k & 3), unit, v[k]);
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = mul_pow2(v[k] * scl, -cexp);
                    if (!valid) {
                        // nothing to write
                    } else if (vec) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            if (k < nd) asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst + 32 * i + k),
                                         "f"(v[k]), "f"(v[k + 1]), "f"(v[k + 2]), "f"(v[k + 3]), "f"(v[k + 4]), "f"(v[k + 5]),
                                         "f"(v[k + 6]), "f"(v[k + 7])
                                         : "memory");
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            if (k < nd) *reinterpret_cast<float4 *>(dst + 32 * i + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                    __syncwarp();  // TMEM loads are the warp's
                }
                if (valid && !direct) {
                    a.pm[pidx] = m_ref;
                    a.pl[pidx] = l_run;
                }
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tbase, kTmemCols);
}

template <int G, int HD>
cudaError_t launch_g(const PrefillArgs &a, int hd, cudaStream_t s) {
    static PerDeviceOnce configured;  // the attributes are per function and device
    const cudaError_t ce = configured.run([&]() -> cudaError_t {
        // setmaxnreg.inc waits for registers of the launch's own: launch only
        // if the kernel starts with what the split was sized for
        cudaFuncAttributes fa{};
        cudaError_t e = cudaFuncGetAttributes(&fa, prefill_q8_kernel<G, HD>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kLaunchRegs || fa.maxThreadsPerBlock < kThreads) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(prefill_q8_kernel<G, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem));
    });
    if (ce != cudaSuccess) return ce;
    if (a.n_tiles <= 0 || (a.n_tiles & 1) || !a.img || !a.img_tile0 || !a.img_slot) return cudaErrorInvalidValue;
    const long long grid = static_cast<long long>(a.n_tiles / 2) * a.n_kv;
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    prefill_q8_kernel<G, HD><<<static_cast<unsigned>(grid), kThreads, kSmem, s>>>(a, a.group, hd);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_q8(const PrefillArgs &a, int hd, cudaStream_t s) {
    if (!prefill_shape_q8(hd, a.group)) return cudaErrorInvalidValue;
    if (hd != kMaxHD) return launch_g<0, 0>(a, hd, s);
    switch (a.group) {
        case 1: return launch_g<1, kMaxHD>(a, hd, s);
        case 2: return launch_g<2, kMaxHD>(a, hd, s);
        case 4: return launch_g<4, kMaxHD>(a, hd, s);
        case 8: return launch_g<8, kMaxHD>(a, hd, s);
        default: return launch_g<0, kMaxHD>(a, hd, s);
    }
}

}  // namespace pkv

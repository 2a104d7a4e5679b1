// pkv_ragged_tc.h -- many query rows over keys of other lengths (cross
// attention's prompts, prompts behind a shared prefix, the stacked rows of a
// batch over the prefix) on the tensor-core kernel of packed rows
// (pkv_packed_tc.h): its tiles, chains and turns, with keys from two stretches
// of rows (the prefix's, then the run's own) and, where a launch has few
// pieces, the key tiles split and partial records written in place of outputs.
//
// Sequences whose own key rows lie in the order of their queries go as stretches
// of rows, so that short ones share tiles: 300 answers of 2 to 24
// tokens behind a prefix of 1,100, 28 heads over 4: 176 us by sequences of their own, 51 so.
//
// The prefix's last tile is filled up with zeros by its own tensor map, so only
// tiles of a run's own keys are looked over for values that are not finite.
#pragma once

#include "pkv_packed_tc.h"

#include <algorithm>

namespace pkv {
namespace {

template <int D, class T, int N, bool kLong, class F>
__global__ void __launch_bounds__(kTcThreads, 1)
    ragged_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mkp,
                     const __grid_constant__ CUtensorMap mvp, const __grid_constant__ RaggedArgs a,
                     const __grid_constant__ RunList<RaggedRun, N> l, int heads) {
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    packed_tc<D, T, kLong, F>(mq, mk, mv, mkp, mvp, a, l, heads);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");  // so that the join behind this launch has all of them
}

template <int D, class T, int N, bool kLong, class F>
cudaError_t tc_n(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches, cudaStream_t s) {
    using C = TcCfg<D>;
    static PerDeviceOnce configured;  // the attributes are per function and device
    cudaError_t e = configured.run([&]() -> cudaError_t {
        // setmaxnreg.inc waits for registers of the launch's own: launch only
        // if the kernel starts with what the split was sized for
        cudaFuncAttributes fa{};
        const cudaError_t c = cudaFuncGetAttributes(&fa, ragged_tc_kernel<D, T, N, kLong, F>);
        if (c != cudaSuccess) return c;
        if (fa.numRegs < kTcLaunchRegs || fa.maxThreadsPerBlock < kTcThreads) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(ragged_tc_kernel<D, T, N, kLong, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(C::kSmem));
    });
    if (e != cudaSuccess) return e;
    const int heads = ragged_tile_heads(a.n_heads / a.n_kv), tokens = ragged_piece_tokens(heads, a.hd);  // of a tile, of a piece
    RunList<RaggedRun, N> l;
    l.n = n;
    int64_t at = 0, q_rows = 0, k_rows = 0;
    for (int32_t i = 0; i < n; ++i) {
        l.run[i] = runs[i];
        l.unit0[i] = static_cast<int32_t>(at);
        if (!F::kStacks) at += static_cast<int64_t>(ragged_pieces(runs[i].nq, tokens)) * runs[i].ns;
        q_rows = std::max<int64_t>(q_rows, static_cast<int64_t>(runs[i].q0) + runs[i].nq);
        k_rows = std::max<int64_t>(k_rows, static_cast<int64_t>(runs[i].k0) + runs[i].nk);
        if (at > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    }
    l.unit0[n] = static_cast<int32_t>(at);
    for (int32_t x = 0; F::kStacks && x < n_stretches; ++x) {
        const RaggedRun &f = runs[first[x]], &e = runs[(x + 1 < n_stretches ? first[x + 1] : n) - 1];
        l.unit0[x] = static_cast<int32_t>(at);
        l.run[x].kind = first[x];
        at += static_cast<int64_t>(ragged_pieces(e.q0 + e.nq - f.q0, tokens)) * f.ns;
        if (at > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    }
    const int64_t grid = at * (a.n_heads / heads);
    if (grid <= 0 || grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    EncodeTiled f;
    CUtensorMap mq, mk, mv, mkp, mvp;
    e = encode_tiled(&f);
    if (e == cudaSuccess) e = rows_map(&mq, f, a.type, a.hd, q_rows, a.Q, a.q_stride, a.n_heads, heads, 128 / heads);
    if (e == cudaSuccess) e = rows_map(&mk, f, a.type, a.hd, k_rows, a.K, a.k_stride, a.n_kv, 1, kKeys);
    if (e == cudaSuccess) e = rows_map(&mv, f, a.type, a.hd, k_rows, a.V, a.v_stride, a.n_kv, 1, kKeys);
    mkp = mk;
    mvp = mv;
    if (a.n_pre > 0) {
        if (e == cudaSuccess) e = rows_map(&mkp, f, a.type, a.hd, a.n_pre, a.Kp, a.kp_stride, a.n_kv, 1, kKeys);
        if (e == cudaSuccess) e = rows_map(&mvp, f, a.type, a.hd, a.n_pre, a.Vp, a.vp_stride, a.n_kv, 1, kKeys);
    }
    if (e != cudaSuccess) return e;
    RaggedArgs b = a;
    b.n_stretches = n_stretches;
    b.out32 = a.hd % 16 == 0 && a.o_stride % 16 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, ragged_tc_kernel<D, T, N, kLong, F>, mq, mk, mv, mkp, mvp, b, l, heads);
}

template <int D, class T>
cudaError_t tc_d(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches, cudaStream_t s) {
    const bool stack = n_stretches > 0;
    constexpr bool kT = D == 64;  // (128-wide heads have ring slots for two and a half tiles only)
    constexpr int kC = TcCfg<D>::kChains, kS = kRaggedSmall, kL = kRaggedLarge;
    bool is_long = false;  // some piece adds more keys than a sum takes
    for (int32_t i = 0; i < n && !stack; ++i) is_long = is_long || ragged_split_tiles(a.n_pre, runs[i]) * kKeys > kLongKeys;
    if constexpr (D > 128) {
        if (is_long) return cudaErrorInvalidValue;
        return stack ? tc_n<D, T, kL, false, Stacks<kL, kC, kT>>(a, runs, n, first, n_stretches, s) : tc_n<D, T, kL, false, Runs<kL, kC, kT>>(a, runs, n, first, n_stretches, s);
    } else {
        if (stack) return n <= kS ? tc_n<D, T, kS, false, Stacks<kS, kC, kT>>(a, runs, n, first, n_stretches, s) : tc_n<D, T, kL, false, Stacks<kL, kC, kT>>(a, runs, n, first, n_stretches, s);
        if (is_long) return tc_n<D, T, kL, true, Runs<kL, kC, false>>(a, runs, n, first, n_stretches, s);  // (sums set aside stay with their chain)
        return n <= kS ? tc_n<D, T, kS, false, Runs<kS, kC, kT>>(a, runs, n, first, n_stretches, s) : tc_n<D, T, kL, false, Runs<kL, kC, kT>>(a, runs, n, first, n_stretches, s);
    }
}
template <class T>
cudaError_t tc_t(const RaggedArgs &a, const RaggedRun *runs, int32_t n, const int32_t *first, int32_t n_stretches, cudaStream_t s) {
    if (a.hd <= 64) return tc_d<64, T>(a, runs, n, first, n_stretches, s);
    if (a.hd <= 128) return tc_d<128, T>(a, runs, n, first, n_stretches, s);
    if (a.hd <= 192) return tc_d<192, T>(a, runs, n, first, n_stretches, s);
    return tc_d<256, T>(a, runs, n, first, n_stretches, s);
}

}  // namespace

}  // namespace pkv

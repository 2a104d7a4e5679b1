"""8-bit pools with a scale per (block, layer, kv head): the append's elements
and scales bit for bit against the oracle, attention over them against the
formula in 64 bits over the same stored values, and packed append / read back.

Attention reads the stored values exactly and keeps f32 accuracy, so its
tolerance is the f32 one of every pool: 1e-5 max|V| + 1e-6.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_nx_gb300 as pkv
from gpu_helpers import tolerance
from synth.workloads import release_order

pytestmark = pytest.mark.gpu


class Q8Pool:
    def __init__(self, n_blocks, n_layers, KV, hd, bs, max_seqs=64, max_blocks=4096, shuffle=True):
        self.KV, self.hd, self.bs, self.n_layers = KV, hd, bs, n_layers
        self.K = torch.full((n_blocks, n_layers, bs, KV * hd), 255, dtype=torch.uint8, device="cuda")
        self.V = torch.full_like(self.K, 255)
        # a scale nobody wrote poisons what reads it
        self.Ks = torch.full((n_blocks, n_layers, KV), float("nan"), device="cuda")
        self.Vs = torch.full_like(self.Ks, float("nan"))
        self.p = pkv.pkv_pool_new_q8(n_blocks, n_layers, KV, hd, bs, self.K, self.V, self.Ks, self.Vs, max_seqs,
                                     max_blocks, torch.cuda.current_stream())
        assert self.p, pkv.pkv_last_error()
        if shuffle:
            for _ in range(n_blocks):
                pkv.pkv_alloc_block(self.p)
            for b in release_order(n_blocks, 5):
                pkv.pkv_unref_block(self.p, int(b))

    def seq(self, max_tokens):
        s = pkv.pkv_seq_new(self.p, max_tokens)
        assert s, pkv.pkv_last_error()
        return s

    def append(self, seqs, x, y, n, layers=None):
        """Ensure, append (every layer) and advance."""
        pkv.check(pkv.pkv_ensure_append_batch(seqs, n))
        for layer in range(self.n_layers) if layers is None else layers:
            pkv.check(pkv.pkv_append_packed(seqs, n, layer, x, y))
        pkv.check(pkv.pkv_advance_batch(seqs, n))

    def values(self, seq, n, layer=0):
        """Stored K, V of rows [0, n) in 64 bits: [n, KV, hd]."""
        ids = torch.tensor(pkv.pkv_seq_page_table(seq), device="cuda")
        out = []
        for e, s in ((self.K, self.Ks), (self.V, self.Vs)):
            v = (e[ids, layer].double() - 128).view(-1, self.bs, self.KV, self.hd) * s[ids, layer].double()[:, None, :, None]
            out.append(v.reshape(-1, self.KV, self.hd)[:n])
        return out

    def ok(self):
        assert pkv.pkv_sync_error(self.p) == pkv.PKV_OK, pkv.pkv_last_error()

    def close(self):
        torch.cuda.synchronize()
        pkv.pkv_pool_free(self.p)


def randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(dtype)


# ------------------------------------------------------------------ append ----

class Model:
    """The oracle's blocks of one sequence (K or V), by page index."""

    def __init__(self, bs, KV, hd):
        self.bs, self.KV, self.hd, self.q, self.e = bs, KV, hd, {}, {}

    def append(self, pos, x):
        x = x.reshape(-1, self.KV, self.hd)
        while len(x):
            pg, off = divmod(pos, self.bs)
            m = min(self.bs - off, len(x))
            for h in range(self.KV):
                q, e = oracle.q8_append(self.q.get((pg, h), np.zeros((self.bs, self.hd))), self.e.get((pg, h), 0),
                                        x[:m, h], off)
                self.q[pg, h], self.e[pg, h] = q, e
            pos += m
            x = x[m:]


@pytest.mark.parametrize("KV,hd,bs", [(2, 128, 16), (3, 64, 5), (1, 20, 4), (4, 96, 32), (2, 6, 1), (1, 256, 100)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
def test_append_bit_exact(KV, hd, bs, dtype):
    """Random chunks of growing and shrinking magnitude into several sequences, strided rows; elements, scales and
    untouched places."""
    pool = Q8Pool(200, 2, KV, hd, bs)
    try:
        rng = np.random.RandomState(KV * hd + bs)
        seqs = [pool.seq(20 * bs + 40) for _ in range(3)]
        models = [[Model(bs, KV, hd) for _ in range(2)] for _ in seqs]
        lens = [0, 0, 0]
        for step in range(9):
            n = [int(rng.choice([1, 1, 2, bs, bs + 1, 2 * bs + 3])) for _ in seqs]
            w = torch.randn(sum(n), 2 * KV * hd + 8, device="cuda") * 2.0 ** int(rng.randint(-6, 7))
            w[0, :3] = 0.0
            w = w.to(dtype)
            x, y = w[:, :KV * hd], w[:, KV * hd + 8:]
            pool.append(seqs, x, y, n, layers=[1])
            at = 0
            for r, s in enumerate(seqs):
                for which, t in enumerate((x, y)):
                    models[r][which].append(lens[r], t[at:at + n[r]].double().cpu().numpy())
                at += n[r]
                lens[r] += n[r]
        pool.ok()
        for r, s in enumerate(seqs):
            ids = pkv.pkv_seq_page_table(s)
            for which, (E, S) in enumerate(((pool.K, pool.Ks), (pool.V, pool.Vs))):
                for pg, b in enumerate(ids):
                    rows = min(bs, lens[r] - pg * bs)
                    e = E[b, 1].cpu().numpy().astype(np.float64).reshape(bs, KV, hd)
                    for h in range(KV):
                        assert np.array_equal(e[:rows, h] - 128, models[r][which].q[pg, h][:rows]), (r, which, pg, h)
                        assert S[b, 1, h].item() == 2.0 ** models[r][which].e[pg, h]
                    assert (e[rows:] == 255).all()          # places nobody wrote
        assert bool((pool.K[:, 0] == 255).all()) and bool(torch.isnan(pool.Ks[:, 0]).all())   # the other layer
    finally:
        pool.close()


def test_append_extremes():
    """Zeros, the smallest and largest magnitudes, exact borders of the scale and of rounding."""
    pool = Q8Pool(40, 1, 1, 4, 1)
    try:
        rows = torch.tensor([[0, 0, 0, 0], [1e-45, 0, 0, 0], [127, 63.5, 0.5, 1.5], [127.00001, 1, 3, 5],
                             [3.4028234663852886e38, 1, 0, -3.4028234663852886e38], [-127, 127, -0.5, 2.5],
                             [2.0 ** -126 * 127, 2.0 ** -126, 2.0 ** -127, 0], [0.9921875, 2.0 ** -8, -2.0 ** -8, 0]],
                            device="cuda")
        s = pool.seq(16)
        pool.append([s], rows, -rows, [len(rows)])
        pool.ok()
        ids = pkv.pkv_seq_page_table(s)
        for i, b in enumerate(ids):
            for sign, (E, S) in ((1, (pool.K, pool.Ks)), (-1, (pool.V, pool.Vs))):
                q, e = oracle.q8_append(np.zeros((1, 4)), 0, sign * rows[i:i + 1].double().cpu().numpy(), 0)
                assert S[b, 0, 0].item() == 2.0 ** e, i
                assert (E[b, 0, 0].cpu().numpy().astype(float) - 128).tolist() == q[0].tolist(), i
    finally:
        pool.close()


def test_not_finite_rows_poison_their_block_and_head_until_it_is_rewritten():
    KV, hd, bs = 2, 64, 4
    pool = Q8Pool(20, 1, KV, hd, bs)
    try:
        s = pool.seq(40)
        x = randn(10, KV * hd, seed=1)
        x[5, 3] = float("inf")                  # page 1, head 0
        pool.append([s], x, x, [10])
        ids = pkv.pkv_seq_page_table(s)
        assert torch.isnan(pool.Ks[ids[1], 0, 0]) and torch.isnan(pool.Vs[ids[1], 0, 0])
        assert bool(torch.isfinite(pool.Ks[ids[1], 0, 1])) and bool(torch.isfinite(pool.Ks[ids[0], 0]).all())
        q = randn(1, 4 * hd, seed=2)
        out = torch.empty(1, 4 * hd, device="cuda")
        n = randn(1, KV * hd, seed=3)
        pkv.check(pkv.pkv_ensure_append(s, 1))
        pkv.check(pkv.pkv_attn_batch([s], [1], q, n, n, 4, KV, hd, 0, 1, 0.125, out))
        pool.ok()
        assert bool(torch.isnan(out[0, :2 * hd]).all()) and bool(torch.isfinite(out[0, 2 * hd:]).all())
        pkv.check(pkv.pkv_seq_truncate(s, 6))   # the rewritten rows start inside the block: it stays NaN
        pool.append([s], n, n, [1])
        assert torch.isnan(pool.Ks[pkv.pkv_seq_page_table(s)[1], 0, 0])
        pkv.check(pkv.pkv_seq_truncate(s, 4))   # from its first row: finite again
        pool.append([s], n, n, [1])
        assert bool(torch.isfinite(pool.Ks[pkv.pkv_seq_page_table(s)[1], 0]).all())
    finally:
        pool.close()


def test_forks_copy_scales():
    """A fork's append copies the shared tail block with its scales; the parent keeps its own."""
    KV, hd, bs = 2, 64, 8
    pool = Q8Pool(20, 2, KV, hd, bs)
    try:
        a = pool.seq(64)
        x = randn(13, KV * hd, seed=1)
        pool.append([a], x, x * 2, [13])
        b = pkv.pkv_seq_fork(a)
        before = [t.clone() for t in pool.values(a, 13, 1)]
        big = randn(2, KV * hd, seed=2) * 100
        pool.append([b], big, big, [2])
        pool.ok()
        assert all(torch.equal(x, y) for x, y in zip(pool.values(a, 13, 1), before))
        kb, _ = pool.values(b, 15, 1)
        step = pool.Ks[pkv.pkv_seq_page_table(b)[1], 1].max().item()
        assert (kb[8:13] - before[0][8:13]).abs().max().item() <= step / 2
        assert (kb[13:].reshape(2, -1) - big.double()).abs().max().item() <= step / 2
        assert torch.equal(kb[:8], before[0][:8])
    finally:
        pool.close()


# -------------------------------------------------------------- packed rows ----

@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8", "q8"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("KV,hd,bs", [(2, 128, 16), (1, 20, 3), (3, 96, 64)])
def test_packed_append_and_read(kind, dtype, KV, hd, bs):
    """What an append of packed rows stores equals the row-by-row append's, and reads back as those values."""
    kd, nb = KV * hd, 64
    flags = {"bf16": pkv.PKV_POOL_BF16, "fp8": pkv.PKV_POOL_FP8}.get(kind, 0)
    st = torch.cuda.current_stream()

    def make():
        p = (pkv.pkv_pool_new_q8(nb, 1, KV, hd, bs, max_seqs=8, max_blocks_per_seq=60, stream=st) if kind == "q8" else
             pkv.pkv_pool_new(nb, 1, kd, bs, max_seqs=8, max_blocks_per_seq=60, stream=st, flags=flags))
        assert p, pkv.pkv_last_error()
        if kind == "fp8":
            pkv.check(pkv.pkv_pool_set_kv_scale(p, 0.5))
        return p, [pkv.pkv_seq_new(p, 60) for _ in range(3)]

    n = [1, 2 * bs % 50 + 3, 17]
    x, y = randn(sum(n), kd + 8, seed=1, dtype=dtype)[:, :kd], randn(sum(n), kd, seed=2, dtype=dtype)
    got = []
    for packed in (True, False):
        p, seqs = make()
        try:
            pkv.check(pkv.pkv_ensure_append_batch(seqs, n))
            at = 0
            if packed:
                pkv.check(pkv.pkv_append_packed(seqs, n, 0, x, y))
            else:
                for s, m in zip(seqs, n):
                    pkv.check(pkv.pkv_append_layer(s, 0, x[at:at + m].float().contiguous(), y[at:at + m].float().contiguous(), m))
                    at += m
            k, v = (torch.full((sum(n) + 2, kd + 16), 3.0, device="cuda") for _ in range(2))
            pkv.check(pkv.pkv_read_packed(seqs, [0, 0, 0], n, 0, k[:, 8:8 + kd], v[:, 8:8 + kd]))
            assert pkv.pkv_sync_error(p) == pkv.PKV_OK
            for t in (k, v):   # nothing beside or behind the rows
                assert bool((t[:, :8] == 3).all()) and bool((t[:, 8 + kd:] == 3).all()) and bool((t[sum(n):] == 3).all())
            got.append((k[:sum(n), 8:8 + kd].clone(), v[:sum(n), 8:8 + kd].clone()))
            if packed:
                # ranges, a sequence twice, another type (each value rounded once)
                h, w = (torch.empty(6, kd, dtype=torch.float16, device="cuda") for _ in range(2))
                pkv.check(pkv.pkv_read_packed([seqs[2], seqs[1], seqs[2]], [5, 1, 0], [3, 1, 2], 0, h, w))
                torch.cuda.synchronize()
                o1, o2 = n[0], n[0] + n[1]
                rows = [o2 + 5, o2 + 6, o2 + 7, o1 + 1, o2, o2 + 1]
                assert torch.equal(h, got[0][0][rows].half()) and torch.equal(w, got[0][1][rows].half())
        finally:
            torch.cuda.synchronize()
            pkv.pkv_pool_free(p)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    if kind == "f32":
        assert torch.equal(got[0][0], x.float()) and torch.equal(got[0][1], y.float())
    elif kind == "bf16":
        assert torch.equal(got[0][0], x.to(torch.bfloat16).float())
    elif kind == "fp8":
        assert torch.equal(got[0][0], (x.float() / 0.5).to(torch.float8_e4m3fn).float() * 0.5)


def test_packed_rows_refusals():
    pool = Q8Pool(8, 1, 1, 64, 4, max_blocks=4)
    try:
        s = pool.seq(16)
        x = randn(4, 64, seed=1)
        assert pkv.pkv_append_packed([s], [2], 0, x, x) == pkv.PKV_ERR_SEQ            # not ensured
        assert pkv.pkv_read_packed([s], [0], [1], 0, x, x) == pkv.PKV_ERR_SEQ         # no pages
        pkv.check(pkv.pkv_ensure_append(s, 3))
        assert pkv.pkv_append_packed([s], [2], 1, x, x) == pkv.PKV_ERR_ARG            # layer
        assert pkv.pkv_append_packed([s, s], [1, 1], 0, x, x) == pkv.PKV_ERR_ARG      # twice
        assert pkv.pkv_read_packed([s], [-1], [1], 0, x, x) == pkv.PKV_ERR_SEQ
        assert pkv.pkv_read_packed([s], [2], [3], 0, x, x) == pkv.PKV_ERR_SEQ
        with pytest.raises(TypeError):
            pkv.pkv_append_packed([s], [3], 0, x[:2], x[:2])
        with pytest.raises(TypeError):
            pkv.pkv_append_packed([s], [3], 0, x.double(), x.double())
        f = pkv.pkv_seq_fork(s)
        assert pkv.pkv_append_packed([f], [1], 0, x, x) == pkv.PKV_ERR_SEQ            # a shared block
        q, o = randn(1, 128, seed=1), torch.empty(1, 128, device="cuda")
        pkv.check(pkv.pkv_seq_free(f))
        assert pkv.pkv_attn_batch([s], [1], q, x, x, 4, 2, 32, 0, 1, 1.0, o) == pkv.PKV_ERR_BAD_DIM   # other heads
        pkv.check(pkv.pkv_attn_batch([s], [1], q, x, x, 2, 1, 64, 0, 1, 1.0, o))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            pkv.check(pkv.pkv_pool_set_stream(pool.p, side))
            g.capture_begin()
            rcs = [pkv.pkv_append_packed([s], [1], 0, x, x), pkv.pkv_read_packed([s], [0], [1], 0, x, x),
                   pkv.pkv_attn_batch([s], [1], q, x, x, 2, 1, 64, 0, 1, 1.0, o)]
            o.add_(1.0)
            g.capture_end()
        assert rcs == [pkv.PKV_ERR_ARG] * 3
        pool.ok()
    finally:
        pool.close()


# --------------------------------------------------------------- attention ----

def attend_case(H, KV, hd, bs, past, nq, causal=1, seed=0, layers=1, host=False, rope=0.0, scales=None, mul=1.0,
                check_alone=True):
    """Histories through packed appends, one batch call, every row against the formula in 64 bits."""
    kd, qd, T = KV * hd, H * hd, sum(nq)
    pool = Q8Pool(sum(-(-(p + n) // bs) for p, n in zip(past, nq)) + 4, layers, KV, hd, bs, max_seqs=len(past) + 1)
    layer = layers - 1
    scale = float(np.float32(hd ** -0.5))
    try:
        seqs = [pool.seq(p + n) for p, n in zip(past, nq)]
        for r, (s, p) in enumerate(zip(seqs, past)):
            if p:
                x, y = randn(p, kd, seed=seed + 10 * r), randn(p, kd, seed=seed + 10 * r + 1)
                if scales is not None:      # rows of very different sizes, so the blocks' steps differ
                    x = x * torch.exp2(torch.randint(-scales[0], 1, (p, 1), device="cuda").float())
                    y = y * torch.exp2(torch.randint(-scales[1], 1, (p, 1), device="cuda").float())
                pool.append([s], x, y, [p])
        q, x, y = randn(T, qd, seed=seed + 5) * mul, randn(T, kd, seed=seed + 6), randn(T, kd, seed=seed + 7)
        pkv.check(pkv.pkv_ensure_append_batch(seqs, nq))
        out = torch.full((T, qd), float("nan"), device="cuda")
        if host:
            ho = torch.empty(T, qd).pin_memory()
            pkv.check(pkv.pkv_attn_batch_host(seqs, nq, q.cpu().pin_memory(), x.cpu().pin_memory(),
                                              y.cpu().pin_memory(), H, KV, hd, layer, causal, scale, ho))
            out.copy_(ho)
        elif rope:
            pkv.check(pkv.pkv_attn_batch_rope(seqs, nq, q, x, y, H, KV, hd, layer, causal, scale, rope, out))
        else:
            pkv.check(pkv.pkv_attn_batch(seqs, nq, q, x, y, H, KV, hd, layer, causal, scale, out))
        pool.ok()
        at = 0
        for s, p, n in zip(seqs, past, nq):
            K, V = pool.values(s, p + n, layer)
            Q = q[at:at + n].double().view(n, KV, H // KV, hd)
            new = x[at:at + n].double()
            if rope:
                pos = np.arange(p, p + n)
                Q = torch.from_numpy(oracle.rope_neox(q[at:at + n].cpu().numpy(), pos, hd, rope)).cuda().double()
                Q = Q.float().double().view(n, KV, H // KV, hd)
                new = torch.from_numpy(oracle.rope_neox_f32(x[at:at + n].cpu().numpy(), pos, hd, rope)).cuda().double()
            # the new rows are stored, within half a step (their block may have been coarser already)
            ids = torch.tensor(pkv.pkv_seq_page_table(s), device="cuda")[torch.arange(p, p + n, device="cuda") // bs]
            step = pool.Ks[ids, layer].double()[:, :, None]
            assert bool(((K[p:] - new.view(n, KV, hd)).abs() <= step / 2).all())
            for j in range(KV):
                sc = torch.einsum("igd,jd->igj", Q[:, j], K[:, j]) * scale
                if causal:
                    lim = p + torch.arange(n, device="cuda")
                    sc = sc.masked_fill(torch.arange(p + n, device="cuda")[None, None] > lim[:, None, None], -math.inf)
                exp = torch.einsum("igj,jd->igd", torch.softmax(sc, -1), V[:, j])
                got = out[at:at + n].double().view(n, KV, H // KV, hd)[:, j]
                err = (got - exp).abs().max().item()
                tol = tolerance(V.abs().max().item())
                if mul > 1:   # large scores: f32 sums of hd products, off by up to e_s in numerator and denominator
                    es = hd * 2.0 ** -24 * scale * (Q[:, j].abs().flatten(0, 1) @ K[:, j].abs().T).max().item()
                    tol += 2 * es * V.abs().max().item()
                assert err <= tol, (err, tol, p, n, j)
            at += n
        if check_alone and len(seqs) > 1 and not host and not rope:
            # a row alone returns the same bits
            at = 0
            for s, n in zip(seqs, nq):
                one = torch.empty(n, qd, device="cuda")
                pkv.check(pkv.pkv_attn_batch([s], [n], q[at:at + n].contiguous(), x[at:at + n].contiguous(),
                                             y[at:at + n].contiguous(), H, KV, hd, layer, causal, scale, one))
                assert torch.equal(one, out[at:at + n])
                at += n
            pool.ok()
        return pkv.pkv_pool_last_work(pool.p)
    finally:
        pool.close()


@pytest.mark.parametrize("KV,hd", [(2, 128), (1, 64), (3, 96), (2, 80), (1, 32), (1, 16), (2, 20), (1, 256), (2, 112)])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode_shapes(KV, hd, G):
    attend_case(KV * G, KV, hd, 16, [0, 1, 15, 16, 17, 63, 500], [1] * 7, seed=hd + G)


@pytest.mark.parametrize("G", [3, 5, 6, 7, 12, 16, 20])
def test_decode_groups(G):
    attend_case(G, 1, 128, 16, [0, 200, 31], [1] * 3, seed=G)


@pytest.mark.parametrize("bs", [1, 2, 3, 5, 8, 32, 33, 64, 100])
def test_decode_block_sizes(bs):
    attend_case(8, 2, 128, bs, [0, 3, 32, 333, 100], [1, 1, 2, 1, 1], seed=bs)


@pytest.mark.parametrize("nq", [[2, 3, 1], [4, 4], [5, 7, 8], [16, 31]])
@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (8, 1, 64), (5, 1, 128)])
def test_short_chunks(nq, causal, H, KV, hd):
    attend_case(H, KV, hd, 16, [70, 0, 1100][:len(nq)], nq, causal=causal, seed=sum(nq))


@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("bs,causal", [(16, 1), (16, 0), (5, 1)])
def test_prefill_chunks(G, bs, causal):
    w = attend_case(2 * G, 2, 128, bs, [0, 100, 7, 2000, 63, 64, 65], [40, 64, 1, 150, 65, 64, 300], seed=G, causal=causal)
    assert w["prefill_tiles"] > 0


@pytest.mark.parametrize("G,KV,hd", [(4, 2, 64), (1, 5, 80), (4, 3, 96), (2, 1, 16), (3, 2, 32), (16, 1, 48), (7, 1, 112),
                                     (5, 2, 128), (12, 1, 128), (64, 1, 64), (1, 1, 128)])
@pytest.mark.parametrize("causal", [1, 0])
def test_prefill_head_widths_and_groups(G, KV, hd, causal):
    """Tiles whose rows are not all used, operands narrower than the images; lone and paired tiles, splits."""
    old = pkv.pkv_get_split_keys()
    try:
        w = attend_case(G * KV, KV, hd, 16, [0, 100, 7, 700, 63], [40, 64, 1, 150, 33], seed=G, causal=causal)
        assert w["prefill_tiles"] > 0
        pkv.check(pkv.pkv_set_split_keys(32))
        attend_case(G * KV, KV, hd, 5, [600, 0], [35, 45], seed=G + 1, causal=causal)
    finally:
        pkv.check(pkv.pkv_set_split_keys(old))


@pytest.mark.parametrize("scales", [(8, 0), (0, 12), (12, 12)])
def test_prefill_blocks_of_very_different_scales(scales):
    attend_case(8, 2, 128, 4, [300, 90], [70, 33], seed=3, scales=scales)


@pytest.mark.parametrize("mul", [0.0, 10.0, 100.0])
def test_prefill_score_ranges(mul):
    attend_case(8, 2, 128, 16, [300, 90], [70, 33], seed=4, mul=mul)


def test_splits_and_merge():
    """Several splits per row, at the setting's smallest size too."""
    attend_case(8, 2, 128, 16, [9000, 4096, 4095, 1], [1, 1, 3, 1], seed=1)
    old = pkv.pkv_get_split_keys()
    try:
        pkv.check(pkv.pkv_set_split_keys(32))
        attend_case(8, 2, 128, 16, [700, 129, 0, 300], [1, 1, 1, 6], seed=2)
        attend_case(4, 1, 64, 5, [700, 129], [1, 9], seed=3, causal=0)
        attend_case(3, 1, 20, 16, [700, 129], [1, 9], seed=4)
        # tensor-core rows with several splits, an odd number of records
        attend_case(8, 2, 128, 16, [1200, 129, 0], [70, 33, 40], seed=5)
        attend_case(3, 3, 128, 16, [1000, 129], [35, 33], seed=6)
        attend_case(8, 1, 128, 7, [1000, 129], [35, 61], seed=7, causal=0)
    finally:
        pkv.check(pkv.pkv_set_split_keys(old))


@pytest.mark.parametrize("rows", [20, 150, 900])
@pytest.mark.parametrize("chunk", [1, 40])
def test_few_and_many_rows(rows, chunk):
    """Descriptors that travel with the launches (two sizes) and that are uploaded, also for tensor-core rows."""
    past = [(37 * r) % 45 for r in range(rows)]
    attend_case(2, 1, 128, 16, past, [chunk] + [1 + r % 2 for r in range(1, rows)], seed=8, check_alone=rows < 50)


@pytest.mark.parametrize("rows", [20, 150, 900])
def test_packed_rows_of_few_and_many_sequences(rows):
    """The same of append and read; a row comes back within half a step of its block."""
    pool = Q8Pool(3 * rows, 1, 1, 64, 4, max_seqs=rows + 1)
    try:
        n = [1 + r % 9 for r in range(rows)]
        seqs = [pool.seq(m) for m in n]
        x, y = randn(sum(n), 64, seed=1), randn(sum(n), 64, seed=2)
        pool.append(seqs, x, y, n)
        k, v = torch.full_like(x, float("nan")), torch.full_like(y, float("nan"))
        pkv.check(pkv.pkv_read_packed(seqs, [0] * rows, n, 0, k, v))
        pool.ok()
        at = 0
        for s, m in zip(seqs, n):
            K, V = pool.values(s, m)
            assert torch.equal(k[at:at + m].double(), K[:, 0]) and torch.equal(v[at:at + m].double(), V[:, 0])
            ids = torch.tensor(pkv.pkv_seq_page_table(s), device="cuda")[torch.arange(m, device="cuda") // 4]
            assert bool(((K[:, 0] - x[at:at + m]).abs() <= pool.Ks[ids, 0] / 2).all())
            assert bool(((V[:, 0] - y[at:at + m]).abs() <= pool.Vs[ids, 0] / 2).all())
            at += m
    finally:
        pool.close()


@pytest.mark.parametrize("scales", [(6, 0), (0, 10), (10, 10)])
@pytest.mark.parametrize("bs", [1, 16])
def test_blocks_of_very_different_scales(scales, bs):
    attend_case(8, 2, 128, bs, [600, 90], [1, 3], seed=3, scales=scales)


@pytest.mark.parametrize("mul", [0.0, 10.0, 100.0])
def test_score_ranges(mul):
    attend_case(8, 2, 128, 16, [600, 90], [1, 3], seed=4, mul=mul)


def test_layers_host_buffers_and_rope():
    attend_case(8, 2, 128, 16, [100, 0], [1, 2], layers=3, seed=1)
    attend_case(8, 2, 128, 16, [100, 7], [1, 1], host=True, seed=2)
    attend_case(8, 2, 128, 16, [100, 7], [3, 40], host=True, seed=2)
    attend_case(8, 2, 128, 16, [100, 7, 33], [1, 3, 40], rope=10000.0, seed=3)
    attend_case(4, 2, 64, 5, [100, 7], [1, 3], rope=500.0, seed=4)


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (8, 2, 64), (15, 3, 96)])
def test_shared_prefix_and_image_cache(H, KV, hd):
    """Forks of one long prefix take the shared-prefix pass; its result agrees with each row's own, with and without
    cached images."""
    bs, n = 16, 20
    pool = Q8Pool(600, 1, KV, hd, bs, max_seqs=n + 2)
    try:
        a = pool.seq(2600)
        x, y = randn(2100, KV * hd, seed=1), randn(2100, KV * hd, seed=2)
        pool.append([a], x, y, [2100])
        seqs = [pkv.pkv_seq_fork(a) for _ in range(n)]
        for r, s in enumerate(seqs):
            z = randn(3 + r, KV * hd, seed=20 + r)
            pool.append([s], z, -z, [3 + r])
        ns = [1] * n
        q, x, y = (randn(n, w * hd, seed=60 + w) for w in (H, KV, KV))
        pkv.check(pkv.pkv_ensure_append_batch(seqs, ns))
        outs = []
        for cascade, cache in ((False, 0), (True, 0), (True, 1 << 27), (True, 1 << 27)):
            if cache and len(outs) == 2:
                pkv.check(pkv.pkv_pool_set_image_cache(pool.p, cache))
            pkv.pkv_set_cascade(cascade)
            o = torch.empty(n, H * hd, device="cuda")
            pkv.check(pkv.pkv_attn_batch(seqs, ns, q, x, y, H, KV, hd, 0, 1, hd ** -0.5, o))
            pool.ok()
            outs.append(o)
            w = pkv.pkv_pool_last_work(pool.p)
            assert (w["prefix_tiles"] > 0) == cascade
        assert w["image_hits"] > 0 and w["image_builds"] == 0
        vmax = pool.values(a, 2100)[1].abs().max().item()
        assert (outs[0] - outs[1]).abs().max().item() <= 2 * tolerance(vmax)
        assert torch.equal(outs[1], outs[2]) and torch.equal(outs[1], outs[3])
    finally:
        pkv.pkv_set_cascade(True)
        pool.close()


def test_pools_on_streams_of_their_own():
    """Steps of two pools issued in turn on two streams return what each returns alone."""
    H, KV, hd, bs, past = 8, 2, 128, 16, [700, 33, 5000, 64]
    nqs = [[1, 1, 1, 1], [40, 1, 3, 33], [1, 20, 1, 1], [1, 1, 1, 1]]
    kd, qd = KV * hd, H * hd

    def step(pool, seqs, i, seed):
        nq = nqs[i]
        q, x, y = (randn(sum(nq), w, seed=seed + 7 * i + j) for j, w in enumerate((qd, kd, kd)))
        torch.cuda.current_stream().synchronize()
        pkv.check(pkv.pkv_ensure_append_batch(seqs, nq))
        out = torch.empty(sum(nq), qd, device="cuda")
        pkv.check(pkv.pkv_attn_batch(seqs, nq, q, x, y, H, KV, hd, 0, 1, hd ** -0.5, out))
        pkv.check(pkv.pkv_advance_batch(seqs, nq))
        return out, (q, x, y)

    def start(seed):
        pool = Q8Pool(500, 1, KV, hd, bs)
        seqs = [pool.seq(p + 200) for p in past]
        pool.append(seqs, randn(sum(past), kd, seed=seed), randn(sum(past), kd, seed=seed + 1), past)
        torch.cuda.current_stream().synchronize()
        return pool, seqs

    alone, pools = [], []
    try:
        for k in range(2):
            pool, seqs = start(50 * k)
            pools.append(pool)
            alone.append([step(pool, seqs, i, 50 * k)[0] for i in range(len(nqs))])
            pool.ok()
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        both = []
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                both.append(start(50 * k))
                pools.append(both[-1][0])
        outs = [[], []]
        for i in range(len(nqs)):
            for k, st in enumerate(streams):
                with torch.cuda.stream(st):
                    outs[k].append(step(*both[k], i, 50 * k))
        torch.cuda.synchronize()
        for k in range(2):
            both[k][0].ok()
            for i in range(len(nqs)):
                assert torch.equal(alone[k][i], outs[k][i][0]), (k, i)
    finally:
        for p in pools:
            p.close()


def test_bad_pages_are_skipped():
    """An id outside the pool in the caller's page table cannot come from the host core; the kernels still check: rows
    past the table's end are refused before any launch."""
    pool = Q8Pool(4, 1, 1, 64, 4, max_blocks=2)
    try:
        s = pool.seq(8)
        assert pkv.pkv_ensure_append(s, 9) == pkv.PKV_ERR_CAPACITY
    finally:
        pool.close()


def test_prompt_then_decode_then_swap():
    """The operators as a server runs them: packed prompts, their K / V into the pages, decode steps, one sequence read
    out and moved to another pool, where it goes on decoding with the same output."""
    H, KV, hd, bs, lens = 8, 2, 128, 16, [45, 130, 7]
    T = sum(lens)
    pool, other = Q8Pool(80, 1, KV, hd, bs), Q8Pool(80, 1, KV, hd, bs)
    try:
        w = randn(T, (H + 2 * KV) * hd, seed=1, dtype=torch.bfloat16)
        q, k, v = w[:, :H * hd], w[:, H * hd:(H + KV) * hd], w[:, (H + KV) * hd:]
        out = torch.empty(T, H * hd, dtype=torch.bfloat16, device="cuda")
        pkv.check(pkv.pkv_attn_packed(q, k, v, lens, H, KV, hd, 1, hd ** -0.5, out, torch.cuda.current_stream()))
        seqs = [pool.seq(n + 20) for n in lens]
        pool.append(seqs, k, v, lens)
        step_in = [[randn(3, x * hd, seed=10 * i + x) for x in (H, KV, KV + 1)] for i in range(5)]
        for i in range(3):
            a, b, c = step_in[i]
            o = torch.empty(3, H * hd, device="cuda")
            pkv.check(pkv.pkv_ensure_append_batch(seqs, [1] * 3))
            pkv.check(pkv.pkv_attn_batch(seqs, [1] * 3, a, b, c[:, :KV * hd].contiguous(), H, KV, hd, 0, 1, hd ** -0.5, o))
            pkv.check(pkv.pkv_advance_batch(seqs, [1] * 3))
        n = pkv.pkv_seq_len(seqs[1])
        assert n == 133
        K, V = (torch.empty(n, KV * hd, device="cuda") for _ in range(2))
        pkv.check(pkv.pkv_read_packed([seqs[1]], [0], [n], 0, K, V))
        moved = other.seq(n + 5)
        other.append([moved], K, V, [n])
        # the prompt's values fit their blocks' steps again exactly, so the moved pages hold the same values
        for a, b in zip(pool.values(seqs[1], n), other.values(moved, n)):
            assert torch.equal(a, b)
        a, b, c = (x[1:2].contiguous() for x in step_in[3])
        c = c[:, :KV * hd].contiguous()
        outs = []
        for s in (seqs[1], moved):
            o = torch.empty(1, H * hd, device="cuda")
            pkv.check(pkv.pkv_ensure_append(s, 1))
            pkv.check(pkv.pkv_attn_batch([s], [1], a, b, c, H, KV, hd, 0, 1, hd ** -0.5, o))
            outs.append(o)
        pool.ok()
        other.ok()
        assert torch.equal(outs[0], outs[1])
        # the cached prompt against the prompt's own attention: keys off by half a step move a score by at most e_s,
        # values by half a step; the packed output has its own roundings (probabilities and output, 2^-8 each)
        o = torch.empty(1, H * hd, device="cuda")
        f = pool.seq(60)
        pool.append([f], k[:44], v[:44], [44])
        pkv.check(pkv.pkv_ensure_append(f, 1))
        pkv.check(pkv.pkv_attn_batch([f], [1], q[44:45].float().contiguous(), k[44:45].float().contiguous(),
                                     v[44:45].float().contiguous(), H, KV, hd, 0, 1, hd ** -0.5, o))
        pool.ok()
        ids = torch.tensor(pkv.pkv_seq_page_table(f), device="cuda")
        es = hd ** -0.5 * q[44].float().abs().view(H, hd).sum(-1).max().item() * pool.Ks[ids].max().item() / 2
        vmax = v[:45].float().abs().max().item()
        tol = pool.Vs[ids].max().item() / 2 + (math.exp(2 * es) - 1 + 2.0 ** -7) * vmax
        assert (o - out[44:45].float()).abs().max().item() <= tol
    finally:
        pool.close()
        other.close()

"""Operand images of 8-bit pools (tensor-core rows and shared prefixes): the
power of two of a 64-key tile comes from its largest scale, wherever that
sits, and the values against the formula in 64 bits over the stored ones.

The tolerance is the pools' own: 1e-5 max|V| + 1e-6.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from gpu_helpers import tolerance
from test_gpu_q8_pool import Q8Pool, randn

pytestmark = pytest.mark.gpu


def exact(pool, s, q, past, H, KV, hd, scale):
    """The causal formula in 64 bits over the stored values of sequence s, and those values of V."""
    n = len(q)
    K, V = pool.values(s, past + n)
    Q = q.double().view(n, KV, H // KV, hd)
    sc = torch.einsum("ikgd,jkd->kgij", Q, K) * scale
    hide = torch.arange(past + n, device="cuda")[None] > past + torch.arange(n, device="cuda")[:, None]
    p = torch.softmax(sc.masked_fill(hide, -math.inf), -1)
    return torch.einsum("kgij,jkd->ikgd", p, V).reshape(n, H * hd), V


@pytest.mark.parametrize("which", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("hd", [128, 80])
def test_largest_scale_of_a_tile_in_every_place(hd, which):
    """One key of each sequence is 64 times as large as the others, another key in each: an image scaled for the
    others would hold 127 * 2^14 there, past f16.  The row's last tile of 64 keys has 38."""
    KV, G, bs, past, n = 1, 4, 1, 70, 32
    H, T = KV * G, past + n
    pool = Q8Pool(T * T + 4, 1, KV, hd, bs, max_seqs=T + 1, max_blocks=T + 1)
    try:
        seqs = [pool.seq(T) for _ in range(T)]
        rows = [randn(T, T, KV * hd, seed=1 + i) for i in range(2)]
        for r in range(T):
            rows[which][r, r] *= 64.0
        q = randn(T * n, H * hd, seed=3) * (1.0 / 64 if which == 0 else 1.0)
        pool.append(seqs, *(x[:, :past].reshape(-1, KV * hd).contiguous() for x in rows), [past] * T)
        x, y = (x[:, past:].reshape(-1, KV * hd).contiguous() for x in rows)
        pkv.check(pkv.pkv_ensure_append_batch(seqs, [n] * T))
        out = torch.full((T * n, H * hd), float("nan"), device="cuda")
        scale = float(np.float32(hd ** -0.5))
        pkv.check(pkv.pkv_attn_batch(seqs, [n] * T, q, x, y, H, KV, hd, 0, 1, scale, out))
        pool.ok()
        assert pkv.pkv_pool_last_work(pool.p)["prefill_tiles"] > 0
        for r, s in enumerate(seqs):
            exp, V = exact(pool, s, q[r * n:(r + 1) * n], past, H, KV, hd, scale)
            top = (pool.Ks, pool.Vs)[which][pkv.pkv_seq_page_table(s), 0, 0]
            assert int(top.argmax()) == r
            err = (out[r * n:(r + 1) * n].double() - exp).abs().max().item()
            assert err <= tolerance(V.abs().max().item()), (r, err)
    finally:
        pool.close()


@pytest.mark.parametrize("which", [0, 1], ids=["k", "v"])
@pytest.mark.parametrize("spread", [13, 20, 30])
def test_blocks_far_apart_in_one_tile(which, spread):
    """Keys of one tile whose scales lie up to 2^30 apart (an image holds a factor down to 2^-24 of 2^8)."""
    KV, G, hd, bs, past, n = 2, 4, 128, 4, 150, 40
    H, T = KV * G, past + n
    pool = Q8Pool(T // bs + 4, 1, KV, hd, bs, max_seqs=2)
    try:
        s = pool.seq(T)
        rows = [randn(T, KV * hd, seed=1 + i) for i in range(2)]
        small = (torch.arange(T, device="cuda") // bs) % 2 == 0       # every other page
        rows[which][small] *= 2.0 ** -spread
        q = randn(n, H * hd, seed=3)
        pool.append([s], *(x[:past].contiguous() for x in rows), [past])
        pkv.check(pkv.pkv_ensure_append(s, n))
        out, scale = torch.empty(n, H * hd, device="cuda"), float(np.float32(hd ** -0.5))
        pkv.check(pkv.pkv_attn_batch([s], [n], q, *(x[past:].contiguous() for x in rows), H, KV, hd, 0, 1, scale, out))
        pool.ok()
        assert pkv.pkv_pool_last_work(pool.p)["prefill_tiles"] > 0
        sc = (pool.Ks, pool.Vs)[which][pkv.pkv_seq_page_table(s), 0]
        assert float(sc.max() / sc.min()) >= 2.0 ** (spread - 2)
        exp, V = exact(pool, s, q, past, H, KV, hd, scale)
        assert (out.double() - exp).abs().max().item() <= tolerance(V.abs().max().item())
    finally:
        pool.close()


@pytest.mark.parametrize("which", [0, 1], ids=["k", "v"])
def test_not_finite_scale_under_tensor_core_rows(which):
    """Queries that see the block's values are NaN in the heads of its kv head; the other kv head, the other
    sequences and the rows after a rewrite are as without it."""
    KV, G, hd, bs, n = 2, 4, 128, 16, 40
    H, past = KV * G, [150, 150, 70]
    pool = Q8Pool(60, 1, KV, hd, bs, max_seqs=4)
    try:
        scale, outs, N = float(np.float32(hd ** -0.5)), [], n * 3
        q, x, y = (randn(N, w * hd, seed=i) for i, w in enumerate((H, KV, KV)))
        seqs = [pool.seq(p + n) for p in past]
        for bad in (False, True, False):
            for r, (s, p) in enumerate(zip(seqs, past)):
                pkv.check(pkv.pkv_seq_truncate(s, 0))
                rows = [randn(p, KV * hd, seed=10 + r + i) for i in range(2)]
                if bad and r == 1:
                    rows[which][100, hd + 7] = math.inf       # kv head 1, page 6
                pool.append([s], *rows, [p])
            pkv.check(pkv.pkv_ensure_append_batch(seqs, [n] * 3))
            o = torch.empty(N, H * hd, device="cuda")
            pkv.check(pkv.pkv_attn_batch(seqs, [n] * 3, q, x, y, H, KV, hd, 0, 1, scale, o))
            pool.ok()
            assert pkv.pkv_pool_last_work(pool.p)["prefill_tiles"] > 0
            outs.append(o)
        clean, got, again = outs
        assert torch.equal(clean, again) and bool(torch.isfinite(clean).all())
        assert torch.equal(got[:n], clean[:n]) and torch.equal(got[2 * n:], clean[2 * n:])
        assert torch.equal(got[:, :G * hd], clean[:, :G * hd])
        assert bool(torch.isnan(got[n:2 * n, G * hd:]).all())
    finally:
        pool.close()


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (8, 2, 64), (15, 3, 96)])
def test_shared_prefix_in_64_bits(H, KV, hd):
    """Forks of one long prefix against the formula, the prefix's values of very different sizes among them."""
    bs, n = 16, 20
    pool = Q8Pool(600, 1, KV, hd, bs, max_seqs=n + 2)
    try:
        a = pool.seq(2600)
        x, y = randn(2100, KV * hd, seed=1), randn(2100, KV * hd, seed=2)
        y[700:900] *= 64.0
        pool.append([a], x, y, [2100])
        seqs = [pkv.pkv_seq_fork(a) for _ in range(n)]
        for r, s in enumerate(seqs):
            z = randn(3 + r, KV * hd, seed=20 + r)
            pool.append([s], z, -z, [3 + r])
        q, x, y = (randn(n, w * hd, seed=60 + w) for w in (H, KV, KV))
        pkv.check(pkv.pkv_ensure_append_batch(seqs, [1] * n))
        out, scale = torch.empty(n, H * hd, device="cuda"), float(np.float32(hd ** -0.5))
        pkv.check(pkv.pkv_attn_batch(seqs, [1] * n, q, x, y, H, KV, hd, 0, 1, scale, out))
        pool.ok()
        assert pkv.pkv_pool_last_work(pool.p)["prefix_tiles"] > 0
        for r, s in enumerate(seqs):
            exp, V = exact(pool, s, q[r:r + 1], pkv.pkv_seq_len(s), H, KV, hd, scale)
            assert (out[r:r + 1].double() - exp).abs().max().item() <= tolerance(V.abs().max().item()), r
    finally:
        pool.close()

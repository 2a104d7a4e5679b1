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

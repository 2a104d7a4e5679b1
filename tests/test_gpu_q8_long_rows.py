"""Tensor-core rows over long histories of 8-bit pools.  The tensor cores round
each f32 sum toward zero, so on values of one sign a sum that grows from 0 by N
additions (two a 16 keys) loses about N 2^-24 / 2 of itself: the row may not go
on adding to it, or 16,000 keys are 6e-5 off.  The tolerance is the pools' own,
1e-5 max|V| + 1e-6, however long the row.  Where scores are large, an f32 sum of
hd products is off by up to e_s in numerator and denominator.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from gpu_helpers import tolerance
from test_gpu_q8_pool import Q8Pool, randn

pytestmark = pytest.mark.gpu


def run(mode, past, n, KV, G, hd, bs=16, causal=1, tiles=True):
    H, T, dev = KV * G, past + n, "cuda"
    pool = Q8Pool(-(-T // bs) + 2, 1, KV, hd, bs, max_seqs=2, max_blocks=-(-T // bs))
    try:
        K, V, Q = randn(T, KV * hd, seed=1), randn(T, KV * hd, seed=2), randn(n, H * hd, seed=3)
        at = torch.arange(T, device=dev)[:, None] / T
        if mode == "one sign":
            V = 1.0 + 0.1 * V
        elif mode in ("scores rise", "scores fall"):   # by 60 along the keys, so that the maximum moves again and again
            Q[:, ::hd] = 8.0
            K[:, ::hd] = (at if mode == "scores rise" else 1 - at) * 60.0 * hd ** 0.5 / 8.0
            V = 1.0 + 0.1 * V
        elif mode == "values grow":
            V = (1.0 + 0.1 * V) * torch.exp2(torch.floor(at * 20))
        elif mode == "values shrink":
            V = (1.0 + 0.1 * V) * torch.exp2(-torch.floor(at * 20))
        s = pool.seq(T)
        pool.append([s], K[:past].contiguous(), V[:past].contiguous(), [past])
        pkv.check(pkv.pkv_ensure_append(s, n))
        out, scale = torch.full((n, H * hd), float("nan"), device=dev), float(np.float32(hd ** -0.5))
        pkv.check(pkv.pkv_attn_batch([s], [n], Q, K[past:].contiguous(), V[past:].contiguous(), H, KV, hd, 0, causal,
                                     scale, out))
        pool.ok()
        assert (pkv.pkv_pool_last_work(pool.p)["prefill_tiles"] > 0) == tiles
        K, V = pool.values(s, T)
        hide = torch.arange(T, device=dev)[None] > past + torch.arange(n, device=dev)[:, None]
        for j in range(KV):
            q = Q.double().view(n, KV, G, hd)[:, j]
            sc = torch.einsum("igd,jd->igj", q, K[:, j]) * scale
            if causal:
                sc = sc.masked_fill(hide[:, None], -math.inf)
            exp = torch.einsum("igj,jd->igd", torch.softmax(sc, -1), V[:, j])
            err = (out.double().view(n, KV, G, hd)[:, j] - exp).abs().max().item()
            tol = tolerance(V.abs().max().item())
            if "scores" in mode:
                es = hd * 2.0 ** -24 * scale * (q.abs().flatten(0, 1) @ K[:, j].abs().T).max().item()
                tol += 2 * es * V.abs().max().item()
            assert err <= tol, (mode, j, err, tol)
    finally:
        pool.close()


@pytest.mark.parametrize("past", [1000, 1472, 1473, 1535, 1536, 2100, 3100, 16000, 40000])
def test_values_of_one_sign(past):
    run("one sign", past, 64, 2, 4, 128)


@pytest.mark.parametrize("mode", ["one sign", "scores rise", "scores fall", "values grow", "values shrink"])
# pairs of tiles, a lone tile, a group that leaves rows unused, narrow heads, splits of one row
@pytest.mark.parametrize("n,KV,G,hd", [(64, 2, 4, 128), (32, 1, 4, 128), (45, 1, 5, 128), (70, 2, 2, 64), (33, 1, 8, 80)])
def test_sums_set_aside(mode, n, KV, G, hd):
    run(mode, 5000, n, KV, G, hd)


def test_all_keys_seen_and_odd_pages():
    run("one sign", 4000, 200, 1, 4, 128, causal=0)
    run("values grow", 3001, 65, 1, 1, 96, bs=5)


def test_splits_of_a_row():
    """Records of splits that set sums aside: 16 x 128 keys a split."""
    old = pkv.pkv_get_split_keys()
    try:
        pkv.check(pkv.pkv_set_split_keys(128))      # splits of 2,048
        run("values shrink", 5000, 40, 1, 4, 128)
        run("scores rise", 5000, 40, 3, 1, 128)
    finally:
        pkv.check(pkv.pkv_set_split_keys(old))


@pytest.mark.parametrize("keys", [32, 1024, 4096, 65536])
@pytest.mark.parametrize("n", [1, 4])
def test_decode_units_of_any_split_setting(keys, n):
    """A decode unit's sums are no longer than its pools' tolerance allows, however many keys a split is set to take."""
    old = pkv.pkv_get_split_keys()
    try:
        pkv.check(pkv.pkv_set_split_keys(keys))
        for KV, G, hd in [(2, 4, 128), (1, 1, 64), (1, 5, 96)]:
            run("one sign", 60000, n, KV, G, hd, tiles=False)
    finally:
        pkv.check(pkv.pkv_set_split_keys(old))

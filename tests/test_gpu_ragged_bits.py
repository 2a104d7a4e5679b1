"""How many bits of the probabilities meet V in cross and shared-prefix attention, where a call says that they keep 16.

Queries and keys are -1, 0 or 1, so that every score is a whole number below 2^9, which f32 holds exactly.  Off the
tensor-core tiles an element of the output is then off by at most (u: half a step of the type)
  u |o|            the output rounded once
  u^2 A            probabilities in two pieces of the type; in f16 a piece is off by 2^-25 at least, which adds
                   2^-25 sum_j |v_j| over the sum of the probabilities (the largest is 1 or more)
  2 e A            with e = 5 X 2^-24 + 2^-22, in numerator and denominator: a scaled score (of size X at most) has three
                   roundings, of the scale, its log2(e) and the product, its difference from the reference (2 X at most) one,
                   and 2^x is good to 2^-22
  (n / 16 + 150) 2^-24 A   a rounding for every sixteen of the n keys, a few in each product of sixteen, a join of up to
                   128 records
  2^-21 A          eight more: the weights of the parts and records, their sums, one division
with A = sum_j p_j |v_j|.  A probability rounded to the type would add u A: outputs of random values, whose terms
cancel, show it.
"""
import math

import pytest
import torch

from ragged_helpers import U, Case

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])


def case(*a, **kw):
    c = Case(*a, **kw)
    for x in (c.q, c.k, c.kp):
        if x is not None:
            x.copy_((x.float() * 1.2).round().clamp(-1, 1))
    return c


def beyond(c, got, scale=None):
    """Elements past the bound."""
    H, KV, hd, u = c.H, c.KV, c.hd, U[c.dtype]
    G, scale, at = H // KV, hd ** -0.5 if scale is None else scale, 0
    past = torch.zeros(sum(c.ql), H, hd, dtype=torch.bool, device="cuda")
    for n, m, k0 in zip(c.ql, c.kl, c.start):
        K, V = (x[k0:k0 + m].double().view(m, KV, hd) for x in (c.k, c.v))
        seen = torch.full((n,), m, device="cuda")
        if c.prefix is not None:
            K, V = (torch.cat([p.double().view(-1, KV, hd), x]) for p, x in ((c.kp, K), (c.vp, V)))
            seen = c.prefix + m - n + 1 + torch.arange(n, device="cuda")
        s, at = slice(at, at + n), at + n
        if n == 0:
            continue
        hide = (torch.arange(len(K), device="cuda")[None, :] >= seen[:, None])[:, None, None]
        Q = c.q[s].double().view(n, KV, G, hd)
        x = (torch.einsum("iagd,jad->iagj", Q, K) * scale).masked_fill(hide, -math.inf)
        p = torch.softmax(x, dim=-1) if len(K) else x
        o, A = (torch.einsum("iagj,jad->iagd", p, y) for y in (V, V.abs()))
        X = x.masked_fill(hide, 0.0).abs().amax(-1, keepdim=True) if len(K) else 0.0
        tol = u * o.abs() + A * (u * u + 2 * (5 * X * 2.0 ** -24 + 2.0 ** -22) + (len(K) / 16 + 150) * 2.0 ** -24 + 2.0 ** -21)
        if c.dtype == F16 and len(K):
            tol = tol + 2.0 ** -25 * p.amax(-1, keepdim=True) * V.abs().sum(0)[None, :, None]
        past[s] = ~((got[s].double().view(n, KV, G, hd) - o).abs() <= tol).view(n, H, hd)
    return past


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (3, 3, 64), (16, 1, 128), (12, 12, 80), (4, 2, 24), (4, 2, 160), (2, 1, 256), (4, 2, 20)])
@DTYPES
def test_cross_calls_of_few_queries(H, KV, hd, dtype):
    """No sequence with 24 (query, head of a kv head) pairs."""
    few = 23 // (H // KV)
    for ql, kl in (([1, 1, 1], [500, 33, 3000]), ([few, 1, 0, few], [700, 20, 5, 129]), ([1], [9000]), ([1] * 70, list(range(1, 71)))):
        c = case(ql, kl, H, KV, hd, dtype, seed=hd)
        for w in ("full", None):
            assert not bool(beyond(c, c.call(workspace=w)).any())


@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (3, 3, 64), (4, 2, 160)])
@DTYPES
def test_one_sequence_of_few_queries_behind_a_prefix(H, KV, hd, dtype):
    few = 23 // (H // KV)
    for ql, kl, prefix in (([1], [1], 900), ([few], [few + 70], 3000), ([1], [2000], 60)):
        c = case(ql, kl, H, KV, hd, dtype, prefix=prefix, seed=hd)
        assert not bool(beyond(c, c.call()).any())


@pytest.mark.parametrize("prefix", [None, 300])
@DTYPES
def test_rows_and_scales_that_no_tile_takes(prefix, dtype):
    ql, kl = [90, 1, 40], [400, 30, 41]
    c = case(ql, kl, 4, 2, 20, dtype, prefix=prefix)  # heads of 40 bytes
    assert not bool(beyond(c, c.call()).any())
    c = case(ql, kl, 4, 2, 64, dtype, prefix=prefix)
    assert not bool(beyond(c, c.call(scale=-0.125), scale=-0.125).any())
    wide = torch.zeros(c.q.shape[0], c.q.shape[1] + 4, dtype=dtype, device="cuda")  # rows of Q off 16-byte boundaries
    wide[:, 4:].copy_(c.q)
    c.q = wide[:, 4:]
    assert not bool(beyond(c, c.call()).any())


def test_the_bound_tells_rounded_probabilities_apart():
    """Tiles round them: a prompt's rows, and a token's beside it, lie past this bound and within ragged_helpers'."""
    c = case([70, 1], [600, 600], 8, 2, 128, BF16)
    past = beyond(c, c.check())
    assert bool(past[:70].any()) and bool(past[70:].any())

"""pkv_rope_packed against the formula in 64 bits, and its inverse as the gradient.

Tolerance of an output y = x0 cos - x1 sin (or x0 sin + x1 cos): half a step of the type, u |y|, and
(|x0| + |x1|) e with e = 2^-21 + |p| 2^-51: cosine and sine are within 2^-22 (the angle's rest rounded to f32, at most
pi/4 2^-24, and two last places of the f32 sine), two products' and a sum's f32 roundings add 2^-23, and the angle itself is off
by 2^-53 of its size in the plain form and, here, by up to 2^-51 of it at the pairs between two powers, whose
frequencies have fallen below 3/4.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from ragged_helpers import Case

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}
BLOCKS, TURNS, AXIAL = pkv.PKV_ROPE_BLOCKS, pkv.PKV_ROPE_TURNS, pkv.PKV_ROPE_AXIAL


def pairs_of(order, pairs):
    """(axis, exponent) of every pair, by the definition."""
    out, left = [], list(pairs)
    if order == TURNS:
        for i in range(sum(pairs)):
            a = i % len(pairs)
            out.append((a if i < len(pairs) * pairs[a] else 0, i / sum(pairs)))
        return out
    for a, n in enumerate(pairs):
        for j in range(n):
            out.append((a, j / n if order == AXIAL else len(out) / sum(pairs)))
    return out


def plain(x, pos, pairs, order, hd, base, inverse=False):
    """(outputs, tolerance without u) of rows x in 64 bits."""
    r = sum(pairs)
    pos = pos.double()
    ang = torch.stack([pos[a] * base ** -e for a, e in pairs_of(order, pairs)], dim=1)
    far = torch.stack([pos[a].abs() for a, _ in pairs_of(order, pairs)], dim=1)[:, None]
    c, s = ang.cos()[:, None], (-ang if inverse else ang).sin()[:, None]
    h = x.double().reshape(x.shape[0], -1, hd)
    a, b = h[..., :r], h[..., r:2 * r]
    y, tol = h.clone(), torch.zeros_like(h)
    y[..., :r], y[..., r:2 * r] = a * c - b * s, a * s + b * c
    tol[..., :r] = tol[..., r:2 * r] = (a.abs() + b.abs()) * (2.0 ** -21 + far * 2.0 ** -51)
    return y.view(x.shape), tol.view(x.shape)


def rows(n, w, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, w, device="cuda", generator=g).to(dtype)


def positions(axes, n, hi, seed=0, lo=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(lo, hi, (axes, n), device="cuda", generator=g, dtype=torch.int64).to(torch.int32)


def close(got, exp, tol):
    half = U[got.dtype] * exp.abs()
    if got.dtype == F16:  # below f16's least normal value, 2^-14, steps no longer shrink: 2^-24 each
        half = half.clamp_min(2.0 ** -25)
    bad = ~((got.double() - exp).abs() <= tol + half)
    assert not bool(bad.any()), (int(bad.sum()), float((got.double() - exp).abs().max()), bad.nonzero()[:4].tolist())


SHAPES = [(BLOCKS, [16, 24, 24], 32, 8, 128), (TURNS, [24, 20, 20], 4, 2, 128), (AXIAL, [20, 20], 3, 3, 80),
          (AXIAL, [10, 10, 12], 2, 1, 64), (BLOCKS, [64], 5, 1, 128), (AXIAL, [18, 18], 2, 2, 72), (BLOCKS, [1, 0, 2], 3, 1, 7),
          (TURNS, [3, 3, 2], 2, 2, 40), (BLOCKS, [32, 32, 32, 32], 2, 1, 256), (BLOCKS, [8, 8], 2, 1, 100)]


@pytest.mark.parametrize("order,pairs,H,KV,hd", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 5, 2001])
@pytest.mark.parametrize("inverse", [False, True])
def test_orders_widths_and_rows(order, pairs, H, KV, hd, dtype, n, inverse):
    q, k, pos = rows(n, H * hd, dtype, 1), rows(n, KV * hd, dtype, 2), positions(len(pairs), n, 5000, n)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    pkv.check(pkv.pkv_rope_packed(q, k, pos, pairs, order, H, KV, hd, 1e4, qo, ko, inverse, torch.cuda.current_stream()))
    close(qo, *plain(q, pos, pairs, order, hd, 1e4, inverse))
    close(ko, *plain(k, pos, pairs, order, hd, 1e4, inverse))


@pytest.mark.parametrize("lo,hi", [(0, 2 ** 31 - 1), (-2 ** 31, 0), (-100, 100), (900_000, 1_100_000)])
def test_far_and_negative_positions(lo, hi):
    q, pos = rows(300, 4 * 128, F32, 1), positions(3, 300, hi, 3, lo)
    out = torch.empty_like(q)
    pkv.check(pkv.pkv_rope_packed(q, None, pos, [16, 24, 24], BLOCKS, 4, 0, 128, 1e6, out, None))
    close(out, *plain(q, pos, [16, 24, 24], BLOCKS, 128, 1e6))


@pytest.mark.parametrize("shift", [0, 8, 4, 1])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_columns_of_wider_rows_in_place_and_one_part_alone(shift, dtype):
    H, KV, hd, pairs, n = 4, 2, 64, [12, 10, 10], 333
    x = rows(n + 3, (H + KV) * hd + 40 + shift, dtype, 3)
    keep = x.clone()
    q, k = x[:n, shift + 8:shift + 8 + H * hd], x[:n, shift + 24 + H * hd:][:, :KV * hd]
    pos = positions(3, n + 5, 700)[:, :n]
    eq, ek = plain(q, pos, pairs, TURNS, hd, 1e5), plain(k, pos, pairs, TURNS, hd, 1e5)
    ko = torch.empty(n, KV * hd, dtype=dtype, device="cuda")
    pkv.check(pkv.pkv_rope_packed(None, k, pos, pairs, TURNS, 0, KV, hd, 1e5, None, ko))
    close(ko, *ek)
    pkv.check(pkv.pkv_rope_packed(q, k, pos, pairs, TURNS, H, KV, hd, 1e5, q, k))
    close(q, *eq)
    close(k, *ek)
    q.copy_(keep[:n, shift + 8:shift + 8 + H * hd])
    k.copy_(keep[:n, shift + 24 + H * hd:][:, :KV * hd])
    assert torch.equal(x, keep)  # nothing beside the rows was touched


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_inverse_is_the_gradient(dtype):
    """Against autograd on the plain form, and against differences of the call itself (linear: any step will do)."""
    H, hd, pairs, n = 3, 80, [20, 20], 57
    q, g, pos = rows(n, H * hd, dtype, 1), rows(n, H * hd, dtype, 2), positions(2, n, 90)
    back = torch.empty_like(q)
    pkv.check(pkv.pkv_rope_packed(g, None, pos, pairs, AXIAL, H, 0, hd, 1e4, back, None, inverse=True))
    leaf = q.double().requires_grad_()
    (plain(leaf, pos, pairs, AXIAL, hd, 1e4)[0] * g.double()).sum().backward()
    close(back, leaf.grad, plain(g, pos, pairs, AXIAL, hd, 1e4, True)[1])
    if dtype == F32:
        d = rows(n, H * hd, F32, 4)
        up, down = torch.empty_like(q), torch.empty_like(q)
        for x, y in ((q + d, up), (q - d, down)):
            pkv.check(pkv.pkv_rope_packed(x, None, pos, pairs, AXIAL, H, 0, hd, 1e4, y, None))
        left = ((up.double() - down.double()) / 2 * g.double()).sum()
        right = (back.double() * d.double()).sum()
        # each of the 2 * n * H * hd terms off by at most 2^-20 of sizes below 40
        assert abs(float(left - right)) < 2 * n * H * hd * 40 * 2.0 ** -20


def test_captured_and_on_another_stream():
    q, pos = rows(100, 256, BF16, 1), positions(3, 100, 800)
    out, s = torch.empty_like(q), torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.check(pkv.pkv_rope_packed(q, None, pos, [16, 24, 24], BLOCKS, 2, 0, 128, 1e4, out, None, stream=s))
    s.synchronize()
    close(out, *plain(q, pos, [16, 24, 24], BLOCKS, 128, 1e4))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.check(pkv.pkv_rope_packed(q, None, pos, [16, 24, 24], BLOCKS, 2, 0, 128, 1e4, out, None,
                                      stream=torch.cuda.current_stream()))
    q.copy_(rows(100, 256, BF16, 5))
    pos.copy_(positions(3, 100, 80_000, 6))
    g.replay()
    close(out, *plain(q, pos, [16, 24, 24], BLOCKS, 128, 1e4))


def test_one_axis_agrees_with_the_paged_append():
    """The same rotation as pkv_attn_batch_rope's: the keys that it leaves in an f32 pool."""
    n, KV, hd, base = 40, 2, 64, 1e4
    k, v, q = rows(n, KV * hd, F32, 1), rows(n, KV * hd, F32, 2), rows(n, 4 * hd, F32, 3)
    stream = torch.cuda.current_stream()
    pool = pkv.pkv_pool_new(8, 1, KV * hd, 16, None, None, 2, 8, stream)
    try:
        s = pkv.pkv_seq_new(pool, 64)
        pkv.check(pkv.pkv_ensure_append(s, n))
        out = torch.empty_like(q)
        pkv.check(pkv.pkv_attn_batch_rope([s], [n], q, k, v, 4, KV, hd, 0, 1, 0.125, base, out))
        pkv.check(pkv.pkv_advance(s, n))
        ks, vs = torch.empty_like(k), torch.empty_like(v)
        pkv.check(pkv.pkv_read_packed([s], [0], [n], 0, ks, vs))
        pkv.check(pkv.pkv_sync_error(pool))
    finally:
        torch.cuda.synchronize()
        pkv.pkv_pool_free(pool)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    ko = torch.empty_like(k)
    pkv.check(pkv.pkv_rope_packed(None, k, pos, [hd // 2], BLOCKS, 0, KV, hd, base, None, ko))
    exp, tol = plain(k, pos, [hd // 2], BLOCKS, hd, base)
    close(ko, exp, tol)
    assert bool(((ko.double() - ks.double()).abs() <= 2 * tol + 2 * U[F32] * exp.abs()).all())


def test_a_layer_of_a_multimodal_step():
    """Turned queries and keys of users' image-and-text prompts behind a shared system prompt, attention over both, then over an
    encoder's states, as a server runs them; gradient of the rotation at the end."""
    H, KV, hd, P, ql = 8, 2, 128, 300, [70, 1, 33]
    pairs, base, n = [16, 24, 24], 1e6, sum([70, 1, 33])
    c = Case(ql, ql, H, KV, hd, BF16, prefix=P, seed=4)
    pos, ppos = positions(3, n, 900, 5), positions(3, P, 300, 6)
    qr, kr, kpr = torch.empty_like(c.q), torch.empty_like(c.k), torch.empty_like(c.kp)
    pkv.check(pkv.pkv_rope_packed(c.q, c.k, pos, pairs, BLOCKS, H, KV, hd, base, qr, kr))
    pkv.check(pkv.pkv_rope_packed(None, c.kp, ppos, pairs, BLOCKS, 0, KV, hd, base, None, kpr))
    close(qr, *plain(c.q, pos, pairs, BLOCKS, hd, base))
    close(kpr, *plain(c.kp, ppos, pairs, BLOCKS, hd, base))
    c.q, c.k, c.kp = qr, kr, kpr
    own = c.check()
    x = Case(ql, [500, 0, 1201], H, KV, hd, BF16, seed=7)
    x.q = own
    x.check()
    back = torch.empty_like(own)
    pkv.check(pkv.pkv_rope_packed(own, None, pos, pairs, BLOCKS, H, 0, hd, base, back, None, inverse=True))
    close(back, *plain(own, pos, pairs, BLOCKS, hd, base, True))

"""pkv_attn_packed: attention over whole prompts packed behind one another.

The plain implementation is the softmax formula in 64 bits, sequence by
sequence.  The tolerance of an output element counts the kernels' roundings
(u: half a step of the type, 2^-8 for bf16 and 2^-11 for f16):
  u * A       every probability rounded to the type before it meets V
  u * |o|     the output rounded once (|o| <= A)
  2 e_s * A   scores off by e_s = (hd + 4) 2^-23 scale max_j sum_d |q_d k_jd| (f32 sums of exact
              products; the 4 for scaling and 2^x), in numerator and denominator
  n 2^-24 max|v|   probabilities below the type's normal range, off by at most 2^-25 (f16) each,
              relative to a sum of at least 1, and the f32 sum of n terms
with A = sum_j p_j |v_j|, computed in 64 bits.
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def plain(q, k, v, lens, H, KV, hd, causal, scale):
    """(outputs, tolerance) in 64 bits, without the type's u."""
    T = sum(lens)
    out = torch.zeros(T, H, hd, dtype=torch.float64, device="cuda")
    A = torch.zeros_like(out)
    es = torch.zeros(T, H, 1, dtype=torch.float64, device="cuda")
    tail = torch.zeros(T, 1, 1, dtype=torch.float64, device="cuda")
    at, G = 0, H // KV
    for n in lens:
        if n == 0:
            continue
        s = slice(at, at + n)
        Q = q[s].double().view(n, KV, G, hd)
        K, V = k[s].double().view(n, KV, hd), v[s].double().view(n, KV, hd)
        x = torch.einsum("ikgd,jkd->kgij", Q, K) * scale
        w = torch.einsum("ikgd,jkd->kgij", Q.abs(), K.abs()) * abs(scale)
        if causal:
            hide = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            x = x.masked_fill(hide, -math.inf)
            w = w.masked_fill(hide, 0.0)
        p = torch.softmax(x, dim=-1)
        out[s] = torch.einsum("kgij,jkd->ikgd", p, V).reshape(n, H, hd)
        A[s] = torch.einsum("kgij,jkd->ikgd", p, V.abs()).reshape(n, H, hd)
        es[s] = (hd + 4) * 2.0 ** -23 * w.amax(-1).permute(2, 0, 1).reshape(n, H, 1)
        tail[s] = n * 2.0 ** -24 * V.abs().max()
        at += n
    return out.view(T, -1), lambda u: (A * (2 * u + 2 * es) + tail).view(T, -1)


def make(lens, H, KV, hd, dtype, seed=0, fused=False, mul=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, qd, kd = sum(lens), H * hd, KV * hd
    x = torch.randn(T, qd + 2 * kd, device="cuda", generator=g)
    x[:, :qd] *= mul
    x = x.to(dtype)
    parts = x[:, :qd], x[:, qd:qd + kd], x[:, qd + kd:]
    return parts if fused else tuple(p.contiguous() for p in parts)


def attend(q, k, v, lens, H, KV, hd, causal=True, scale=None, out=None, stream=None):
    scale = hd ** -0.5 if scale is None else scale
    if out is None:
        out = torch.full((q.shape[0], H * hd), float("nan"), dtype=q.dtype, device="cuda")
    s = stream if stream is not None else torch.cuda.current_stream()
    pkv.check(pkv.pkv_attn_packed(q, k, v, lens, H, KV, hd, int(causal), scale, out, s))
    return out


def check(q, k, v, lens, H, KV, hd, causal=True, scale=None):
    got = attend(q, k, v, lens, H, KV, hd, causal, scale)
    assert pkv.pkv_contiguous_sync_error(torch.cuda.current_stream()) == pkv.PKV_OK, pkv.pkv_last_error()
    exp, tol = plain(q, k, v, lens, H, KV, hd, causal, hd ** -0.5 if scale is None else scale)
    T = sum(lens)
    err = (got[:T].double() - exp).abs()
    bad = err > tol(U[q.dtype])
    assert not bool(bad.any()) and bool(torch.isfinite(got[:T].double()).all()), (
        int(bad.sum()), float(err.max()), bad.nonzero()[:4].tolist())
    return got


LENS = [[1], [5, 0, 1, 130], [127, 128, 129], [257, 1, 255, 64, 33], [700], [0, 0, 3, 0]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (3, 3, 64)])
def test_lengths(lens, causal, dtype, H, KV, hd):
    check(*make(lens, H, KV, hd, dtype), lens, H, KV, hd, causal)


@pytest.mark.parametrize("H,KV,hd", [
    (4, 4, 128), (16, 2, 128), (16, 1, 128), (7, 1, 128), (6, 2, 96), (10, 2, 80), (12, 4, 64), (5, 1, 64), (4, 2, 32),
    (4, 1, 16), (2, 1, 8), (32, 1, 64), (64, 2, 128), (6, 3, 72),
    (4, 2, 20), (3, 1, 33), (2, 1, 1), (4, 1, 160), (2, 2, 256)])
def test_heads_and_widths(H, KV, hd):
    lens = [300, 17, 131]
    check(*make(lens, H, KV, hd, torch.bfloat16, seed=hd), lens, H, KV, hd)
    check(*make(lens, H, KV, hd, torch.float16, seed=hd + 1, fused=True), lens, H, KV, hd, causal=False)


@pytest.mark.parametrize("hd", [20, 60, 131, 136, 160, 192, 200, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_widths_off_the_tensor_core_tiles(hd, causal, dtype):
    lens = [1, 31, 32, 33, 64, 65, 129]
    check(*make(lens, 4, 2, hd, dtype), lens, 4, 2, hd, causal)


@pytest.mark.parametrize("hd,shift", [(128, 0), (128, 8), (128, 1), (64, 3), (40, 8)])
def test_strides_and_alignment(hd, shift):
    """Columns of wider rows; shift 1 and 3 leave the 16-byte boundaries."""
    H, KV, lens = 4, 2, [200, 61]
    qd, kd = H * hd, KV * hd
    x = torch.randn(sum(lens), qd + 2 * kd + 3 * 16 + shift, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, shift:shift + qd], x[:, shift + qd + 16:shift + qd + 16 + kd], x[:, shift + qd + 32 + kd:][:, :kd]
    wide = torch.full((sum(lens) + 3, qd + 24 + shift), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, shift + 8:shift + 8 + qd]
    attend(q, k, v, lens, H, KV, hd, out=out)
    torch.cuda.synchronize()
    exp, tol = plain(q, k, v, lens, H, KV, hd, True, hd ** -0.5)
    assert bool(((out[:sum(lens)].double() - exp).abs() <= tol(U[torch.bfloat16])).all())
    # rows behind the last sequence and the columns beside the output stay as they were
    assert bool((wide[sum(lens):] == 7).all())
    assert bool((wide[:, :shift + 8] == 7).all()) and bool((wide[:, shift + 8 + qd:] == 7).all())


@pytest.mark.parametrize("hd", [128, 64, 20, 160, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("causal", [True, False])
def test_values_that_are_not_finite_stay_where_they_are_seen(hd, bad, causal):
    """A poisoned K or V row reaches the queries that see it and nobody else."""
    H, KV, lens = 4, 2, [150, 200, 90]
    q, k, v = make(lens, H, KV, hd, torch.bfloat16, seed=9)
    clean = attend(q, k, v, lens, H, KV, hd, causal)
    for which in (0, 1):
        k2, v2 = k.clone(), v.clone()
        (k2, v2)[which][150 + 70, 3] = bad     # row 70 of the middle sequence, kv head 0
        got = attend(q, k2, v2, lens, H, KV, hd, causal)
        torch.cuda.synchronize()
        first = 150 + 70 if causal else 150
        keep = torch.ones(440, dtype=torch.bool, device="cuda")
        keep[first:350] = False
        assert torch.equal(got[keep], clean[keep])
        assert torch.equal(got[:, 2 * hd:], clean[:, 2 * hd:])  # the other kv head's query heads
        seen = got[first:350, :2 * hd].double()
        if which == 1:      # column 3 of both query heads is bad, the others are untouched
            exp = torch.full_like(seen[:, 3], bad)
            for c in (3, hd + 3):
                assert bool((torch.isnan(seen[:, c]) if math.isnan(bad) else
                             (seen[:, c] == exp) | torch.isnan(seen[:, c])).all())
                seen[:, c] = 0
            ref = clean[first:350, :2 * hd].double()
            ref[:, 3] = 0
            ref[:, hd + 3] = 0
            assert torch.allclose(seen, ref, rtol=0, atol=2.0 ** -6 * 5)
        elif math.isnan(bad):
            assert bool(torch.isnan(seen).all())


def test_not_finite_everywhere_in_v():
    """Every value NaN: every output is NaN, and the neighbours are not touched."""
    H, KV, hd, lens = 4, 1, 128, [300, 300, 40]
    q, k, v = make(lens, H, KV, hd, torch.float16, seed=4)
    clean = attend(q, k, v, lens, H, KV, hd)
    v2 = v.clone()
    v2[300:600] = float("nan")
    got = attend(q, k, v2, lens, H, KV, hd)
    torch.cuda.synchronize()
    assert bool(torch.isnan(got[300:600]).all())
    assert torch.equal(got[:300], clean[:300]) and torch.equal(got[600:], clean[600:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("mul", [0.0, 8.0, 40.0])
def test_score_ranges(dtype, mul):
    """Flat, peaked and nearly one-hot probabilities."""
    H, KV, hd, lens = 4, 2, 128, [513, 200]
    check(*make(lens, H, KV, hd, dtype, seed=3, mul=mul), lens, H, KV, hd)


@pytest.mark.parametrize("hd", [128, 64])
@pytest.mark.parametrize("slope", [0.05, 1.0, -1.0])
def test_running_maximum(hd, slope):
    """Scores that rise (or fall) along the keys, so the maximum moves tile after tile."""
    n, H, KV = 900, 2, 1
    q = torch.randn(n, H * hd, device="cuda") * 0.1
    k = torch.randn(n, KV * hd, device="cuda") * 0.1
    q[:, ::hd] = 8.0
    k[:, 0] = torch.arange(n, device="cuda") * slope * hd ** 0.5 / 8.0
    v = torch.randn(n, KV * hd, device="cuda")
    check(*(x.to(torch.float16) for x in (q, k, v)), [n], H, KV, hd)


def test_many_sequences():
    """More sequences than one launch takes, zero lengths among them."""
    rng = np.random.RandomState(1)
    lens = [int(x) for x in rng.randint(0, 4, size=5000)]
    check(*make(lens, 2, 1, 64, torch.bfloat16), lens, 2, 1, 64)


def test_same_inputs_same_bits_and_alone():
    """A sequence's rows do not depend on what else is in the batch."""
    H, KV, hd, lens = 8, 2, 128, [333, 1, 129, 800]
    q, k, v = make(lens, H, KV, hd, torch.bfloat16, seed=12)
    a, b = attend(q, k, v, lens, H, KV, hd), attend(q, k, v, lens, H, KV, hd)
    assert torch.equal(a, b)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        assert torch.equal(attend(q[s], k[s], v[s], [n], H, KV, hd), a[s])
        at += n


def test_other_stream_and_graphs():
    """On a side stream; captured twice and replayed in turn on new inputs."""
    H, KV, hd, lens = 8, 2, 128, [300, 77]
    q, k, v = make(lens, H, KV, hd, torch.bfloat16, seed=2)
    exp = attend(q, k, v, lens, H, KV, hd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = torch.zeros_like(exp)
    side.wait_stream(torch.cuda.current_stream())
    attend(q, k, v, lens, H, KV, hd, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, exp)
    graphs, outs = [], []
    for _ in range(2):
        o, g = torch.zeros_like(exp), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(q, k, v, lens, H, KV, hd, out=o)
        graphs.append(g)
        outs.append(o)
    q2, k2, v2 = make(lens, H, KV, hd, torch.bfloat16, seed=5)
    exp2 = attend(q2, k2, v2, lens, H, KV, hd)
    for dst, src in ((q, q2), (k, k2), (v, v2)):
        dst.copy_(src)
    for i in (0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], exp2)


def test_binding_refuses():
    q, k, v = make([4], 2, 1, 16, torch.bfloat16)
    o = torch.empty_like(q)
    for bad in ((q.float(), k, v, o), (q, k.half(), v, o), (q, k, v, o[:, :16]), (q[:3], k, v, o), (q, k, v, o.cpu())):
        with pytest.raises(TypeError):
            pkv.pkv_attn_packed(bad[0], bad[1], bad[2], [4], 2, 1, 16, 1, 0.25, bad[3])

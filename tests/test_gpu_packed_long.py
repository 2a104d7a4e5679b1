"""Packed prompts of tens of thousands of tokens.

The tensor cores round each f32 sum toward zero, so on values of one sign a sum
loses steadily: 7e-9 of itself a key, f16's half step (u = 2^-11) after 70,000.
The mean of the outputs' errors, in which their own roundings cancel, has to
stay below u / 4 at any length; single outputs keep the tolerance of shorter
prompts (test_gpu_packed.py) on the rows compared.
"""
import math

import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from test_gpu_packed import U, attend, make

pytestmark = pytest.mark.gpu


def exact(q, k, v, rows, H, KV, hd, causal):
    """The formula in 64 bits for some rows of one prompt: outputs, sum_j p_j |v_j|, and the scores' error."""
    G, scale = H // KV, hd ** -0.5
    Q = q[rows].double().view(-1, KV, G, hd)
    K, V = k.double().view(-1, KV, hd), v.double().view(-1, KV, hd)
    out, A, es = [], [], []
    for j in range(KV):
        x = torch.einsum("igd,jd->gij", Q[:, j], K[:, j]) * scale
        if causal:
            hide = torch.arange(len(K), device=q.device)[None] > rows[:, None]
            x = x.masked_fill(hide, -math.inf)
        p = torch.softmax(x, -1)
        out.append(torch.einsum("gij,jd->igd", p, V[:, j]))
        A.append(torch.einsum("gij,jd->igd", p, V[:, j].abs()))
        w = torch.einsum("igd,jd->gij", Q[:, j].abs(), K[:, j].abs()).amax(-1) * scale
        es.append(((hd + 4) * 2.0 ** -23 * w).t()[:, :, None])
    es = [t.expand(-1, -1, hd) for t in es]
    return tuple(torch.cat(t, 1).reshape(len(rows), H * hd) for t in (out, A, es))


@pytest.mark.parametrize("hd", [128, 96, 64, 160])
@pytest.mark.parametrize("n,causal", [(40000, True), (17000, False)])
def test_values_of_one_sign(hd, n, causal):
    H, KV, dt = 2, 1, torch.float16
    q, k, v = make([n], H, KV, hd, dt, seed=hd)
    v = (1.0 + 0.1 * v.float()).to(dt)
    got = attend(q, k, v, [n], H, KV, hd, causal)
    assert pkv.pkv_contiguous_sync_error(torch.cuda.current_stream()) == pkv.PKV_OK
    rows = torch.arange(n - 128, n, device="cuda")
    exp, _, _ = exact(q, k, v, rows, H, KV, hd, causal)
    assert abs(((got[rows].double() - exp) / exp).mean().item()) <= U[dt] / 4


@pytest.mark.parametrize("hd", [128, 64, 160])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("slope", [60.0, -60.0, 0.0])
def test_maximum_moves_along_a_long_prompt(hd, dtype, slope):
    """Scores that rise or fall by 60 along the keys, or stay; several heads of two kv heads."""
    n, H, KV = 20000, 4, 2
    q, k, v = (t.float() for t in make([n], H, KV, hd, dtype, seed=3))
    if slope:
        q[:, ::hd] = 8.0
        k[:, ::hd] = torch.arange(n, device="cuda")[:, None] / n * slope * hd ** 0.5 / 8.0
    q, k, v = (t.to(dtype) for t in (q, k, v))
    got = attend(q, k, v, [n], H, KV, hd)
    assert pkv.pkv_contiguous_sync_error(torch.cuda.current_stream()) == pkv.PKV_OK
    rows = torch.cat([torch.arange(a, a + 40, device="cuda") for a in (0, 8180, 16370, 19960)])
    exp, A, es = exact(q, k, v, rows, H, KV, hd, True)
    tail = n * 2.0 ** -24 * v.double().abs().max()
    assert bool(((got[rows].double() - exp).abs() <= A * (2 * U[dtype] + 2 * es) + tail).all())


@pytest.mark.parametrize("hd", [128, 64])
def test_rows_do_not_depend_on_a_long_neighbour(hd):
    """Prompts on both sides of the length from which sums have their leading part set aside, together and alone; a value
    that is not finite in the long one."""
    H, KV, lens = 4, 1, [9000, 20000, 300, 16384, 16385]
    q, k, v = make(lens, H, KV, hd, torch.bfloat16, seed=7)
    got = attend(q, k, v, lens, H, KV, hd)
    at = 0
    for n in lens:
        s = slice(at, at + n)
        assert torch.equal(attend(q[s], k[s], v[s], [n], H, KV, hd), got[s]), n
        at += n
    v2 = v.clone()
    v2[9000 + 17000, 5] = math.inf
    bad = attend(q, k, v2, lens, H, KV, hd)
    torch.cuda.synchronize()
    assert torch.equal(bad[:26000], got[:26000]) and torch.equal(bad[29000:], got[29000:])
    cols = torch.arange(H * hd, device="cuda") % hd == 5
    assert bool((~torch.isfinite(bad[26000:29000, cols])).all())
    assert torch.equal(bad[26000:29000, ~cols], got[26000:29000, ~cols])

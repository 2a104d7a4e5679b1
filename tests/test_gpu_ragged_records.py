"""Split keys: a record whose weight underflows to 0 still counts where it holds an infinity or a NaN (0 times either is
NaN), so that what a call answers does not go by how its keys were split."""
import pytest
import torch

from ragged_helpers import Case

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def steep(c, high):
    """Scores of 0 at the key rows in `high`, 40 sqrt(hd) below elsewhere: weights below 2^-257, which f32 holds as 0."""
    c.q.fill_(1.0)
    for x in (c.k, c.kp):
        if x is not None:
            x.fill_(-40.0)
    high.fill_(0.0)


@pytest.mark.parametrize("hd", [128, 64, 20, 160])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ql,n", [([1, 1], 20_000), ([2, 1], 5000), ([40, 1], 9000)], ids=["tokens", "few", "tiles"])
def test_a_weight_of_zero_keeps_what_is_not_finite(ql, n, bad, dtype, hd):
    c = Case(ql, [n, 300], 8, 2, hd, dtype)
    steep(c, c.k[n - 200:])
    clean = [c.call(workspace=w) for w in ("full", None)]
    c.v[50, 3] = bad  # of kv head 0: column 3 of heads 0 to 3
    hit = torch.zeros_like(clean[0], dtype=torch.bool)
    hit[:ql[0]].view(ql[0], 8, hd)[:, :4, 3] = True
    for w, before in zip(("full", None), clean):
        got = c.call(workspace=w)
        torch.cuda.synchronize()
        assert bool(torch.isnan(got[hit].float()).all())
        assert torch.equal(got[~hit], before[~hit]) and bool(torch.isfinite(got[~hit].float()).all())


@pytest.mark.parametrize("hd", [128, 20])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["v", "vp"])
def test_a_prefix_of_weight_zero_keeps_what_is_not_finite(which, bad, hd):
    """Stacked over a long prefix, whose records and the own keys' are joined."""
    n = 24
    c = Case([1] * n, [600] * n, 8, 2, hd, BF16, prefix=9000)
    steep(c, c.kp[8900:] if which == "v" else c.k)
    clean = [c.call(workspace=w) for w in ("full", None)]
    if which == "v":
        c.v[c.start[5] + 2, 7] = bad
    else:
        c.vp[100, 7] = bad
    hit = torch.zeros_like(clean[0], dtype=torch.bool)
    hit.view(n, 8, hd)[slice(5, 6) if which == "v" else slice(n), :4, 7] = True
    for w, before in zip(("full", None), clean):
        got = c.call(workspace=w)
        torch.cuda.synchronize()
        assert bool(torch.isnan(got[hit].float()).all()) and torch.equal(got[~hit], before[~hit])


def test_splits_that_see_no_key_leave_nothing():
    """A causal query whose last splits hold no key that it sees, beside ones whose keys all have weights."""
    c = Case([3, 1], [3000, 3000], 2, 1, 64, BF16, prefix=2000)
    c.check()
    c.v[c.start[0] + 2999] = float("inf")  # seen by query 2 alone
    got = c.call()
    torch.cuda.synchronize()
    assert bool(torch.isfinite(got[[0, 1, 3]].float()).all()) and not bool(torch.isfinite(got[2].float()).any())


@pytest.mark.parametrize("hd", [128, 64, 20, 160])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("workspace", ["full", None])
@pytest.mark.parametrize("ql", [[1, 1], [60, 1]], ids=["tokens", "tiles"])
def test_scores_that_are_infinite(ql, workspace, dtype, hd):
    """A score of minus infinity is a weight of 0, as if its key were not there; one of infinity makes the row NaN."""
    c = Case(ql, [3001, 200], 4, 2, hd, dtype, gap=0)
    c.q.copy_(c.q.abs() + 0.5)
    c.k[3000, 3] = -float("inf")  # of kv head 0
    got = c.call(workspace=workspace)
    short = Case(ql, [3000, 200], 4, 2, hd, dtype, k_start=[0, 3001])
    short.q, short.k, short.v = c.q, c.k, c.v
    exp, tol = short.plain()
    whole, tol1 = c.plain()
    exp[:, 2 * hd:], tol[:, 2 * hd:] = whole[:, 2 * hd:], tol1[:, 2 * hd:]  # kv head 1 sees all its keys
    assert bool(((got.double() - exp).abs() <= tol).all())
    c.k[3000, 3] = float("inf")
    bad = c.call(workspace=workspace)
    torch.cuda.synchronize()
    assert bool(torch.isnan(bad[:ql[0], :2 * hd].float()).all())
    assert torch.equal(bad[:, 2 * hd:], got[:, 2 * hd:]) and torch.equal(bad[ql[0]:], got[ql[0]:])

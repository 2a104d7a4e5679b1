"""pkv_attn_cross and pkv_attn_prefix against the formula in 64 bits (tolerance: ragged_helpers)."""
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from ragged_helpers import Case

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
DTYPES = pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
# head shapes of the 128- and 64-wide kernels, wide heads, widths that are no whole 16 bytes
SHAPES = [(8, 2, 128), (3, 3, 64), (7, 1, 80), (16, 1, 128), (32, 1, 64), (4, 2, 24), (4, 2, 160), (2, 2, 256), (4, 2, 20),
          (2, 1, 131), (3, 1, 1)]

BAD = pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])

CROSS = [([1], [1]), ([1, 1, 0, 1], [0, 5, 7, 33]), ([130, 1, 17], [129, 640, 64]), ([5, 33, 64, 2], [16, 128, 0, 255]),
         ([300], [700]), ([1, 1], [9000, 300]), ([40, 3], [5000, 2500])]


@pytest.mark.parametrize("ql,kl", CROSS, ids=str)
@DTYPES
@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (3, 3, 64)])
def test_cross_lengths(ql, kl, dtype, H, KV, hd):
    c = Case(ql, kl, H, KV, hd, dtype, seed=len(ql))
    c.check()
    c.check(workspace=None)


@pytest.mark.parametrize("H,KV,hd", SHAPES)
@DTYPES
def test_cross_heads_and_widths(H, KV, hd, dtype):
    Case([3, 1, 70, 1], [300, 17, 131, 2000], H, KV, hd, dtype, gap=5, seed=hd).check()


PREFIX = [(0, [1, 3], [4, 3]), (1, [1], [1]), (127, [1, 2, 0, 5], [9, 2, 6, 40]), (128, [40, 1, 1], [40, 300, 1]),
          (1000, [1] * 9, [1, 2, 16, 17, 64, 65, 100, 333, 5]), (300, [129, 64], [140, 64]), (2500, [2, 7, 130], [2, 70, 130]),
          (5000, [1, 1, 1], [1, 1, 900])]


@pytest.mark.parametrize("prefix,ql,kl", PREFIX, ids=str)
@DTYPES
@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (3, 3, 64)])
def test_prefix_lengths(prefix, ql, kl, dtype, H, KV, hd):
    c = Case(ql, kl, H, KV, hd, dtype, prefix=prefix, seed=prefix)
    c.check()
    c.check(workspace=None)


@pytest.mark.parametrize("H,KV,hd", SHAPES)
@DTYPES
def test_prefix_heads_and_widths(H, KV, hd, dtype):
    Case([3, 1, 70, 1, 1], [30, 17, 71, 200, 1], H, KV, hd, dtype, prefix=333, gap=3, seed=hd).check()


@pytest.mark.parametrize("hd", [136, 160, 192, 200, 256])
@DTYPES
def test_wide_heads_on_tiles(hd, dtype):
    """One chain a piece; lengths around its tiles, split keys, and more keys than one sum takes."""
    Case([1, 129, 64, 65, 300], [700, 128, 129, 1, 255], 4, 2, hd, dtype, seed=hd).check()
    Case([130, 1], [6000, 16], 2, 1, hd, dtype, seed=hd).check()
    Case([100], [17_000], 1, 1, hd, dtype, seed=hd).check()
    Case([90, 1, 40], [400, 30, 40], 3, 1, hd, dtype, prefix=1000, gap=40, seed=hd).check()


@pytest.mark.parametrize("H,KV,hd", [(20, 20, 64), (8, 4, 40), (6, 2, 56)])
@DTYPES
def test_one_tile_of_queries_takes_its_keys_on_both_chains(H, KV, hd, dtype):
    """Pieces of one query tile and one to many key tiles, after one another and among whole ones, many to a block."""
    ql = [24, 128, 1, 100, 300, 33, 129, 50, 64, 90, 260, 40]
    kl = [1, 128, 700, 129, 900, 255, 256, 257, 385, 1500, 640, 513]
    Case(ql, kl, H, KV, hd, dtype, seed=hd).check()
    Case(ql, kl, H, KV, hd, dtype, seed=hd).check(workspace=None)
    Case([60], [15_000], H, KV, hd, dtype, seed=hd).check()
    Case([30, 100, 128, 70], [300, 100, 500, 70], H, KV, hd, dtype, prefix=700, gap=90, seed=hd).check()
    Case([60] * 90, [400 + 130 * (i % 4) for i in range(90)], H, KV, hd, dtype, seed=hd).check()


@pytest.mark.parametrize("workspace", ["full", None])
@pytest.mark.parametrize("hd", [8, 64])
@BAD
def test_a_piece_with_hidden_values_waits_for_the_output_before_it(hd, bad, workspace):
    """Blocks go from pieces whose last tile, on one chain, hides rows that are not finite to pieces where the other
    chain's first tile does: its output there still holds its part of the piece before."""
    ql = [53, 62, 58, 80, 1, 1, 12, 1, 58, 5, 97, 1, 1, 40, 80, 3, 1, 46, 41, 1, 77, 28, 1, 44, 1, 38, 56, 29, 1, 26, 1, 1, 1,
          61, 1, 2, 81, 1, 36, 1, 1, 85, 1, 1, 52, 1]
    kl = [53, 62, 58, 80, 1, 168, 516, 75, 80, 5, 124, 1, 211, 40, 80, 3, 368, 46, 238, 1, 90, 415, 1, 44, 226, 38, 56, 29, 45,
          468, 1, 1, 498, 61, 22, 2, 81, 1, 36, 1, 1, 85, 1, 1, 52, 1]
    c = Case(ql, kl, 17, 1, hd, BF16, prefix=128, gap=7, seed=hd)
    for s, n in zip(c.start, c.kl):
        c.v[s + n:s + n + 7] = bad
    c.check(workspace=c.workspace() if workspace else None)
    c = Case([40] * 90, [300] * 45 + [200] * 45, 6, 6, hd, BF16, gap=3, seed=hd)
    for s, n in zip(c.start, c.kl):
        c.v[s + n:s + n + 3] = bad
    c.check(workspace=c.workspace() if workspace else None)


@pytest.mark.parametrize("which", ["k", "v"])
@BAD
def test_both_chains_keep_values_out_of_sight(which, bad):
    c = Case([100, 60, 128, 90], [130, 389, 600, 257], 3, 3, 64, BF16, gap=3, seed=1)
    clean = c.call()
    rows = getattr(c, which)
    for s, n in zip(c.start, c.kl):
        rows[s + n:s + n + 3] = bad
    assert torch.equal(c.call(), clean)
    p = Case([100, 60, 90], [400, 389, 257], 3, 3, 64, BF16, prefix=200, gap=90, seed=1)
    clean = p.call()
    getattr(p, which)[p.start[1] + 360] = bad  # seen by queries 31 .. of sequence 1
    got = p.call()
    torch.cuda.synchronize()
    assert torch.equal(got[:131], clean[:131]) and torch.equal(got[160:], clean[160:])
    assert not bool(torch.isfinite(got[131:160].float()).all(dim=1).any())


@pytest.mark.parametrize("ql,kl", [([100, 1, 3, 60], [700, 700, 1, 129]), ([100, 1, 1, 1, 1], [300, 600, 600, 300, 4]),
                                   ([1, 300, 0, 2, 1], [128, 1000, 50, 0, 2000]), ([60, 1], [20, 5000])],
                         ids=["along", "too_many", "one_without_keys", "too_long"])
@pytest.mark.parametrize("H,KV,hd", [(20, 20, 64), (8, 2, 128), (4, 4, 80), (4, 2, 256)])
@DTYPES
def test_tokens_among_prompts(ql, kl, dtype, H, KV, hd):
    c = Case(ql, kl, H, KV, hd, dtype, seed=hd)
    c.check()
    c.check(workspace=None)


def test_more_sequences_than_one_launch_takes():
    n = 2003
    r = torch.Generator().manual_seed(5)
    kl = torch.randint(0, 40, (n,), generator=r).tolist()
    ql = torch.randint(0, 3, (n,), generator=r).tolist()
    Case(ql, kl, 4, 2, 64, BF16, seed=1).check()
    Case(ql, [a + b for a, b in zip(ql, kl)], 4, 2, 64, BF16, prefix=200, seed=2).check()


@pytest.mark.parametrize("prefix", [None, 700])
@pytest.mark.parametrize("hd,shift", [(128, 0), (128, 8), (128, 1), (64, 3), (40, 8), (160, 8)])
def test_strides_alignment_and_rows_left_alone(hd, shift, prefix):
    """Columns of wider rows; shift 1 and 3 leave the 16-byte boundaries.  Rows behind the last sequence and the
    columns beside the output stay as they were."""
    H, KV, ql, kl = 4, 2, [2, 61, 1], [200, 61, 900]
    c = Case(ql, kl, H, KV, hd, BF16, prefix=prefix)
    T, qd, kd = sum(ql), H * hd, KV * hd

    def wide(x):
        y = torch.full((x.shape[0] + 2, x.shape[1] + 24 + shift), 3.0, dtype=BF16, device="cuda")
        z = y[:x.shape[0], shift + 8:shift + 8 + x.shape[1]]
        z.copy_(x)
        return y, z
    (_, c.q), (_, c.k), (_, c.v) = wide(c.q), wide(c.k), wide(c.v)
    if prefix:
        (_, c.kp), (_, c.vp) = wide(c.kp), wide(c.vp)
    all_, out = wide(torch.full((T, qd), 7.0, dtype=BF16, device="cuda"))
    all_.fill_(7.0)
    c.call(out=out)
    c.check(got=out)
    assert bool((all_[T:] == 7).all()) and bool((all_[:, :shift + 8] == 7).all()) and bool((all_[:, shift + 8 + qd:] == 7).all())


@pytest.mark.parametrize("workspace", [16, 50_000, 400_000])
@pytest.mark.parametrize("prefix", [None, 3000])
def test_a_short_workspace(workspace, prefix):
    c = Case([1, 4, 1, 60], [7000, 300, 1, 900], 8, 2, 128, BF16, prefix=prefix)
    whole = torch.full((workspace + 4096,), 7, dtype=torch.uint8, device="cuda")
    c.check(workspace=whole[:workspace])
    assert bool((whole[workspace:] == 7).all())


def test_beams_share_their_rows():
    ql, kl = [1, 1, 1, 2, 1, 1], [900, 900, 900, 50, 0, 900]
    start = [10, 10, 10, 0, 77, 10]
    Case(ql, kl, 8, 2, 128, BF16, k_start=start).check()
    Case(ql, kl, 8, 2, 20, BF16, k_start=start).check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-30, 40.0])
@DTYPES
def test_scales(scale, dtype):
    Case([1, 70, 3], [500, 300, 40], 4, 2, 64, dtype).check(scale=scale)
    Case([1, 70, 3], [5, 300, 40], 4, 2, 64, dtype, prefix=400).check(scale=scale)


@pytest.mark.parametrize("mul", [30.0, 1e-3])
def test_steep_and_flat_scores(mul):
    Case([1, 70, 3], [5000, 300, 40], 4, 2, 128, BF16, mul=mul).check()
    Case([1, 70, 3], [5, 300, 40], 4, 2, 128, F16, prefix=4000, mul=mul).check()


def test_rising_scores_move_the_reference():
    """Every key scores higher than the ones before it, far past the headroom of the running maximum."""
    c = Case([1, 90], [4000, 2000], 2, 1, 64, BF16)
    c.q.fill_(1.0)
    c.k.copy_((torch.arange(c.k.shape[0], device="cuda") % 4000 / 40.0)[:, None].expand_as(c.k))
    c.check(scale=0.125)
    c.k.copy_(c.k.flip(0))
    c.check(scale=0.125)




@pytest.mark.parametrize("hd", [128, 64, 20, 160])
@BAD
@pytest.mark.parametrize("which", ["k", "v"])
def test_cross_reads_no_row_of_another_sequence(hd, bad, which):
    c = Case([3, 1, 140, 1], [30, 500, 131, 3], 4, 2, hd, BF16, gap=2, seed=9)
    clean = c.call()
    rows = getattr(c, which)
    for s, n in zip(c.start, c.kl):
        rows[s + n:s + n + 2] = bad  # between the sequences
    assert torch.equal(c.call(), clean)
    rows[c.start[1] + 77, 3] = bad   # kv head 0 of sequence 1
    got = c.call()
    torch.cuda.synchronize()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[3, :2 * hd] = False
    assert torch.equal(got[keep], clean[keep])
    if which == "v":
        col = got[3].view(4, hd)[:2, 3].float()
        assert not bool(torch.isfinite(col).any())
        assert bool(torch.isfinite(got[3].float()).sum() == 4 * hd - 2)


@pytest.mark.parametrize("hd", [128, 64, 20, 160])
@BAD
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("workspace", ["full", None])
def test_prefix_queries_read_no_later_row(hd, bad, which, workspace):
    c = Case([3, 1, 140, 90], [30, 50, 140, 300], 4, 2, hd, BF16, prefix=200, seed=9)
    clean = c.call(workspace=workspace)
    row = c.start[2] + 60  # seen by queries 60 .. of sequence 2
    getattr(c, which)[row] = bad
    got = c.call(workspace=workspace)
    torch.cuda.synchronize()
    assert torch.equal(got[:4 + 60], clean[:4 + 60]) and torch.equal(got[144:], clean[144:])
    assert not bool(torch.isfinite(got[4 + 60:144].float()).all(dim=1).any())


def test_an_infinity_in_sight_is_an_infinity():
    c = Case([1, 1], [300, 40], 2, 2, 64, BF16, prefix=500)
    c.vp[100, 5] = float("inf")
    c.v[7, 9] = -float("inf")
    got = c.call()
    torch.cuda.synchronize()
    assert bool((got[:, 5] == float("inf")).all()) and float(got[0, 9]) == -float("inf")
    rest = torch.ones(128, dtype=torch.bool, device="cuda")
    rest[[5, 9]] = False
    assert bool(torch.isfinite(got[:, rest].float()).all())


@pytest.mark.parametrize("prefix", [None, 1500])
def test_the_same_call_twice_gives_the_same_bits(prefix):
    c = Case([1, 70, 2, 1], [6000, 900, 3, 200], 8, 2, 128, BF16, prefix=prefix)
    first = c.call().clone()
    for _ in range(3):
        assert torch.equal(c.call(), first)


@pytest.mark.parametrize("prefix", [None, 1500])
def test_captured_and_replayed(prefix):
    c = Case([1, 70, 2, 1], [6000, 900, 3, 200], 8, 2, 128, BF16, prefix=prefix)
    out, w = torch.zeros(74, 1024, dtype=BF16, device="cuda"), c.workspace()
    c.call(out=out, workspace=w)  # (sets up what a first call sets up)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(out=out, workspace=w, stream=torch.cuda.current_stream())
    for seed in (1, 2):
        other = Case([1, 70, 2, 1], [6000, 900, 3, 200], 8, 2, 128, BF16, prefix=prefix, seed=seed)
        for name in ("q", "k", "v") + (("kp", "vp") if prefix else ()):
            getattr(c, name).copy_(getattr(other, name))
        w.fill_(255)
        g.replay()
        c.check(got=out)


@pytest.mark.parametrize("prefix", [None, 1500])
def test_two_streams(prefix):
    """Calls in flight at once, a workspace each, on streams of their own."""
    cases = [Case([1, 70, 2, 1], [6000, 900, 3, 200], 8, 2, 128, BF16, prefix=prefix, seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(c.q) for c in cases]
    spaces = [c.workspace() for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, o, w in zip(cases, streams, outs, spaces):
            c.call(out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(got=o)


def test_one_sign_over_many_keys():
    """Sums that the tensor core rounds toward zero: values of one sign, 70,000 keys."""
    for kw in (dict(ql=[1, 130], kl=[70_000, 70_000]), dict(ql=[1, 1, 130], kl=[1, 1, 130], prefix=70_000)):
        c = Case(H=2, KV=1, hd=64, dtype=F16, mul=0.01, **kw)
        for x in (c.v, c.vp):
            if x is not None:
                x.copy_(x.abs() + 1.0)
        c.check()


def test_offsets_past_32_bits():
    """A row stride that puts the last rows past 2^32 elements (8.6 GB of which 3 rows are touched)."""
    hd, stride = 64, (1 << 32) // 600
    room = torch.empty(stride * 640 + 4096, dtype=BF16, device="cuda")
    c = Case([1, 33], [640, 600], 2, 1, hd, BF16, k_start=[0, 40])
    for name, at in (("k", 0), ("v", 1024)):
        big = room[at:].as_strided((640, hd), (stride, 1))
        big.copy_(getattr(c, name))
        setattr(c, name, big)
    c.check()
    p = Case([1, 33], [4, 600], 2, 1, hd, BF16, prefix=640)
    p.kp, p.vp = c.k, c.v
    p.check()


# ---- short sequences whose tiles hold the rows of several ----

SHORT = [([7, 1, 30, 2, 64, 65, 1, 1, 200, 3], 0), ([5] * 60, 0), ([1] * 130, 0), ([24, 9, 40, 33], 6), ([300, 2, 290, 5], 3)]


@pytest.mark.parametrize("ql,more", SHORT, ids=["mixed", "fives", "ones", "behind_own_keys", "long_and_short"])
@pytest.mark.parametrize("prefix", [0, 100, 640, 2000])
@pytest.mark.parametrize("H,KV,hd", [(8, 2, 128), (3, 3, 64), (7, 1, 80), (32, 2, 128), (6, 2, 160), (2, 1, 256)])
@DTYPES
def test_short_sequences_behind_one_another(ql, more, prefix, H, KV, hd, dtype):
    c = Case(ql, [n + more for n in ql], H, KV, hd, dtype, prefix=prefix, gap=more, seed=len(ql))
    c.check()
    c.check(workspace=None)


@pytest.mark.parametrize("hd", [128, 64, 160])
@BAD
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("gap", [0, 5])
def test_a_shared_tile_keeps_sequences_apart(hd, bad, which, gap):
    ql = [20, 7, 60, 1, 33, 90, 4]
    c = Case(ql, ql, 4, 2, hd, BF16, prefix=300, gap=gap, seed=3)
    clean = c.call()
    rows = getattr(c, which)
    for s, n in zip(c.start, c.kl):
        rows[s + n:s + n + gap] = bad
    got = c.call()
    torch.cuda.synchronize()
    assert torch.equal(got, clean)
    rows[c.start[2] + 25] = bad  # seen by queries 25 .. 59 of sequence 2: rows 52 .. 86
    got = c.call()
    torch.cuda.synchronize()
    assert torch.equal(got[:52], clean[:52]) and torch.equal(got[87:], clean[87:])
    assert not bool(torch.isfinite(got[52:87].float()).all(dim=1).any())

"""Appends to 8-bit pools that are long enough for the walk over pages (from
9,728 pages x kv heads x 2 on): elements, scales and untouched places bit for
bit against the oracle."""
import math

import numpy as np
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from test_gpu_q8_pool import Model, Q8Pool

pytestmark = pytest.mark.gpu
WALK = 4 * 2 * 152 * 8    # (page, head, K or V) triples


# pages beside the launch's parameters and in them; rows of whole and of half warps, odd pages, a page of one row
@pytest.mark.parametrize("KV,hd,bs,pages", [(8, 128, 16, 157), (8, 64, 5, 155), (2, 256, 8, 613), (4, 32, 17, 307),
                                            (16, 128, 1, 83)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
def test_long_append_bit_exact(KV, hd, bs, pages, dtype):
    """Sequences that start inside a page, then two long appends, the second of larger rows (the step of the page
    between them grows), strided rows, one value that is not finite."""
    kd, layer = KV * hd, 1
    steps = [([1, bs + 1, 2 * bs, 3, bs - 1 or 1], 1.0),
             ([pages * bs + 1, pages * bs, (pages - 2) * bs + 3, pages * bs + bs // 2, 2], 0.25),
             ([2, pages * bs - 1, (pages + 1) * bs, pages * bs + 2, pages * bs], 9.0)]
    total = [sum(n[r] for n, _ in steps) for r in range(5)]
    pool = Q8Pool(sum(-(-t // bs) for t in total) + 7, 2, KV, hd, bs)
    try:
        seqs = [pool.seq(t) for t in total]
        models = [[Model(bs, KV, hd) for _ in range(2)] for _ in seqs]
        bad = [[set(), set()] for _ in seqs]        # (page, head) whose scale is NaN
        lens = [0] * 5
        g = torch.Generator(device="cuda")
        for i, (n, mul) in enumerate(steps):
            g.manual_seed(100 * hd + i)
            w = torch.randn(sum(n), 2 * kd + 16, device="cuda", generator=g)
            w *= torch.exp2(torch.randint(-3, 4, (sum(n), 1), device="cuda", generator=g).float()) * mul
            w = w.to(dtype)
            x, y = w[:, 8:8 + kd], w[:, 16 + kd:]
            poison = n[0] + n[1] // 2 if i == 2 else None       # a row of sequence 1
            host = [t.double().cpu().numpy() for t in (x, y)]   # the oracle takes finite rows
            if poison is not None:
                x[poison, hd + 1] = math.inf
                y[poison, 5] = math.nan
                page = (lens[1] + n[1] // 2) // bs
                bad[1][0].add((page, 1))
                bad[1][1].add((page, 0))
            items = sum((lens[r] + n[r] - 1) // bs - lens[r] // bs + 1 for r in range(5))
            assert (2 * items * KV >= WALK) == (i > 0)
            pool.append(seqs, x, y, n, layers=[layer])
            at = 0
            for r in range(5):
                for which in range(2):
                    models[r][which].append(lens[r], host[which][at:at + n[r]])
                at += n[r]
                lens[r] += n[r]
        pool.ok()
        for r, s in enumerate(seqs):
            ids = torch.tensor(pkv.pkv_seq_page_table(s), device="cuda")
            for which, (E, S) in enumerate(((pool.K, pool.Ks), (pool.V, pool.Vs))):
                e = E[ids, layer].cpu().numpy().astype(np.float64).reshape(-1, KV, hd)
                sc = S[ids, layer].double().cpu().numpy()
                m = models[r][which]
                for pg in range(len(ids)):
                    rows = slice(pg * bs, min((pg + 1) * bs, lens[r]))
                    for h in range(KV):
                        if (pg, h) in bad[r][which]:
                            assert math.isnan(sc[pg, h]), (r, which, pg, h)
                            continue
                        assert sc[pg, h] == 2.0 ** m.e[pg, h], (r, which, pg, h)
                        assert np.array_equal(e[rows, h] - 128, m.q[pg, h][:rows.stop - rows.start]), (r, which, pg, h)
                assert (e[lens[r]:] == 255).all()
        assert bool((pool.K[:, 0] == 255).all()) and bool(torch.isnan(pool.Vs[:, 0]).all())    # the other layer
    finally:
        pool.close()


def test_more_warps_than_32_bits_count_are_refused():
    """Pages of one token and a million heads of one element: refused before anything is read or launched."""
    n, heads = 1025, 1 << 20
    pool = pkv.pkv_pool_new_q8(n, 1, heads, 1, 1, max_seqs=1, max_blocks_per_seq=n, stream=torch.cuda.current_stream())
    if not pool:
        pytest.skip("11 GB of pool: " + pkv.pkv_last_error())
    try:
        s = pkv.pkv_seq_new(pool, n)
        pkv.check(pkv.pkv_ensure_append(s, n))
        rows = 4096     # no address: the call must not get as far
        launches = pkv.pkv_launch_count()
        assert pkv.pkv_append_layer(s, 0, rows, rows, n) == pkv.PKV_ERR_BAD_DIM, pkv.pkv_last_error()
        assert pkv._lib.pkv_append_packed(pkv.seq_array([s]), 1, pkv.i32_array([n]), 0, rows, heads, rows, heads,
                                          pkv.PKV_F32) == pkv.PKV_ERR_BAD_DIM
        assert pkv.pkv_launch_count() == launches
        assert pkv.pkv_sync_error(pool) == pkv.PKV_OK
    finally:
        torch.cuda.synchronize()
        pkv.pkv_pool_free(pool)

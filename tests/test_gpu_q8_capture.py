"""Calls on an 8-bit pool inside a graph capture: refused before anything is enqueued or changed, so that the same
call afterwards, outside the capture, is right."""
import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from test_gpu_q8_pool import Q8Pool, randn

pytestmark = pytest.mark.gpu
H, KV, hd, bs, scale = 4, 2, 64, 16, 0.125


class Captured:
    """A capture on a side stream that the pool is bound to for its length."""

    def __init__(self, pool):
        self.pool, self.g, self.side = pool, torch.cuda.CUDAGraph(), torch.cuda.Stream()

    def __enter__(self):
        self.x = torch.zeros(1, device="cuda")
        torch.cuda.synchronize()
        self.ctx = torch.cuda.stream(self.side)
        self.ctx.__enter__()
        pkv.check(pkv.pkv_pool_set_stream(self.pool.p, self.side))
        self.g.capture_begin()
        return self

    def __exit__(self, *a):
        self.x.add_(1.0)
        self.g.capture_end()
        self.ctx.__exit__(*a)
        self.g.replay()
        torch.cuda.synchronize()
        assert self.x.item() == 1.0
        pkv.check(pkv.pkv_pool_set_stream(self.pool.p, torch.cuda.current_stream()))


@pytest.mark.parametrize("pinned", [True, False])
@pytest.mark.parametrize("n_q", [1, 40])
def test_host_buffers(pinned, n_q):
    pool = Q8Pool(40, 1, KV, hd, bs)
    try:
        s, twin = pool.seq(200), pool.seq(200)
        x, y = randn(100, KV * hd, seed=1), randn(100, KV * hd, seed=2)
        for t in (s, twin):
            pool.append([t], x, y, [100])
            pkv.check(pkv.pkv_ensure_append(t, n_q))
        q, x, y = (randn(n_q, w * hd, seed=3 + w) for w in (H, KV, KV))
        host = [t.cpu().pin_memory() if pinned else t.cpu() for t in (q, x, y)]
        out = torch.full((n_q, H * hd), 7.0)
        out = out.pin_memory() if pinned else out
        with Captured(pool):
            rc = pkv.pkv_attn_batch_host([s], [n_q], *host, H, KV, hd, 0, 1, scale, out)
        assert rc == pkv.PKV_ERR_ARG and "captured" in pkv.pkv_last_error()
        assert bool((out == 7.0).all())
        pkv.check(pkv.pkv_attn_batch_host([s], [n_q], *host, H, KV, hd, 0, 1, scale, out))
        exp = torch.empty(n_q, H * hd, device="cuda")
        pkv.check(pkv.pkv_attn_batch([twin], [n_q], q, x, y, H, KV, hd, 0, 1, scale, exp))
        pool.ok()
        assert torch.equal(out, exp.cpu())
    finally:
        pool.close()


def test_copies_and_page_tables():
    """pkv_ensure_append where it would copy a shared block, and pkv_pool_flush: the same step afterwards reads right."""
    pool = Q8Pool(40, 1, KV, hd, bs)
    try:
        s = pool.seq(200)
        x, y = randn(100, KV * hd, seed=1), randn(100, KV * hd, seed=2)
        pool.append([s], x, y, [100])
        f = pkv.pkv_seq_fork(s)
        fresh = pool.seq(50)
        before = [t.clone() for t in pool.values(s, 100)]
        table, free = pkv.pkv_seq_page_table(f), pkv.pkv_pool_free_blocks(pool.p)
        with Captured(pool):
            rcs = [pkv.pkv_ensure_append(f, 1)]
            pkv.check(pkv.pkv_ensure_append(fresh, 20))        # nothing to copy: the host's lists alone
            rcs.append(pkv.pkv_pool_flush(pool.p))
        assert rcs == [pkv.PKV_ERR_ARG] * 2
        assert pkv.pkv_seq_page_table(f) == table and pkv.pkv_pool_free_blocks(pool.p) == free - 2
        n = [1, 20]
        pkv.check(pkv.pkv_ensure_append(f, 1))
        q, x, y = (randn(21, w * hd, seed=3 + w) for w in (H, KV, KV))
        out = torch.empty(21, H * hd, device="cuda")
        pkv.check(pkv.pkv_attn_batch([f, fresh], n, q, x, y, H, KV, hd, 0, 1, scale, out))
        pool.ok()
        assert all(torch.equal(a, b) for a, b in zip(pool.values(s, 100), before))
        # the fork's copy holds the parent's rows, in the step that the new row asks for
        step = pool.Ks[pkv.pkv_seq_page_table(f)[-1], 0].max().item()
        assert (pool.values(f, 100)[0] - before[0]).abs().max().item() <= step / 2
        exp = torch.empty_like(out)
        other = Q8Pool(40, 1, KV, hd, bs)
        try:
            a, b = other.seq(200), other.seq(50)
            other.append([a], randn(100, KV * hd, seed=1), randn(100, KV * hd, seed=2), [100])
            pkv.check(pkv.pkv_ensure_append_batch([a, b], n))
            pkv.check(pkv.pkv_attn_batch([a, b], n, q, x, y, H, KV, hd, 0, 1, scale, exp))
            other.ok()
        finally:
            other.close()
        assert torch.equal(out, exp)
    finally:
        pool.close()

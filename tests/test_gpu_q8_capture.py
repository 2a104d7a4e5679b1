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

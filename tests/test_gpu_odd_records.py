"""Partial records whose number is odd: the sums of V behind the maxima still start on a 16-byte boundary, in the
allocating and in the static scratch."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_nx_gb300 as pkv
from gpu_helpers import assert_close, bits_equal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 3), (5, 1)])
@pytest.mark.parametrize("n_q,past", [(33, 1167), (35, 1465), (1, 95)])
def test_odd_number_of_records(H, KV, n_q, past):
    """Three splits of an odd number of queries: 3 * n_q * H records, tensor-core tiles (groups of 1) or decode units."""
    hd, tk, stream = 128, past + n_q, torch.cuda.current_stream()
    g = torch.Generator(device="cuda")
    g.manual_seed(n_q)
    Q, K, V = (torch.randn(n, w * hd, device="cuda", generator=g) for n, w in ((n_q, H), (tk, KV), (tk, KV)))
    scale = float(np.float32(1.0 / math.sqrt(hd)))
    old = pkv.pkv_get_split_keys()
    try:
        pkv.check(pkv.pkv_set_split_keys(32))
        outs = [torch.full((n_q, H * hd), float("nan"), device="cuda") for _ in range(2)]
        for f, o in zip((pkv.pkv_attn_contiguous, pkv.pkv_attn_contiguous_noalloc), outs):
            pkv.check(f(Q, K, V, n_q, tk, H, KV, hd, 1, scale, o, stream))
        assert pkv.pkv_contiguous_sync_error(stream) == pkv.PKV_OK, pkv.pkv_last_error()
    finally:
        pkv.check(pkv.pkv_set_split_keys(old))
    assert bits_equal(*outs)
    rc, exp = oracle.attend(Q.cpu().numpy(), K.cpu().numpy(), V.cpu().numpy(), n_q, tk, H, KV, hd, 1, scale)
    assert rc == 0
    assert_close(outs[1].cpu().numpy(), exp, V.abs().max().item())

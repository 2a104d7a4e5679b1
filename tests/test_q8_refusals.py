"""Refusals of the packed-prompt and 8-bit-pool entry points, and the pins of
the 8-bit format's oracle (CPU: every check comes before any CUDA call)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_gqa_nx_gb300 as pkv

lib = pkv._lib


def _packed(lens=(3, 2), H=4, KV=2, hd=16, dtype=pkv.PKV_BF16, Q=4096, K=4096, V=4096, out=4096, qs=64, ks=32, vs=32,
            os_=64, n=None):
    arr = (ctypes.c_int32 * max(1, len(lens)))(*lens) if lens is not None else None
    return lib.pkv_attn_packed(Q, qs, K, ks, V, vs, dtype, arr, len(lens) if n is None else n, H, KV, hd, 1, 0.25, out,
                               os_, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(lens=()), pkv.PKV_ERR_BAD_DIM),
    (dict(lens=None, n=2), pkv.PKV_ERR_BAD_DIM),
    (dict(lens=(3, -1)), pkv.PKV_ERR_BAD_DIM),
    (dict(H=0), pkv.PKV_ERR_BAD_DIM),
    (dict(hd=0), pkv.PKV_ERR_BAD_DIM),
    (dict(hd=257, qs=5000, ks=5000, vs=5000, os_=5000), pkv.PKV_ERR_BAD_DIM),
    (dict(H=3), pkv.PKV_ERR_BAD_GQA),
    (dict(dtype=pkv.PKV_F32), pkv.PKV_ERR_ARG),
    (dict(dtype=7), pkv.PKV_ERR_ARG),
    (dict(qs=63), pkv.PKV_ERR_ARG),
    (dict(ks=31), pkv.PKV_ERR_ARG),
    (dict(vs=31), pkv.PKV_ERR_ARG),
    (dict(os_=63), pkv.PKV_ERR_ARG),
    (dict(qs=1 << 39), pkv.PKV_ERR_BAD_DIM),
    (dict(lens=(2 ** 31 - 1, 2 ** 31 - 1)), pkv.PKV_ERR_BAD_DIM),
    (dict(Q=None), pkv.PKV_ERR_ARG),
    (dict(K=None), pkv.PKV_ERR_ARG),
    (dict(V=None), pkv.PKV_ERR_ARG),
    (dict(out=None), pkv.PKV_ERR_ARG),
    (dict(Q=4097), pkv.PKV_ERR_ARG),
    (dict(out=4097), pkv.PKV_ERR_ARG),
])
def test_packed_attention_refuses(kw, rc):
    assert _packed(**kw) == rc, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


def test_packed_attention_of_nothing_is_ok():
    # no tokens: nothing is read, written or launched, whatever the pointers
    assert _packed(lens=(0, 0, 0), Q=None, K=None, V=None, out=None) == pkv.PKV_OK


@pytest.mark.parametrize("args", [
    dict(n_kv_heads=0), dict(head_dim=0), dict(head_dim=257), dict(n_kv_heads=1, head_dim=6), dict(n_blocks=0),
    dict(block_size=0), dict(flags=pkv.PKV_POOL_BF16), dict(flags=pkv.PKV_POOL_FP8 | pkv.PKV_POOL_HOST_ONLY),
    dict(k_pool=4096), dict(k_pool=4096, v_pool=4096), dict(k_scale=4096, v_scale=4096),
    dict(k_pool=4096, v_pool=4096, k_scale=4098, v_scale=4096),
])
def test_q8_pool_refuses(args):
    a = dict(n_blocks=4, n_layers=1, n_kv_heads=2, head_dim=16, block_size=4, max_seqs=2, max_blocks_per_seq=4, flags=0)
    a.update(args)
    assert not pkv.pkv_pool_new_q8(**a)
    assert pkv.pkv_last_error()


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_q8_pool_refuses_scales_off_16_byte_boundaries(which):
    # a copy of a block moves its scales four at a time
    a = dict(k_pool=4096, v_pool=4096, k_scale=4096, v_scale=4096)
    a[which] += 4
    assert not pkv.pkv_pool_new_q8(4, 2, 2, 16, 4, max_seqs=2, max_blocks_per_seq=4, **a)
    assert "16-byte" in pkv.pkv_last_error()


@pytest.fixture
def host_pool():
    p = pkv.pkv_pool_new_q8(8, 2, 2, 16, 4, max_seqs=3, max_blocks_per_seq=4, flags=pkv.PKV_POOL_HOST_ONLY)
    assert p, pkv.pkv_last_error()
    yield p
    pkv.pkv_pool_free(p)


def test_q8_host_pool_keeps_metadata(host_pool):
    assert pkv.pkv_pool_k_scales(host_pool) is None and pkv.pkv_pool_v_scales(host_pool) is None
    assert pkv.pkv_pool_k_scales(None) is None
    assert pkv.pkv_pool_set_kv_scale(host_pool, 2.0) == pkv.PKV_ERR_ARG
    s = pkv.pkv_seq_new(host_pool, 16)
    pkv.check(pkv.pkv_ensure_append(s, 6))
    pkv.check(pkv.pkv_advance(s, 6))
    f = pkv.pkv_seq_fork(s)
    pkv.check(pkv.pkv_ensure_append(f, 1))       # copies the shared tail block
    assert pkv.pkv_seq_page_table(s)[0] == pkv.pkv_seq_page_table(f)[0]
    assert pkv.pkv_seq_page_table(s)[1] != pkv.pkv_seq_page_table(f)[1]
    pkv.check(pkv.pkv_seq_truncate(f, 3))
    assert pkv.pkv_pool_free_blocks(host_pool) == 6


@pytest.mark.parametrize("read", [False, True])
def test_packed_pages_refuse(host_pool, read):
    s = pkv.pkv_seq_new(host_pool, 16)
    one = (ctypes.c_void_p * 1)(s)

    def call(seqs=one, M=1, n=(2,), start=(0,), layer=0, K=4096, V=4096, ks=32, vs=32, dtype=pkv.PKV_F32):
        na = None if n is None else (ctypes.c_int32 * len(n))(*n)
        sa = None if start is None else (ctypes.c_int32 * len(start))(*start)
        if read:
            return lib.pkv_read_packed(seqs, M, sa, na, layer, K, ks, V, vs, dtype)
        return lib.pkv_append_packed(seqs, M, na, layer, K, ks, V, vs, dtype)

    assert call(M=0) == pkv.PKV_ERR_BAD_DIM
    assert call(n=None) == pkv.PKV_ERR_BAD_DIM
    assert call(n=(0,)) == pkv.PKV_ERR_BAD_DIM
    assert call(seqs=None) == pkv.PKV_ERR_SEQ
    assert call(seqs=(ctypes.c_void_p * 1)(None)) == pkv.PKV_ERR_SEQ
    if read:
        assert call(start=None) == pkv.PKV_ERR_BAD_DIM
    assert call() == pkv.PKV_ERR_ARG and "host-only" in pkv.pkv_last_error()


class Rows:
    """A stand-in for packed rows on a GPU."""

    def __init__(self, n, w, device=0, stride=None, dtype=torch.bfloat16):
        self.shape, self.dtype, self.is_cuda, self.device, self.s = (n, w), dtype, True, device, stride or w

    def stride(self):
        return self.s, 1

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.device


def test_packed_attention_wants_the_current_device(monkeypatch):
    monkeypatch.setattr(pkv, "_current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_lib", type("Lib", (), {"pkv_attn_packed": staticmethod(lambda *a: 0)}))

    def call(*dev, lens=(2, 3)):
        q, k, v, o = (Rows(5, 64 if i in (0, 3) else 32, d) for i, d in enumerate(dev))
        return pkv.pkv_attn_packed(q, k, v, lens, 4, 2, 16, 1, 0.25, o)

    assert call(0, 0, 0, 0) == 0
    for dev in [(1, 1, 1, 1), (1, 0, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1)]:
        with pytest.raises(TypeError, match="current device"):
            call(*dev)
    with pytest.raises(TypeError, match="rows"):
        call(0, 0, 0, 0, lens=(2, 4))


def test_packed_pages_want_counts_and_widths_that_fit(host_pool):
    s = pkv.pkv_seq_new(host_pool, 16)
    assert pkv.pkv_seq_kv_dim(s) == 32 and pkv.pkv_seq_kv_dim(None) == -1
    ok = Rows(4, 32)
    assert pkv.pkv_append_packed([s], [2], 0, ok, ok) == pkv.PKV_ERR_ARG and "host-only" in pkv.pkv_last_error()
    assert pkv.pkv_read_packed([s], [0], [2], 0, ok, ok) == pkv.PKV_ERR_ARG
    assert pkv.pkv_append_packed([None], [2], 0, ok, ok) == pkv.PKV_ERR_SEQ
    for args in [([s], [2, 2]), ([s, s], [2])]:
        with pytest.raises(TypeError, match="entry"):
            pkv.pkv_append_packed(*args, 0, ok, ok)
        with pytest.raises(TypeError, match="entry"):
            pkv.pkv_read_packed(args[0], [0] * len(args[0]), args[1], 0, ok, ok)
    with pytest.raises(TypeError, match="entry"):
        pkv.pkv_read_packed([s], [0, 0], [2], 0, ok, ok)
    narrow = Rows(4, 16, stride=64)             # columns of a wider tensor, but too few of them
    for k, v in [(narrow, narrow), (ok, narrow), (narrow, ok)]:
        with pytest.raises(TypeError, match="wide"):
            pkv.pkv_append_packed([s], [2], 0, k, v)
    with pytest.raises(TypeError, match="element type"):
        pkv.pkv_append_packed([s], [2], 0, ok, Rows(4, 32, dtype=torch.float16))


@pytest.mark.parametrize("m,e", [
    (0.0, -126), (127.0, 0), (127.00001, 1), (126.999, 0), (63.5, -1), (63.6, 0), (1.0, -6), (0.9921875, -7),
    (float(np.nextafter(np.float32(0.9921875), np.float32(1))), -6), (1e-45, -126), (127 * 2.0 ** -126, -126),
    (128 * 2.0 ** -126, -125), (3.4028234663852886e38, 122),
])
def test_oracle_exponent_pins(m, e):
    assert oracle.q8_exponent(m) == e
    assert m <= 127.0 * 2.0 ** e and (e == -126 or m > 127.0 * 2.0 ** (e - 1))


def test_oracle_append_pins():
    q, e = oracle.q8_append(np.zeros((4, 2)), 5, [[127.0, -1.5]], 0)
    assert e == 0 and q[0].tolist() == [127.0, -2.0]             # the old exponent is not looked at; ties to even
    q, e = oracle.q8_append(q, e, [[200.0, 3.0]], 1)             # the step doubles: kept rows in the new step
    assert e == 1 and q[:2].tolist() == [[64.0, -1.0], [100.0, 2.0]]   # 63.5 -> 64, 1.5 -> 2 (ties to even)
    q, e = oracle.q8_append(q, e, [[1.0, 0.5]], 2)               # the step stays
    assert e == 1 and q[2].tolist() == [0.0, 0.0]                # 0.5 -> 0, 0.25 -> 0


def test_growths_stay_within_one_step():
    # half a step at the write, and half of each later step; steps at least double
    rng = np.random.default_rng(3)
    for _ in range(50):
        x = rng.standard_normal((16, 8)) * np.exp2(np.sort(rng.uniform(-9, 9, 16)))[:, None]
        q, e = np.zeros((16, 8)), 0
        for r in range(16):
            q, e = oracle.q8_append(q, e, x[r:r + 1], r)
        assert np.abs(q).max() <= 127
        assert np.abs(q * 2.0 ** e - x).max() < 2.0 ** e
    assert math.isfinite(e)

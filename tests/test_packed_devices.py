"""Packed append and read back refuse rows of another device than the pool's (CPU: stand-ins for the library and the
tensors, as the check comes before any launch)."""
import pytest

import paged_kv_gqa_nx_gb300 as pkv
from test_q8_refusals import Rows


class Lib:
    """The library as it would answer for a sequence of a pool of rows 32 wide on device 1."""

    def __init__(self, device):
        self.calls, self.device = 0, device

    def pkv_seq_kv_dim(self, seq):
        return 32

    def pkv_seq_device(self, seq):
        return self.device

    def pkv_append_packed(self, *a):
        self.calls += 1
        return 0

    pkv_read_packed = pkv_append_packed


@pytest.mark.parametrize("call", [lambda k, v: pkv.pkv_append_packed([8], [2], 0, k, v),
                                  lambda k, v: pkv.pkv_read_packed([8], [0], [2], 0, k, v)], ids=["append", "read"])
def test_rows_of_another_device(monkeypatch, call):
    lib = Lib(1)
    monkeypatch.setattr(pkv, "_lib", lib)
    assert call(Rows(2, 32, 1), Rows(2, 32, 1)) == 0 and lib.calls == 1
    for k, v in [(0, 0), (0, 1), (1, 0), (2, 2)]:
        with pytest.raises(TypeError, match="device"):
            call(Rows(2, 32, k), Rows(2, 32, v))
    lib.device = -1     # a host-only pool, which the library refuses: the two still have to agree
    assert call(Rows(2, 32, 1), Rows(2, 32, 1)) == 0
    with pytest.raises(TypeError, match="device"):
        call(Rows(2, 32, 0), Rows(2, 32, 1))
    assert lib.calls == 2


def test_device_of_no_device_pool():
    assert pkv.pkv_seq_device(None) == -1
    p = pkv.pkv_pool_new_q8(8, 2, 2, 16, 4, max_seqs=3, max_blocks_per_seq=4, flags=pkv.PKV_POOL_HOST_ONLY)
    try:
        assert pkv.pkv_seq_device(pkv.pkv_seq_new(p, 16)) == -1
    finally:
        pkv.pkv_pool_free(p)


@pytest.mark.gpu
def test_device_of_a_pool():
    import torch
    p = pkv.pkv_pool_new_q8(8, 1, 2, 16, 4, max_seqs=3, max_blocks_per_seq=4, stream=torch.cuda.current_stream())
    try:
        assert pkv.pkv_seq_device(pkv.pkv_seq_new(p, 16)) == torch.cuda.current_device()
    finally:
        torch.cuda.synchronize()
        pkv.pkv_pool_free(p)

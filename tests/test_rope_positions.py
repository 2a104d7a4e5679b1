"""pkv_rope_packed with positions as a view: the axes of text rows share one row of positions (`pos.expand(3, n)`), rows of
positions lie apart or overlap.  What the binding hands on is looked at with a stand-in for the library, on the CPU."""
import ctypes

import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv
from test_q8_refusals import Rows

PAIRS = (3, 3, 2)


class Positions(torch.Tensor):
    """A CPU tensor that says it is on device 0."""

    def get_device(self):
        return 0


def handed_on(monkeypatch, pos):
    """(address, stride, axes, rows) that the library gets."""
    got = []
    monkeypatch.setattr(pkv, "_current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_lib", type("Lib", (), {"pkv_rope_packed": staticmethod(lambda *a: got.append(a) or 0)}))
    n, axes = pos.shape[1], pos.shape[0]
    pos = pos.as_subclass(Positions)
    assert pkv.pkv_rope_packed(Rows(n, 64), Rows(n, 32), pos, PAIRS[:axes], 0, 4, 2, 16, 1e4, Rows(n, 64), Rows(n, 32)) == 0
    return got[0][5], got[0][6], got[0][7], got[0][10]


@pytest.mark.parametrize("view", [lambda p: p[0].expand(3, 9), lambda p: p[1:2].expand(3, 9), lambda p: p[:, :9], lambda p: p[:, 4:5],
                                  lambda p: p[0, :1].expand(3, 1), lambda p: p[::2, :9], lambda p: p.as_strided((3, 9), (1, 1)),
                                  lambda p: p[:, :9].contiguous()], ids=["shared", "one_row", "columns", "one_column", "one_position",
                                                                          "every_second", "overlapping", "whole"])
def test_the_library_gets_the_views_own_stride(monkeypatch, view):
    base = torch.arange(3 * 9, dtype=torch.int32).view(3, 9)
    pos = view(base)
    address, stride, axes, rows = handed_on(monkeypatch, pos)
    assert (axes, rows) == tuple(pos.shape) and address == pos.data_ptr()
    # every element that the kernel reads, positions[axis * stride + t], is the view's own
    assert all(stride * a + t == pos.stride(0) * a + pos.stride(1) * t for a in range(axes) for t in range(rows))


def test_one_axis_has_no_stride_to_keep(monkeypatch):
    pos = torch.arange(9, dtype=torch.int32).expand(1, 9)
    assert handed_on(monkeypatch, pos)[1:] == (9, 1, 9)


def test_the_library_takes_shared_positions_and_refuses_overlapping_ones():
    def call(stride, pos=4096, axes=3, n=5):
        pairs = (ctypes.c_int32 * 3)(*PAIRS)
        return pkv._lib.pkv_rope_packed(4096, 64, 4096, 32, pkv.PKV_BF16, pos, stride, axes, pairs, 0, n, 4, 2, 16, 1e4, 0, 8192, 64,
                                        8192, 32, None)
    for stride in (1, 4, -1, -5):
        assert call(stride) == pkv.PKV_ERR_ARG and "overlap" in pkv.pkv_last_error()
    # (stopped by the check behind the one of the stride, before any CUDA call)
    assert call(0, pos=None) == pkv.PKV_ERR_ARG and "NULL" in pkv.pkv_last_error()
    assert call(5, pos=None) == pkv.PKV_ERR_ARG and "NULL" in pkv.pkv_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 9, 2000])
@pytest.mark.parametrize("order,pairs", [(pkv.PKV_ROPE_BLOCKS, [16, 24, 24]), (pkv.PKV_ROPE_TURNS, [24, 20, 20]),
                                         (pkv.PKV_ROPE_AXIAL, [32, 32])])
def test_shared_positions_turn_as_a_copy_of_them(n, order, pairs):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    q, k = (torch.randn(n, w, device="cuda", generator=g).bfloat16() for w in (4 * 128, 2 * 128))
    row = torch.randint(0, 9000, (n + 3,), device="cuda", generator=g, dtype=torch.int32)
    for pos in (row[:n].expand(len(pairs), n), row[3:][None].expand(len(pairs), n)):
        outs = [[torch.full_like(x, float("nan")) for x in (q, k)] for _ in range(2)]
        for p, (qo, ko) in zip((pos, pos.contiguous()), outs):
            pkv.check(pkv.pkv_rope_packed(q, k, p, pairs, order, 4, 2, 128, 1e6, qo, ko, stream=torch.cuda.current_stream()))
        assert all(torch.equal(a, b) for a, b in zip(*outs))
        assert all(bool(torch.isfinite(x.float()).all()) for x in outs[0])

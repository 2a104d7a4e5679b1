"""pkv_rope_packed with positions as a view: the axes of text rows share one row of positions (`pos.expand(3, n)`), rows of
positions lie apart or overlap.  What the binding hands on is looked at with a stand-in for the library, on the CPU.
And with positions and bases that make its angles very small or very large."""
import ctypes
import math
from decimal import Decimal, getcontext

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


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.gpu
@pytest.mark.parametrize("base", [1e4, 1e6, 1e8, 1e15])
def test_sines_of_slow_pairs_and_far_positions(base):
    """A pair (0, 1) turns into (-sin, cos).  Bound: the angle's, 2^-50 of its size and |p| 2^-64 of a turn, and 2^-21 of the
    sine or cosine (the rest of an angle rounded to f32, two last places of the f32 function)."""
    getcontext().prec = 50
    r, places = 32, [0, 1, -1, 7, 1000, -12345, 131071, 1 << 20, 999_999_937, -(1 << 30) - 3, (1 << 31) - 1, -(1 << 31)]
    x = torch.cat([torch.zeros(len(places), r), torch.ones(len(places), r)], dim=1).cuda()
    pos = torch.tensor([places], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    pkv.check(pkv.pkv_rope_packed(x, None, pos, [r], pkv.PKV_ROPE_BLOCKS, 1, 0, 2 * r, base, out, None,
                                  stream=torch.cuda.current_stream()))
    got = out.double().cpu()
    for i in range(r):
        f = Decimal(int(base)) ** (Decimal(-i) / Decimal(r))
        for t, p in enumerate(places):
            a = p * f
            turn = a / (2 * PI) % 1
            near = float((turn - (turn * 4).to_integral_value() / 4) * 2 * PI)  # less the nearest quarter turn
            quarter = int((turn * 4).to_integral_value()) % 4
            s, c = [(math.sin(near), math.cos(near)), (math.cos(near), -math.sin(near)), (-math.sin(near), -math.cos(near)),
                    (-math.cos(near), math.sin(near))][quarter]
            off = abs(float(a)) * 2.0 ** -50 + abs(p) * 2.0 ** -64 * 2 * math.pi
            for y, exact in ((-float(got[t, i]), s), (float(got[t, i + r]), c)):
                assert abs(y - exact) <= off + 2.0 ** -21 * abs(exact), (i, p, y, exact, off)

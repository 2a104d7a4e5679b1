"""Refusals of the cross, shared-prefix and multi-axis rotary entry points (CPU: every check comes before any CUDA call)."""
import ctypes

import pytest
import torch

import paged_kv_gqa_nx_gb300 as pkv

lib = pkv._lib
BAD_DIM, BAD_GQA, ARG, OK = pkv.PKV_ERR_BAD_DIM, pkv.PKV_ERR_BAD_GQA, pkv.PKV_ERR_ARG, pkv.PKV_OK


def arr(v):
    return (ctypes.c_int32 * max(1, len(v)))(*v) if v is not None else None


def cross(ql=(3, 1), kl=(5, 0), k0=None, n=None, H=4, KV=2, hd=16, dtype=pkv.PKV_BF16, Q=4096, K=4096, V=4096, out=4096, qs=64,
          ks=32, vs=32, os_=64, w=None, wn=0, qn=1 << 20, kn=1 << 20):
    return lib.pkv_attn_cross(Q, qs, qn, arr(ql), K, ks, V, vs, kn, arr(kl), arr(k0), dtype, len(ql) if n is None else n, H, KV, hd, 0.25,
                              out, os_, w, wn, None)


def prefix(ql=(3, 1), kl=(5, 1), k0=None, P=7, n=None, H=4, KV=2, hd=16, dtype=pkv.PKV_BF16, Q=4096, K=4096, V=4096, Kp=4096,
           Vp=4096, out=4096, qs=64, ks=32, vs=32, ps=32, xs=32, os_=64, w=None, wn=0, qn=1 << 20, kn=1 << 20):
    return lib.pkv_attn_prefix(Q, qs, qn, arr(ql), Kp, ps, Vp, xs, P, K, ks, V, vs, kn, arr(kl), arr(k0), dtype,
                               len(ql) if n is None else n, H, KV, hd, 0.25, out, os_, w, wn, None)


BIG = 2 ** 31 - 1
COMMON = [
    (dict(n=0), BAD_DIM), (dict(n=-1), BAD_DIM), (dict(kl=None), BAD_DIM), (dict(ql=(3, -1)), BAD_DIM),
    (dict(kl=(5, -1)), BAD_DIM), (dict(H=0), BAD_DIM), (dict(KV=0), BAD_DIM), (dict(hd=0), BAD_DIM),
    (dict(hd=257, qs=5000, ks=5000, vs=5000, os_=5000), BAD_DIM), (dict(H=3), BAD_GQA), (dict(dtype=pkv.PKV_F32), ARG),
    (dict(dtype=9), ARG), (dict(qs=63), ARG), (dict(ks=31), ARG), (dict(vs=31), ARG), (dict(os_=63), ARG),
    (dict(qs=1 << 40), BAD_DIM), (dict(ks=1 << 40), BAD_DIM), (dict(k0=(0, -1)), BAD_DIM), (dict(k0=(BIG, 0)), BAD_DIM),
    (dict(kl=(BIG, 1)), BAD_DIM), (dict(Q=None), ARG), (dict(K=None), ARG), (dict(V=None), ARG), (dict(out=None), ARG),
    (dict(Q=4097), ARG), (dict(K=4097), ARG), (dict(V=4097), ARG), (dict(out=4097), ARG), (dict(w=4104, wn=64), ARG),
    (dict(w=None, wn=64), ARG), (dict(w=4096, wn=-1), ARG), (dict(qn=3), ARG), (dict(kn=4), ARG), (dict(kn=14, k0=(10, 0)), ARG)]


@pytest.mark.parametrize("kw,rc", COMMON + [(dict(ql=(BIG, BIG), kl=(1, 1)), BAD_DIM)], ids=str)
def test_cross_refuses(kw, rc):
    assert cross(**kw) == rc, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


@pytest.mark.parametrize("kw,rc", COMMON + [
    (dict(P=-1), BAD_DIM), (dict(P=BIG), BAD_DIM), (dict(ql=(6, 1)), BAD_DIM), (dict(Kp=None), ARG), (dict(Vp=None), ARG),
    (dict(Kp=4097), ARG), (dict(Vp=4097), ARG), (dict(ps=31), ARG), (dict(xs=31), ARG), (dict(ps=1 << 40), BAD_DIM)], ids=str)
def test_prefix_refuses(kw, rc):
    assert prefix(**kw) == rc, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


def test_nothing_to_do_is_ok():
    none = dict(Q=None, K=None, V=None, out=None)
    assert cross(ql=(0, 0), **none) == OK and prefix(ql=(0, 0), Kp=None, Vp=None, **none) == OK
    assert rope(n=0, Q=None, K=None, pos=None, Qo=None, Ko=None) == OK


@pytest.mark.parametrize("H,KV,hd", [(32, 8, 128), (3, 3, 64), (4, 1, 160)])
def test_workspace_sizes(H, KV, hd):
    """Enough keys and few rows want records; many rows, or too few keys to share out, want none; bad arguments say -1."""
    size = lambda ql, kl, **kw: lib.pkv_attn_cross_workspace(arr(ql), arr(kl), arr(kw.get("k0")), len(ql), H, KV, hd)
    per = 4 * H * (hd + 2)
    assert size((1,), (100_000,)) >= 2 * per
    assert size((1,), (200,)) == 0
    assert size((1, 1), (100_000, 50)) % 16 == 0
    assert size((1,), (-1,)) == -1 and lib.pkv_attn_cross_workspace(arr((1,)), arr((1,)), None, 1, 3, 2, hd) == -1
    pre = lambda P, ql, kl: lib.pkv_attn_prefix_workspace(P, arr(ql), arr(kl), len(ql), H, KV, hd)
    assert pre(40_000, (1, 1, 1), (3, 9, 1)) >= 2 * 3 * per   # own keys and the prefix apart
    assert pre(4000, (1, 1), (3, 9)) == 0                       # so small that clusters of blocks share the keys
    assert pre(4000, (2,), (1,)) == -1 and pre(-1, (1,), (1,)) == -1


def rope(n=5, H=4, KV=2, hd=16, dtype=pkv.PKV_BF16, pairs=(3, 3, 2), order=0, base=1e4, Q=4096, K=4096, Qo=8192, Ko=8192,
         pos=4096, ps=5, qs=64, ks=32, qos=64, kos=32, axes=None):
    return lib.pkv_rope_packed(Q, qs, K, ks, dtype, pos, ps, len(pairs) if axes is None else axes, arr(pairs), order, n, H, KV,
                               hd, base, 0, Qo, qos, Ko, kos, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), BAD_DIM), (dict(n=BIG), BAD_DIM), (dict(axes=0), BAD_DIM), (dict(axes=5), BAD_DIM), (dict(pairs=None, axes=1), BAD_DIM),
    (dict(pairs=(3, -1, 2)), BAD_DIM), (dict(pairs=(0, 0)), BAD_DIM), (dict(pairs=(5, 4)), BAD_DIM), (dict(H=0), BAD_DIM),
    (dict(KV=0), BAD_DIM), (dict(hd=0), BAD_DIM), (dict(hd=258, qs=5000, ks=5000, qos=5000, kos=5000), BAD_DIM),
    (dict(order=1, pairs=(1, 3, 4)), BAD_DIM),  # turns that do not come out at the axes' pairs
    (dict(dtype=3), ARG), (dict(order=3), ARG), (dict(order=-1), ARG), (dict(base=0.5), ARG), (dict(base=float("nan")), ARG),
    (dict(base=float("inf")), ARG), (dict(qs=63), ARG), (dict(ks=31), ARG), (dict(qos=63), ARG), (dict(kos=31), ARG),
    (dict(ps=4), ARG), (dict(qs=1 << 40), BAD_DIM), (dict(Q=None), ARG), (dict(Qo=None), ARG), (dict(K=None), ARG),
    (dict(Ko=None), ARG), (dict(Q=None, Qo=None, K=None, Ko=None), ARG), (dict(pos=None), ARG), (dict(pos=4098), ARG),
    (dict(Q=4097), ARG), (dict(Ko=4097), ARG), (dict(dtype=pkv.PKV_F32, Q=4098), ARG), (dict(Q=4096, Qo=4096, qos=72), ARG)], ids=str)
def test_rope_refuses(kw, rc):
    assert rope(**kw) == rc, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


def test_the_binding_refuses_host_tensors():
    x, pos = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkv.pkv_attn_cross(x, [4], x, x, [4], 4, 4, 16, 0.25, x)
    with pytest.raises(TypeError):
        pkv.pkv_attn_prefix(x, [4], x, x, x, x, [4], 4, 4, 16, 0.25, x)
    with pytest.raises(TypeError):
        pkv.pkv_rope_packed(x, x, pos, [3, 3, 2], 0, 4, 4, 16, 1e4, x, x)
    with pytest.raises(TypeError, match="entry for each"):
        pkv.pkv_attn_cross(x, [4], x, x, [4, 1], 4, 4, 16, 0.25, x)
    with pytest.raises(TypeError, match="entry for each"):
        pkv.pkv_attn_cross_workspace([4], [4], 4, 4, 16, k_start=[0, 1])


def test_the_binding_wants_the_current_device_and_one_type(monkeypatch):
    from test_q8_refusals import Rows

    class Space:
        nbytes = 64

        def __init__(self, device):
            self.device = device

        def is_contiguous(self):
            return True

        def get_device(self):
            return self.device

        def data_ptr(self):
            return 4096

    done = staticmethod(lambda *a: 0)
    monkeypatch.setattr(pkv, "_current_device", lambda: 0)
    monkeypatch.setattr(pkv, "_lib", type("Lib", (), {n: done for n in ("pkv_attn_cross", "pkv_attn_prefix", "pkv_rope_packed")}))

    def one(which, i, **kw):
        r = [Rows(9, w) for w in ((64, 32, 32, 64) if which == "cross" else (64, 32, 32, 32, 32, 64))]
        if i is not None:
            r[i] = Rows(9, kw.get("w", r[i].shape[1]), kw.get("device", 0), dtype=kw.get("dtype", torch.bfloat16))
        space = Space(kw.get("space", 0))
        if which == "cross":
            return pkv.pkv_attn_cross(r[0], [9], r[1], r[2], [9], 4, 2, 16, 0.25, r[3], workspace=space)
        return pkv.pkv_attn_prefix(r[0], [9], r[1], r[2], r[3], r[4], [9], 4, 2, 16, 0.25, r[5], workspace=space)

    for which, n in (("cross", 4), ("prefix", 6)):
        assert one(which, None) == 0
        with pytest.raises(TypeError, match="workspace"):
            one(which, None, space=1)
        for i in range(n):
            with pytest.raises(TypeError, match="device"):
                one(which, i, device=1)
            with pytest.raises(TypeError, match="type"):
                one(which, i, dtype=torch.float16)
            with pytest.raises(TypeError, match="wide"):
                one(which, i, w=48)

    def turn(q=Rows(9, 64), k=Rows(9, 32), qo=Rows(9, 64), ko=Rows(9, 32), pos=None, pairs=(3, 3, 2)):
        return pkv.pkv_rope_packed(q, k, pos or Rows(3, 9, dtype=torch.int32), list(pairs), 0, 4, 2, 16, 1e4, qo, ko)

    assert turn() == 0 and turn(q=None, qo=None) == 0 and turn(k=None, ko=None) == 0
    for kw in (dict(q=None), dict(qo=None), dict(k=None), dict(ko=None), dict(q=None, qo=None, k=None, ko=None),
               dict(q=Rows(8, 64)), dict(ko=Rows(8, 32)), dict(q=Rows(9, 60)), dict(q=Rows(9, 64, 1)),
               dict(ko=Rows(9, 32, dtype=torch.float32)), dict(pos=Rows(3, 9, dtype=torch.int64)), dict(pos=Rows(2, 9, dtype=torch.int32)),
               dict(pos=Rows(3, 9, 1, dtype=torch.int32)), dict(pos=Rows(3, 10, dtype=torch.int32))):
        with pytest.raises(TypeError):
            turn(**kw)

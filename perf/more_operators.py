"""Cases of the multi-axis rotary, cross-attention and shared-prefix operators, their plain forms and their exact values.

Three kinds of case:

* ``rope``    rotary positions with several axes (time, height, width) on packed query and key rows, forth or back
  (back is also the gradient): ``pkv_rope_packed``.
* ``cross``   attention of packed queries over an encoder's rows of other lengths (bf16 / f16, grouped heads), whole
  prompts and single tokens: ``pkv_attn_cross``.
* ``prefix``  attention of a batch whose sequences share one long prefix and have keys of their own behind it, prompts
  and single tokens: ``pkv_attn_prefix``.
"""
import ctypes
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ORDERS = {"blocks": 0, "turns": 1, "axial": 2}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one decode step of a batch of image-and-text chats: all launch latency
        dict(name="rope_step_m64", op="rope", n=64, heads=32, kv=8, hd=128, dtype="bf16", order="blocks", pairs="16,24,24",
             base=1000000.0, inverse=False, fused=True, pos_hi=9000),
        # a long video prompt, query and key columns of one projection's output, frequencies dealt to the axes in turn
        dict(name="rope_video", op="rope", n=16384, heads=32, kv=8, hd=128, dtype="bf16", order="turns", pairs="24,20,20",
             base=500000.0, inverse=False, fused=True, pos_hi=40000),
        # the gradient of an image encoder's patches (height and width, a ramp of frequencies each), an odd number of them
        dict(name="rope_patches_back", op="rope", n=2111, heads=16, kv=16, hd=80, dtype="f32", order="axial", pairs="20,20",
             base=10000.0, inverse=True, fused=False, pos_hi=90),
        # one token of one request over half a minute of audio: what a transcription step costs, all launch latency
        dict(name="cross_one_token", op="cross", n=1, q_lo=1, q_hi=1, k_lo=1500, k_hi=1500, lens_seed=1, heads=20, kv=20,
             hd=64, dtype="f16", slots=False, none=False),
        # a decode step of a batch over images of different sizes, in slots of a cache
        dict(name="cross_step_m64", op="cross", n=64, q_lo=1, q_hi=1, k_lo=200, k_hi=6000, lens_seed=2, heads=32, kv=8,
             hd=128, dtype="bf16", slots=True, none=False),
        # a decode step of a few requests over long documents
        dict(name="cross_step_long", op="cross", n=3, q_lo=1, q_hi=1, k_lo=50000, k_hi=120000, lens_seed=3, heads=32, kv=8,
             hd=128, dtype="bf16", slots=False, none=False),
        # prompts of a transcription batch
        dict(name="cross_prompts", op="cross", n=24, q_lo=4, q_hi=448, k_lo=700, k_hi=1500, lens_seed=4, heads=20, kv=20,
             hd=64, dtype="bf16", slots=False, none=False),
        # long texts over long encoder outputs
        dict(name="cross_long", op="cross", n=2, q_lo=4000, q_hi=4100, k_lo=8000, k_hi=8300, lens_seed=5, heads=32, kv=8,
             hd=128, dtype="f16", slots=False, none=False),
        # a decode step of a few samples of one question
        dict(name="prefix_step_few", op="prefix", n=5, prefix=2000, q_lo=1, q_hi=1, past_lo=1, past_hi=90, lens_seed=6,
             heads=32, kv=8, hd=128, dtype="bf16", slots=True),
        # a decode step of a batch behind one system prompt
        dict(name="prefix_step_m64", op="prefix", n=64, prefix=8192, q_lo=1, q_hi=1, past_lo=10, past_hi=700, lens_seed=7,
             heads=32, kv=8, hd=128, dtype="bf16", slots=True),
        # the users' prompts of a prefill batch behind one system prompt
        dict(name="prefix_prompts", op="prefix", n=32, prefix=4099, q_lo=16, q_hi=700, past_lo=0, past_hi=0, lens_seed=8,
             heads=32, kv=8, hd=128, dtype="bf16", slots=False),
        # many short answers scored behind one question, a group that is no power of two
        dict(name="prefix_answers", op="prefix", n=300, prefix=1100, q_lo=2, q_hi=24, past_lo=0, past_hi=0, lens_seed=9,
             heads=28, kv=4, hd=128, dtype="f16", slots=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "cross", "cross", "prefix", "prefix"])
    if op == "rope":
        heads, kv, hd, order, pairs = rng.choice([
            (32, 8, 128, "blocks", "16,24,24"), (16, 2, 128, "turns", "24,20,20"), (28, 4, 128, "blocks", "16,24,24"),
            (16, 16, 80, "axial", "20,20"), (12, 12, 64, "axial", "10,10,12"), (16, 16, 72, "axial", "18,18"),
            (8, 8, 64, "blocks", "8,4,4"), (40, 8, 128, "blocks", "64"), (5, 5, 96, "turns", "16,16,16")])
        return dict(op=op, n=_log_int(rng, 1, 16384), heads=heads, kv=kv, hd=hd, dtype=rng.choice(["bf16", "f16", "f32"]),
                    order=order, pairs=pairs, base=rng.choice([10000.0, 500000.0, 1000000.0]), inverse=rng.random() < 0.4,
                    fused=rng.random() < 0.5, pos_hi=_log_int(rng, 4, 200_000))
    heads, kv, hd = rng.choice([(32, 8, 128), (16, 2, 128), (20, 20, 64), (28, 4, 128), (12, 12, 80), (15, 3, 96),
                                (64, 8, 128), (10, 1, 64), (8, 4, 40), (6, 2, 160)])
    c = dict(op=op, lens_seed=rng.randrange(1 << 20), heads=heads, kv=kv, hd=hd, dtype=rng.choice(["bf16", "f16"]),
             slots=rng.random() < 0.5)
    few = rng.random() < 0.5
    wide = 2.0e10 if hd <= 128 else 4.0e9  # score elements times head width that a drawn case may cost
    if op == "cross":
        q_hi = rng.choice([1, 1, 2, 5]) if few else _log_int(rng, 8, 3000)
        k_hi = _log_int(rng, 20, 60_000 if few else 6000)
        per = max(1.0, q_hi * float(k_hi) * heads * hd)
        top = max(1, min(128, int(wide * 16 / per), int(400_000 / (k_hi + q_hi))))
        n = _log_int(rng, 1, top)
        return dict(c, n=n, q_lo=q_hi if few else _log_int(rng, 1, q_hi), q_hi=q_hi, k_lo=_log_int(rng, 1, k_hi), k_hi=k_hi,
                    none=n > 2 and rng.random() < 0.3)
    prefix = _log_int(rng, 100, 16_000)
    q_hi = rng.choice([1, 1, 2, 4]) if few else _log_int(rng, 6, 1500)
    past = _log_int(rng, 1, 4000) if few else rng.choice([0, 0, 300])
    per = max(1.0, q_hi * float(prefix + past + q_hi) * heads * hd)
    top = max(1, min(200, int(wide * 16 / per), int(200_000 / (past + q_hi))))
    return dict(c, n=_log_int(rng, 1, top), prefix=prefix, q_lo=q_hi if few else _log_int(rng, 1, q_hi), q_hi=q_hi,
                past_lo=min(past, 1), past_hi=past)


def _lengths(n, lo, hi, seed):
    """n lengths, log-uniform in [lo, hi] (0 counts as below 1)."""
    r = np.random.RandomState(seed)
    if hi <= 0:
        return np.zeros(n, dtype=np.int64)
    v = np.exp(r.uniform(math.log(max(lo, 0.5)), math.log(hi + 0.5), size=n))
    return np.clip(np.rint(v), lo, hi).astype(np.int64)


def _lens(case):
    """Queries and keys of their own of every sequence."""
    q = _lengths(case["n"], case["q_lo"], case["q_hi"], case["lens_seed"])
    if case["op"] == "prefix":
        return q, q + _lengths(case["n"], case["past_lo"], case["past_hi"], case["lens_seed"] + 1)
    k = _lengths(case["n"], case["k_lo"], case["k_hi"], case["lens_seed"] + 1)
    if case["none"]:
        k[case["n"] // 2] = 0  # a request without an encoder's states
    return q, k


def _pairs(case):
    return [int(x) for x in case["pairs"].split(",")]


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    h, kv, hd = case["heads"], case["kv"], case["hd"]
    if case["op"] == "rope":
        t, width = float(case["n"]), (h + kv) * hd
        return {"bytes": 2 * t * width * e + 4 * t * len(_pairs(case)), "flops": 3 * t * width}
    q, k = (x.astype(float) for x in _lens(case))
    shared = float(case.get("prefix", 0))
    seen = q * k if case["op"] == "cross" else q * shared + q * (k - q) + q * (q + 1) / 2
    return {"bytes": e * (2.0 * float(q.sum()) * h * hd + 2.0 * (float(k.sum()) + shared) * kv * hd),
            "flops": 4.0 * hd * h * float(seen.sum())}


# ----------------------------------------------------------------- inputs ----

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _index(values):
    return torch.from_numpy(np.ascontiguousarray(values, dtype=np.int64)).cuda()


def _positions(case, seed):
    """[axes, n] positions below pos_hi: runs of text (all axes alike) and grids of patches."""
    r = np.random.RandomState(seed % (1 << 31))
    axes, n = len(_pairs(case)), case["n"]
    side = max(2, min(48, case["pos_hi"] // 2))
    place = np.arange(n) + int(r.randint(0, 1 << 16))
    grid = np.stack([place // (side * side), place // side % side, place % side])[3 - axes:]
    text = (place // 997) % 2 == 0
    pos = np.where(text[None, :] if axes == 3 else False, place[None, :], grid + int(r.randint(0, case["pos_hi"])))
    return (pos % case["pos_hi"]).astype(np.int32)


def _columns(g, rows, widths, dtype, fused):
    """Random rows of the given widths, side by side in one tensor where fused."""
    if not fused:
        return [torch.randn(rows, w, device="cuda", generator=g).to(dtype) for w in widths]
    x = torch.randn(rows, sum(widths), device="cuda", generator=g).to(dtype)
    return list(x.split(widths, dim=1))


def _inputs(case, seed):
    g, dt = _generator(seed), DTYPES[case["dtype"]]
    qd, kd = case["heads"] * case["hd"], case["kv"] * case["hd"]
    if case["op"] == "rope":
        q, k = _columns(g, case["n"], [qd, kd], dt, case["fused"])
        return {"q": q, "k": k, "pos": torch.from_numpy(_positions(case, seed)).cuda()}
    ql, kl = _lens(case)
    if case["slots"]:  # a slot of the same size for every sequence
        room = int(kl.max()) + 7
        start, rows = np.arange(case["n"]) * room, case["n"] * room
    else:
        start, rows = np.concatenate([[0], np.cumsum(kl)[:-1]]), int(kl.sum())
    s = {"ql": [int(x) for x in ql], "kl": [int(x) for x in kl], "start": [int(x) for x in start]}
    s["q"], = _columns(g, int(ql.sum()), [qd], dt, False)
    s["k"], s["v"] = _columns(g, max(rows, 1), [kd, kd], dt, True)
    if case["op"] == "prefix":
        s["kp"], s["vp"] = _columns(g, case["prefix"], [kd, kd], dt, True)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "rope":
        s["q_out"], s["k_out"] = torch.empty_like(s["q"], memory_format=torch.contiguous_format), torch.empty_like(
            s["k"], memory_format=torch.contiguous_format)
        return s
    # the batch's plan: places of its rows in a padded batch, and the lengths as the calls take them
    ql, kl, start = (np.asarray(s[x], dtype=np.int64) for x in ("ql", "kl", "start"))
    first = np.concatenate([[0], np.cumsum(ql)[:-1]])
    place = np.arange(max(int(ql.max()), 1))
    there = place[None, :] < ql[:, None]
    s["q_at"] = _index(np.where(there, first[:, None] + place[None, :], 0))
    s["back"] = _index(np.flatnonzero(there.reshape(-1)))
    place = np.arange(max(int(kl.max()), 1))
    s["k_at"] = _index(np.where(place[None, :] < kl[:, None], start[:, None] + place[None, :], 0))
    s["ql_dev"], s["kl_dev"] = _index(ql), _index(kl)
    s["n_q"], s["n_k"], s["k0"] = ((ctypes.c_int32 * len(s[x]))(*s[x]) for x in ("ql", "kl", "start"))
    s["out"] = torch.empty_like(s["q"])
    if own:
        import paged_kv_gqa_nx_gb300 as pkv
        heads = (case["heads"], case["kv"], case["hd"])
        n = (pkv.pkv_attn_cross_workspace(s["n_q"], s["n_k"], *heads, k_start=s["k0"]) if case["op"] == "cross" else
             pkv.pkv_attn_prefix_workspace(case["prefix"], s["n_q"], s["n_k"], *heads, k_start=s["k0"]))
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------ plain forms ----

def _axis_of_pairs(order, pairs):
    """Axis of every frequency pair, and its number among the pairs of its ramp."""
    n = sum(pairs)
    i = np.arange(n)
    if order == "turns":
        a = i % len(pairs)
        return np.where(i < len(pairs) * np.asarray(pairs)[a], a, 0), i
    axis = np.repeat(np.arange(len(pairs)), pairs)
    return axis, i - (np.cumsum(pairs) - pairs)[axis] if order == "axial" else i


def _plain_rope(s):
    c = s["case"]
    pairs, hd = _pairs(c), c["hd"]
    axis, number = _axis_of_pairs(c["order"], pairs)
    ramp = np.asarray(pairs)[axis] if c["order"] == "axial" else sum(pairs)
    freq = torch.from_numpy(c["base"] ** (-number / ramp)).cuda()
    angle = s["pos"].double()[_index(axis)].t() * freq  # far positions: 64 bits
    if c["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = sum(pairs)
    out = {}
    for name in ("q", "k"):
        x = s[name].float().view(s[name].shape[0], -1, hd)
        a, b = x[..., :r], x[..., r:2 * r]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos, x[..., 2 * r:]], dim=-1)
        out[name] = y.reshape(s[name].shape).to(s[name].dtype)
    return out


def _softmax_rows(x):
    """exp(x - max) / sum in place over the last dimension; rows of -inf give zeros."""
    x -= x.amax(dim=-1, keepdim=True).clamp_min(-1e30)
    x.exp_()
    x /= x.sum(dim=-1, keepdim=True).clamp_min(1e-30)
    return x


def _plain_attend(s):
    c = s["case"]
    h, kv, hd = c["heads"], c["kv"], c["hd"]
    (b, tq), tk = s["q_at"].shape, s["k_at"].shape[1]
    g = h // kv
    q = s["q"].float()[s["q_at"]].view(b, tq, kv, g, hd).permute(0, 2, 3, 1, 4) * float(np.float32(hd ** -0.5))
    k = s["k"].float()[s["k_at"]].view(b, tk, kv, hd).permute(0, 2, 3, 1)
    place = torch.arange(tk, device=q.device)
    if c["op"] == "cross":
        hidden = (place[None, None, :] >= s["kl_dev"][:, None, None]).expand(b, tq, tk)
    else:
        last = (s["kl_dev"] - s["ql_dev"])[:, None] + torch.arange(tq, device=q.device)[None, :]
        hidden = place[None, None, :] > last[:, :, None]
    p = c.get("prefix", 0)
    x = torch.empty(b, kv, g, tq, p + tk, device=q.device)
    x[..., p:] = torch.matmul(q.reshape(b, kv, g * tq, hd), k).view(b, kv, g, tq, tk)
    x[..., p:].masked_fill_(hidden[:, None, None], -math.inf)
    del k
    if p:  # the prefix, once for all sequences
        qs = q.permute(1, 0, 2, 3, 4).reshape(kv, b * g * tq, hd)
        kp = s["kp"].float().view(p, kv, hd).permute(1, 2, 0)
        x[..., :p] = torch.matmul(qs, kp).view(kv, b, g, tq, p).transpose(0, 1)
        del qs, kp
    _softmax_rows(x)
    v = s["v"].float()[s["k_at"]].view(b, tk, kv, hd).transpose(1, 2)
    o = torch.matmul(x[..., p:].reshape(b, kv, g * tq, tk), v).view(b, kv, g, tq, hd)
    if p:
        vp = s["vp"].float().view(p, kv, hd).transpose(0, 1)
        o += torch.matmul(x[..., :p].transpose(0, 1).reshape(kv, b * g * tq, p), vp).view(kv, b, g, tq, hd).transpose(0, 1)
    return o.permute(0, 3, 1, 2, 4).reshape(b * tq, h * hd)[s["back"]].to(s["q"].dtype)


# -------------------------------------------------------------------- run ----

def run(s):
    c = s["case"]
    if not own:
        return _plain_rope(s) if c["op"] == "rope" else _plain_attend(s)
    import paged_kv_gqa_nx_gb300 as pkv
    h, kv, hd, stream = c["heads"], c["kv"], c["hd"], torch.cuda.current_stream()
    if c["op"] == "rope":
        pkv.check(pkv.pkv_rope_packed(s["q"], s["k"], s["pos"], _pairs(c), ORDERS[c["order"]], h, kv, hd, c["base"],
                                      s["q_out"], s["k_out"], inverse=c["inverse"], stream=stream))
        return {"q": s["q_out"], "k": s["k_out"]}
    if c["op"] == "cross":
        pkv.check(pkv.pkv_attn_cross(s["q"], s["n_q"], s["k"], s["v"], s["n_k"], h, kv, hd, hd ** -0.5, s["out"],
                                     k_start=s["k0"], workspace=s["workspace"], stream=stream))
        return s["out"]
    pkv.check(pkv.pkv_attn_prefix(s["q"], s["n_q"], s["kp"], s["vp"], s["k"], s["v"], s["n_k"], h, kv, hd, hd ** -0.5,
                                  s["out"], k_start=s["k0"], workspace=s["workspace"], stream=stream))
    return s["out"]


# ------------------------------------------------------------ exact values ----

def _exact_rope(case, d):
    pairs, hd = _pairs(case), case["hd"]
    total, axes = sum(pairs), len(pairs)
    axis, exponent = [], []
    for i in range(total):
        if case["order"] == "turns":
            a = i % axes
            axis.append(a if i < axes * pairs[a] else 0)
            exponent.append(2.0 * i / (2 * total))
        else:
            a = next(a for a in range(axes) if i < sum(pairs[:a + 1]))
            axis.append(a)
            exponent.append(2.0 * (i - sum(pairs[:a])) / (2 * pairs[a]) if case["order"] == "axial" else 2.0 * i / (2 * total))
    pos = d["pos"].double()
    turn = torch.stack([pos[a] * case["base"] ** -e for a, e in zip(axis, exponent)], dim=1)
    w = torch.polar(torch.ones_like(turn), -turn if case["inverse"] else turn)[:, None]
    out = {}
    for name in ("q", "k"):
        x = d[name].double().reshape(case["n"], -1, hd).clone()
        z = torch.complex(x[..., :total].contiguous(), x[..., total:2 * total].contiguous()) * w
        x[..., :total], x[..., total:2 * total] = z.real, z.imag
        out[name] = x.view(case["n"], -1)
    return out


def exact(case, seed):
    if case["op"] == "rope":
        return _exact_rope(case, _inputs(case, seed))
    if work(case)["flops"] > 1.5e12:
        return None
    d = _inputs(case, seed)
    h, kv, hd = case["heads"], case["kv"], case["hd"]
    g = h // kv
    out = torch.zeros(d["q"].shape[0], kv, g, hd, dtype=torch.float64, device="cuda")
    pre = [d[w].double().view(-1, kv, hd) for w in ("kp", "vp")] if case["op"] == "prefix" else None
    at = 0
    for n, m, k0 in zip(d["ql"], d["kl"], d["start"]):
        kk, vv = (d[w][k0:k0 + m].double().view(m, kv, hd) for w in ("k", "v"))
        seen = torch.full((n,), m, device="cuda")
        if pre is not None:
            kk, vv = torch.cat([pre[0], kk]), torch.cat([pre[1], vv])
            seen = case["prefix"] + m - n + 1 + torch.arange(n, device="cuda")
        if n and kk.shape[0]:
            q = d["q"][at:at + n].double().view(n, kv, g, hd)
            for j in range(kv):
                x = torch.einsum("ngd,md->ngm", q[:, j], kk[:, j]) * hd ** -0.5
                x.masked_fill_((torch.arange(kk.shape[0], device="cuda")[None, :] >= seen[:, None])[:, None], -math.inf)
                out[at:at + n, j] = torch.einsum("ngm,md->ngd", torch.softmax(x, dim=-1), vv[:, j])
        at += n
    return out.view(-1, h * hd)

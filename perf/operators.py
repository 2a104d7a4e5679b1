"""Cases of the packed-prompt and 8-bit-cache operators, their plain forms and their exact values.

Three kinds of case:

* ``packed``  attention over whole prompts of different lengths that lie behind one another (bf16 / f16, grouped
  heads, causal or not): ``pkv_attn_packed``.
* ``append``  K / V rows written into the pages of an 8-bit cache with a power-of-two scale for each block of tokens
  and kv head, then read back as the values they stand for: ``pkv_append_packed``, ``pkv_read_packed``.
* ``q8``      append + offset-causal attention over such a cache for a batch of sequences (decode rows, short chunks,
  prefill chunks): ``pkv_attn_batch`` on a ``pkv_pool_new_q8`` pool.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one short prompt: what a single chat turn costs, all launch latency
        dict(name="packed_one_short", op="packed", n=1, lo=23, hi=23, lens_seed=1, heads=32, kv=8, hd=128, dtype="bf16",
             causal=True, fused=False),
        # a prefill batch of a server: prompts of very different lengths
        dict(name="packed_ragged", op="packed", n=24, lo=16, hi=4096, lens_seed=2, heads=32, kv=8, hd=128, dtype="bf16",
             causal=True, fused=True),
        # one long document
        dict(name="packed_long", op="packed", n=1, lo=16384, hi=16384, lens_seed=3, heads=32, kv=8, hd=128, dtype="f16",
             causal=True, fused=False),
        # narrow heads without grouping, both directions visible (an embedding model), q, k, v in one projection's output
        dict(name="packed_hd64_full", op="packed", n=16, lo=64, hi=1024, lens_seed=4, heads=20, kv=20, hd=64,
             dtype="bf16", causal=False, fused=True),
        # a group that is no power of two and a head width between the tile widths
        dict(name="packed_group7_hd96", op="packed", n=6, lo=1, hi=1500, lens_seed=5, heads=28, kv=4, hd=96,
             dtype="f16", causal=True, fused=False),
        # the rows of one decode step go into half-filled pages
        dict(name="append_step_m64", op="append", n=64, lo=1, hi=1, lens_seed=6, past_lo=1, past_hi=200, kv=8, hd=128,
             bs=16, dtype="f32", fused=False),
        # prompts of a prefill batch, k and v side by side in one projection's output
        dict(name="append_prompts", op="append", n=16, lo=1, hi=3000, lens_seed=7, past_lo=0, past_hi=40, kv=8, hd=128,
             bs=16, dtype="bf16", fused=True),
        # long documents
        dict(name="append_long", op="append", n=8, lo=16000, hi=16384, lens_seed=8, past_lo=0, past_hi=0, kv=8, hd=128,
             bs=16, dtype="bf16", fused=False),
        # one sequence decoding alone
        dict(name="q8_decode_one", op="q8", n=1, past_lo=700, past_hi=700, lens_seed=9, nq=1, heads=32, kv=8, hd=128,
             bs=16, causal=True),
        # the batched-decode workload
        dict(name="q8_decode_m64", op="q8", n=64, past_lo=512, past_hi=4096, lens_seed=10, nq=1, heads=32, kv=8, hd=128,
             bs=16, causal=True),
        # the continuous-batching workload: lengths log-uniform in [128, 32768]
        dict(name="q8_decode_m256", op="q8", n=256, past_lo=128, past_hi=32768, lens_seed=11, nq=1, heads=32, kv=8,
             hd=128, bs=16, causal=True),
        # the chunked-prefill workload, one layer
        dict(name="q8_chunk_512", op="q8", n=8, past_lo=2048, past_hi=2048, lens_seed=12, nq=512, heads=32, kv=8,
             hd=128, bs=16, causal=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed", "append", "q8", "q8"])
    seed = rng.randrange(1 << 20)
    if op == "packed":
        heads, kv, hd = rng.choice([(32, 8, 128), (16, 2, 128), (8, 8, 64), (28, 4, 128), (12, 12, 80), (15, 3, 96),
                                    (64, 8, 128), (10, 1, 64), (4, 2, 32)])
        hi = _log_int(rng, 1, 6000)
        n = _log_int(rng, 1, max(1, min(64, 40_000 // hi)))
        return dict(op=op, n=n, lo=_log_int(rng, 1, hi), hi=hi, lens_seed=seed, heads=heads, kv=kv, hd=hd,
                    dtype=rng.choice(["bf16", "f16"]), causal=rng.random() < 0.75, fused=rng.random() < 0.5)
    kv, hd = rng.choice([(8, 128), (2, 128), (4, 64), (1, 64), (3, 96), (5, 80), (16, 128)])
    bs = rng.choice([16, 16, 32, 64, 8, 5, 100])
    if op == "append":
        hi = _log_int(rng, 1, 12_000)
        return dict(op=op, n=_log_int(rng, 1, max(1, min(200, 100_000 // hi))), lo=_log_int(rng, 1, hi), hi=hi,
                    lens_seed=seed, past_lo=0, past_hi=_log_int(rng, 1, 300), kv=kv, hd=hd, bs=bs,
                    dtype=rng.choice(["bf16", "f16", "f32"]), fused=rng.random() < 0.5)
    nq = rng.choice([1, 1, 1, 2, 4, 7, 40, 300])
    hi = _log_int(rng, 1, 20_000 if nq < 32 else 3000)
    return dict(op=op, n=_log_int(rng, 1, max(1, min(128 if nq == 1 else 16, 600_000 // (hi + nq)))),
                past_lo=_log_int(rng, 1, hi), past_hi=hi, lens_seed=seed, nq=nq, heads=kv * rng.choice([1, 2, 4, 8, 5]),
                kv=kv, hd=hd, bs=bs, causal=rng.random() < 0.9)


def _lengths(n, lo, hi, seed):
    """n lengths, log-uniform in [lo, hi] (0 counts as below 1)."""
    r = np.random.RandomState(seed)
    if hi <= 0:
        return np.zeros(n, dtype=np.int64)
    v = np.exp(r.uniform(math.log(max(lo, 0.5)), math.log(hi + 0.5), size=n))
    return np.clip(np.rint(v), lo, hi).astype(np.int64)


def _lens(case):
    return _lengths(case["n"], case["lo"], case["hi"], case["lens_seed"])


def _pasts(case):
    return _lengths(case["n"], case["past_lo"], case["past_hi"], case["lens_seed"] + 1)


def work(case):
    if case["op"] == "packed":
        L = _lens(case).astype(float)
        e, t = 2, float(L.sum())
        pairs = float((L * (L + 1) / 2 if case["causal"] else L * L).sum())
        return {"bytes": t * (2 * case["heads"] + 2 * case["kv"]) * case["hd"] * e,
                "flops": 4.0 * case["hd"] * case["heads"] * pairs}
    kv_dim = case["kv"] * case["hd"]
    if case["op"] == "append":
        t, e = float(_lens(case).sum()), 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * t * kv_dim * (e + 1 + 1 + e), "flops": 2 * t * kv_dim * 4.0}
    past, nq = _pasts(case).astype(float), case["nq"]
    t = float(nq * case["n"])
    pairs = float((nq * past + nq * (nq + 1) / 2 if case["causal"] else nq * (past + nq)).sum())
    return {"bytes": 2.0 * kv_dim * float((past + nq).sum()) + t * (2 * 4 * case["heads"] * case["hd"] + 2 * 4 * kv_dim),
            "flops": 4.0 * case["hd"] * case["heads"] * pairs}


# ----------------------------------------------------------------- inputs ----

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _index(values):
    return torch.from_numpy(np.ascontiguousarray(values, dtype=np.int64)).cuda()


def _packed_inputs(case, seed):
    g, lens = _generator(seed), _lens(case)
    t, qd, kd = int(lens.sum()), case["heads"] * case["hd"], case["kv"] * case["hd"]
    dt = DTYPES[case["dtype"]]
    if case["fused"]:  # columns of one projection's output
        x = torch.randn(t, qd + 2 * kd, device="cuda", generator=g).to(dt)
        q, k, v = x[:, :qd], x[:, qd:qd + kd], x[:, qd + kd:]
    else:
        q, k, v = (torch.randn(t, d, device="cuda", generator=g).to(dt) for d in (qd, kd, kd))
    return {"q": q, "k": k, "v": v, "lens": [int(x) for x in lens]}


def _cache_inputs(case, seed, past, new, q_dim):
    """A shuffled pool whose sequences hold `past` tokens, and `new` rows for each."""
    g = _generator(seed)
    bs, kd = case["bs"], case["kv"] * case["hd"]
    pages = -(-(past + new) // bs)
    n_blocks = int(pages.sum()) + 3
    # allocating every block and giving them back in this order shuffles the free list: the last one given back comes first
    given = np.random.RandomState(case["lens_seed"] + 2).permutation(n_blocks)
    taken = given[::-1]
    first = np.concatenate([[0], np.cumsum(pages)])
    d = {"n_blocks": n_blocks, "given": given, "past": [int(x) for x in past], "new": [int(x) for x in new],
         "max_blocks": int(pages.max())}
    table = np.zeros((len(past), d["max_blocks"]), dtype=np.int64)
    for r in range(len(past)):
        table[r, :pages[r]] = taken[first[r]:first[r + 1]]
    d["table"] = table
    # a history of about N(0, 1) values: elements around 32 steps, steps of 2^-6 .. 2^-4
    for which in ("k", "v"):
        pool = torch.empty(n_blocks, 1, bs, kd, dtype=torch.uint8, device="cuda")
        flat = pool.view(-1)
        step = 1 << 28
        for at in range(0, flat.numel(), step):
            part = flat[at:at + step]
            part.copy_(torch.randn(part.numel(), device="cuda", generator=g).mul_(32.0).round_().clamp_(-127.0, 127.0)
                       .add_(128.0))
        e = torch.randint(-6, -3, (n_blocks, 1, case["kv"]), device="cuda", generator=g)
        d[which + "_pool"], d[which + "_scale"] = pool, torch.exp2(e.float())
    t, dt = int(new.sum()), DTYPES[case.get("dtype", "f32")]
    if case.get("fused"):
        x = torch.randn(t, 2 * kd, device="cuda", generator=g).mul_(1.5).to(dt)
        d["k"], d["v"] = x[:, :kd], x[:, kd:]
    else:
        d["k"], d["v"] = (torch.randn(t, kd, device="cuda", generator=g).mul_(1.5).to(dt) for _ in range(2))
    if q_dim:
        d["q"] = torch.randn(t, q_dim, device="cuda", generator=g)
    return d


def _inputs(case, seed):
    if case["op"] == "packed":
        return _packed_inputs(case, seed)
    past = _pasts(case)
    if case["op"] == "append":
        return _cache_inputs(case, seed, past, _lens(case), 0)
    return _cache_inputs(case, seed, past, np.full(case["n"], case["nq"], dtype=np.int64), case["heads"] * case["hd"])


class _Handle:
    """A pool with its sequences, as a server keeps them; released with the state."""

    def __init__(self, pkv, pool):
        self.pkv, self.pool, self.seqs = pkv, pool, []

    def __del__(self):
        if self.pool:
            self.pkv.pkv_pool_free(self.pool)
            self.pool = None


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "packed":
        if not own:
            lens = np.asarray(s["lens"])
            s["at"], s["valid"], s["back"] = _pad_plan(lens)
        else:
            import paged_kv_gqa_nx_gb300 as pkv
            s["pkv"], s["n_dev"] = pkv, pkv.i32_array(s["lens"])
            s["out"] = torch.empty(s["q"].shape[0], s["q"].shape[1], dtype=s["q"].dtype, device="cuda")
        return s
    if not own:
        s.update(_append_plan(s, case["bs"]))
        if case["op"] == "q8":
            s["table_dev"] = _index(s["table"])
            s["past_dev"] = _index(s["past"])
        return s
    import paged_kv_gqa_nx_gb300 as pkv
    pool = pkv.pkv_pool_new_q8(s["n_blocks"], 1, case["kv"], case["hd"], case["bs"], s["k_pool"], s["v_pool"], s["k_scale"],
                               s["v_scale"], len(s["past"]), s["max_blocks"], torch.cuda.current_stream())
    if not pool:
        raise RuntimeError(pkv.pkv_last_error())
    h = s["handle"] = _Handle(pkv, pool)
    for _ in range(s["n_blocks"]):
        pkv.pkv_alloc_block(pool)
    for b in s["given"].tolist():
        pkv.pkv_unref_block(pool, b)
    for p, n in zip(s["past"], s["new"]):
        q = pkv.pkv_seq_new(pool, p + n)
        pkv.check(pkv.pkv_ensure_append(q, p + n))
        if p:
            pkv.check(pkv.pkv_advance(q, p))
        h.seqs.append(q)
    s["pkv"], s["seqs"], s["n_new"] = pkv, pkv.seq_array(h.seqs), pkv.i32_array(s["new"])
    t, kd = s["k"].shape
    if case["op"] == "append":
        s["start"] = pkv.i32_array(s["past"])
        s["k_out"], s["v_out"] = (torch.empty(t, kd, dtype=s["k"].dtype, device="cuda") for _ in range(2))
    else:
        s["out"] = torch.empty(t, case["heads"] * case["hd"], device="cuda")
    pkv.check(pkv.pkv_pool_flush(pool))
    return s


# ------------------------------------------------------------ plain forms ----

def _pad_plan(lens):
    """Packed rows <-> a padded batch: row of (sequence, position), which positions exist, and the way back."""
    b, top = len(lens), int(lens.max())
    start = np.concatenate([[0], np.cumsum(lens)])[:-1]
    at = start[:, None] + np.arange(top)[None, :]
    valid = np.arange(top)[None, :] < lens[:, None]
    back = np.flatnonzero(valid.reshape(-1))
    return _index(np.where(valid, at, 0)), torch.from_numpy(valid).cuda(), _index(back)


def _append_plan(s, bs):
    """The pages that the new rows fall in: block, rows kept before them, and the source row of each place of the page."""
    blk, keep, src, new = [], [], [], []
    row0 = 0
    for r, (p, n) in enumerate(zip(s["past"], s["new"])):
        pos = np.arange(p // bs, (p + n - 1) // bs + 1)[:, None] * bs + np.arange(bs)[None, :]
        blk.append(s["table"][r, p // bs:(p + n - 1) // bs + 1])
        keep.append(np.clip(p - pos[:, 0], 0, bs))
        new.append((pos >= p) & (pos < p + n))
        src.append(np.clip(row0 + pos - p, row0, row0 + n - 1))
        row0 += n
    new = np.concatenate(new)
    return {"blk": _index(np.concatenate(blk)), "keep": _index(np.concatenate(keep)), "src": _index(np.concatenate(src)),
            "is_new": torch.from_numpy(new).cuda(), "back": _index(np.flatnonzero(new.reshape(-1)))}


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _exponent(x):
    """The exponent of a power of two."""
    return (x.view(torch.int32) >> 23) - 127


def _quantise(s, which, kv, hd):
    """The plain append: the touched pages' new elements and scales, stored into the pool. Values of the pages come back."""
    pool, scale, x = s[which + "_pool"], s[which + "_scale"], s[which]
    new = s["is_new"][:, :, None, None]
    x = x.float()[s["src"]].view(s["src"].shape + (kv, hd))
    x = torch.where(new, x, torch.zeros_like(x))
    f, e = torch.frexp(x.abs().amax(dim=(1, 3)))
    need = torch.where(f <= 127.0 / 128.0, e - 7, e - 6)
    need = torch.where(f > 0, need, torch.full_like(need, -126)).clamp_min(-126)
    old_e = _exponent(scale[s["blk"], 0])
    top = torch.where(s["keep"][:, None] > 0, torch.maximum(old_e, need), need)
    kept = pool[s["blk"], 0].view(x.shape).float() - 128.0
    shift = _pow2((old_e - top).clamp(-126, 0))[:, None, :, None]
    kept = torch.where((s["keep"][:, None] > 0)[:, :, None, None], torch.round(kept * shift), kept)
    place = torch.arange(x.shape[1], device=x.device)[None, :] < s["keep"][:, None]
    q = torch.where(new, torch.round(x * _pow2(-top)[:, None, :, None]), kept)
    write = (s["is_new"] | place)[:, :, None, None]
    stored = torch.where(write, (q + 128.0).to(torch.uint8), pool[s["blk"], 0].view(x.shape))
    pool[s["blk"], 0] = stored.view(x.shape[0], x.shape[1], kv * hd)
    step = _pow2(top)
    scale[s["blk"], 0] = step
    return (stored.float() - 128.0) * step[:, None, :, None]


def _softmax_rows(x):
    """exp(x - max) / sum in place over the last dimension."""
    x -= x.amax(dim=-1, keepdim=True)
    x.exp_()
    x /= x.sum(dim=-1, keepdim=True)
    return x


def _plain_packed(s):
    c = s["case"]
    h, kv, hd = c["heads"], c["kv"], c["hd"]
    b, top = s["at"].shape
    q = s["q"].float()[s["at"]].view(b, top, kv, h // kv, hd).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, hd)
    k = s["k"].float()[s["at"]].view(b, top, kv, hd).permute(0, 2, 3, 1)
    v = s["v"].float()[s["at"]].view(b, top, kv, hd).permute(0, 2, 1, 3)
    x = torch.matmul(q * float(np.float32(hd ** -0.5)), k).view(b, kv, h // kv, top, top)
    hidden = ~s["valid"][:, None, None, None, :]
    if c["causal"]:
        place = torch.arange(top, device=x.device)
        hidden = hidden | (place[None, :] > place[:, None])
    x.masked_fill_(hidden, -math.inf)
    o = torch.matmul(_softmax_rows(x).view(b, kv, -1, top), v).view(b, kv, h // kv, top, hd)
    o = o.permute(0, 3, 1, 2, 4).reshape(b * top, h * hd)[s["back"]]
    return o.to(s["q"].dtype)


def _plain_append(s):
    c = s["case"]
    out = []
    for which in ("k", "v"):
        vals = _quantise(s, which, c["kv"], c["hd"])
        out.append(vals.view(-1, c["kv"] * c["hd"])[s["back"]].to(s[which].dtype))
    return {"k": out[0], "v": out[1], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_values(s, which, kv, hd, bs):
    """The cache's values of every sequence, padded to the longest: [batch, kv, positions, hd]."""
    page = s[which + "_pool"][s["table_dev"], 0]
    b, n = s["table_dev"].shape
    x = page.view(b, n, bs, kv, hd).permute(0, 3, 1, 2, 4).float()
    x -= 128.0
    x *= s[which + "_scale"][s["table_dev"], 0].permute(0, 2, 1)[:, :, :, None, None]
    return x.reshape(b, kv, n * bs, hd)


def _plain_q8(s):
    c = s["case"]
    h, kv, hd, bs, nq = c["heads"], c["kv"], c["hd"], c["bs"], c["nq"]
    _quantise(s, "k", kv, hd)
    _quantise(s, "v", kv, hd)
    b = len(s["past"])
    q = s["q"].view(b, nq, kv, h // kv, hd).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, hd)
    k = _plain_values(s, "k", kv, hd, bs)
    top = k.shape[2]
    x = torch.matmul(q * float(np.float32(hd ** -0.5)), k.transpose(2, 3)).view(b, kv, h // kv, nq, top)
    del k
    place = torch.arange(top, device=x.device)
    last = s["past_dev"][:, None] + (torch.arange(nq, device=x.device)[None, :] if c["causal"] else nq - 1)
    x.masked_fill_((place[None, None, :] > last.expand(b, nq)[:, :, None])[:, None, None], -math.inf)
    v = _plain_values(s, "v", kv, hd, bs)
    # places behind the sequence hold whatever the pages held: their probability is 0 and their elements are finite
    o = torch.matmul(_softmax_rows(x).view(b, kv, -1, top), v).view(b, kv, h // kv, nq, hd)
    o = o.permute(0, 3, 1, 2, 4).reshape(b * nq, h * hd)
    return {"out": o, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# -------------------------------------------------------------------- run ----

def run(s):
    c = s["case"]
    if not own:
        return {"packed": _plain_packed, "append": _plain_append, "q8": _plain_q8}[c["op"]](s)
    pkv = s["pkv"]
    scale = c["hd"] ** -0.5
    if c["op"] == "packed":
        pkv.check(pkv.pkv_attn_packed(s["q"], s["k"], s["v"], s["n_dev"], c["heads"], c["kv"], c["hd"], int(c["causal"]), scale,
                                      s["out"], torch.cuda.current_stream()))
        return s["out"]
    if c["op"] == "append":
        pkv.check(pkv.pkv_append_packed(s["seqs"], s["n_new"], 0, s["k"], s["v"]))
        pkv.check(pkv.pkv_read_packed(s["seqs"], s["start"], s["n_new"], 0, s["k_out"], s["v_out"]))
        return {"k": s["k_out"], "v": s["v_out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    pkv.check(pkv.pkv_attn_batch(s["seqs"], s["n_new"], s["q"], s["k"], s["v"], c["heads"], c["kv"], c["hd"], 0,
                                 int(c["causal"]), scale, s["out"]))
    return {"out": s["out"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------ exact values ----

def _exact_attend(q, k, v, offset, causal, scale):
    """q [n, g, d], k, v [m, d] in 64 bits; query i sees keys 0 .. offset + i (all of them where not causal)."""
    out = torch.empty_like(q)
    m = k.shape[0]
    for i0 in range(0, q.shape[0], 4096):
        part = q[i0:i0 + 4096]
        x = torch.einsum("ngd,md->ngm", part, k) * scale
        if causal:
            seen = offset + i0 + torch.arange(part.shape[0], device=q.device)
            x = torch.where(torch.arange(m, device=q.device)[None, :] <= seen[:, None], x.transpose(0, 1),
                            torch.full((), -math.inf, dtype=x.dtype, device=q.device)).transpose(0, 1)
        out[i0:i0 + 4096] = torch.einsum("ngm,md->ngd", torch.softmax(x, dim=-1), v)
    return out


def _exact_page(old, old_scale, rows, keep):
    """One page of one kv head in 64 bits on the host's arithmetic: elements (signed) and the scale after the append."""
    top = float(np.abs(rows).max())
    e = -126
    if top > 0:
        e = max(-126, int(math.floor(math.log2(top))) - 8)
        while top > 127.0 * 2.0 ** e:
            e += 1
    q = old.copy()
    if keep:
        e0 = int(round(math.log2(old_scale)))
        e = max(e, e0)
        q[:keep] = np.rint(old[:keep] * 2.0 ** (e0 - e))
    q[keep:keep + len(rows)] = np.rint(rows * 2.0 ** -e)
    return q, 2.0 ** e


def _exact_pages(case, d, which):
    """The appended pages: {block: elements [bs, kv, hd]}, and the scales of the whole pool, in 64 bits."""
    bs, kv, hd = case["bs"], case["kv"], case["hd"]
    x = d[which].double().cpu().numpy().reshape(-1, kv, hd)
    scales = d[which + "_scale"].double().cpu().numpy()
    want = [int(b) for r, (p, n) in enumerate(zip(d["past"], d["new"])) for b in d["table"][r, p // bs:(p + n - 1) // bs + 1]]
    old = dict(zip(want, d[which + "_pool"][torch.tensor(want, device="cuda"), 0].cpu().numpy().astype(np.float64)))
    pages, row = {}, 0
    for r, (p, n) in enumerate(zip(d["past"], d["new"])):
        done = 0
        while done < n:
            pos = p + done
            b, keep = int(d["table"][r, pos // bs]), pos % bs
            m = min(bs - keep, n - done)
            page = old[b].reshape(bs, kv, hd) - 128.0
            for h in range(kv):
                page[:, h], scales[b, 0, h] = _exact_page(page[:, h], scales[b, 0, h], x[row:row + m, h], keep)
            pages[b] = page
            row += m
            done += m
    return pages, scales


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "packed":
        lens = d["lens"]
        if sum(float(n) * n for n in lens) * case["heads"] * case["hd"] > 1.5e12:
            return None
        h, kv, hd = case["heads"], case["kv"], case["hd"]
        out = torch.empty(d["q"].shape[0], h, hd, dtype=torch.float64, device="cuda")
        at = 0
        for n in lens:
            for j in range(kv):
                g = slice(j * (h // kv), (j + 1) * (h // kv))
                q = d["q"][at:at + n].double().view(n, h, hd)[:, g]
                k, v = (d[w][at:at + n].double().view(n, kv, hd)[:, j] for w in ("k", "v"))
                out[at:at + n, g] = _exact_attend(q, k, v, 0, case["causal"], hd ** -0.5)
            at += n
        return out.view(-1, h * hd)
    if sum(d["new"]) * case["kv"] > 120_000:
        return None
    bs, kv, hd = case["bs"], case["kv"], case["hd"]
    pages, scales = {}, {}
    for w in ("k", "v"):
        pages[w], scales[w] = _exact_pages(case, d, w)
    found = {w + "_scale": torch.from_numpy(scales[w]) for w in ("k", "v")}
    if case["op"] == "append":
        for w in ("k", "v"):
            rows = []
            for r, (p, n) in enumerate(zip(d["past"], d["new"])):
                for pos in range(p, p + n):
                    b = int(d["table"][r, pos // bs])
                    rows.append(pages[w][b][pos % bs] * scales[w][b, 0][:, None])
            vals = torch.from_numpy(np.stack(rows).reshape(-1, kv * hd))
            # the values are multiples of a power of two with 7 bits: every type here holds them
            found[w] = vals
        return {k: found[k] for k in ("k", "v", "k_scale", "v_scale")}
    h, nq = case["heads"], case["nq"]
    if sum(float(nq) * (p + nq) for p in d["past"]) * h * hd > 1.5e12:
        return None
    for w in ("k", "v"):
        ids = sorted(pages[w])
        d[w + "_pool"][torch.tensor(ids, device="cuda"), 0] = torch.from_numpy(
            np.stack([pages[w][b] + 128.0 for b in ids]).reshape(len(ids), bs, kv * hd)).to(torch.uint8).cuda()
    out = torch.empty(nq * case["n"], h, hd, dtype=torch.float64, device="cuda")
    for r, p in enumerate(d["past"]):
        n = p + nq
        ids = torch.from_numpy(d["table"][r, :-(-n // bs)]).cuda()
        val = {}
        for w in ("k", "v"):
            x = d[w + "_pool"][ids, 0].view(-1, bs, kv, hd).double() - 128.0
            x = x * torch.from_numpy(scales[w]).cuda()[ids, 0][:, None, :, None]
            val[w] = x.view(-1, kv, hd)[:n]
        for j in range(kv):
            g = slice(j * (h // kv), (j + 1) * (h // kv))
            out[r * nq:(r + 1) * nq, g] = _exact_attend(d["q"][r * nq:(r + 1) * nq].double().view(nq, h, hd)[:, g],
                                                        val["k"][:, j], val["v"][:, j], p, case["causal"], hd ** -0.5)
    return {"out": out.view(-1, h * hd), **found}

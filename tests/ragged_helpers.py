"""Inputs, the 64-bit plain form and the tolerance of the cross and shared-prefix attention tests.

The tolerance of an output element counts the kernels' roundings (u: half a step of the type, 2^-8 for
bf16 and 2^-11 for f16):
  u * A       every probability rounded to the type before it meets V (the kernel of few rows keeps it in
              two pieces, off by u^2)
  u * |o|     the output rounded once (|o| <= A)
  2 e_s * A   scores off by e_s = (hd + 4) 2^-23 scale max_j sum_d |q_d k_jd| (f32 sums of exact products;
              the 4 for scaling and 2^x), in numerator and denominator
  n 2^-24 max|v|   probabilities below the type's normal range, off by at most 2^-25 (f16) each, relative to
              a sum of at least 1, and the f32 sum of n terms
with A = sum_j p_j |v_j|, computed in 64 bits.
"""
import math

import torch

import paged_kv_gqa_nx_gb300 as pkv

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Case:
    """Random rows of a call: prefix (None: cross attention), packed or in slots with `gap` rows between."""

    def __init__(self, ql, kl, H, KV, hd, dtype, prefix=None, gap=None, seed=0, mul=1.0, k_start=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.ql, self.kl, self.H, self.KV, self.hd, self.dtype, self.prefix = list(ql), list(kl), H, KV, hd, dtype, prefix
        self.start, at = [], 0
        for n in kl:
            self.start.append(at)
            at += n + (gap or 0)
        self.k_start = [s + 0 for s in self.start] if gap is not None else None
        if k_start is not None:
            self.start = self.k_start = list(k_start)
            at = max([a + b for a, b in zip(self.start, kl)] + [1])

        def rows(n, w, m=1.0):
            return (torch.randn(max(n, 1), w, device="cuda", generator=g) * m).to(dtype)
        self.q = rows(sum(ql), H * hd, mul)
        self.k, self.v = rows(at, KV * hd), rows(at, KV * hd)
        self.kp, self.vp = (rows(prefix, KV * hd)[:prefix] for _ in range(2)) if prefix is not None else (None, None)

    def workspace(self, k_start=True):
        if self.prefix is None:
            n = pkv.pkv_attn_cross_workspace(self.ql, self.kl, self.H, self.KV, self.hd, self.k_start)
        else:
            n = pkv.pkv_attn_prefix_workspace(self.prefix, self.ql, self.kl, self.H, self.KV, self.hd)
        assert n >= 0, pkv.pkv_last_error()
        return torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")  # (NaN as floats)

    def call(self, out=None, workspace="full", scale=None, stream=None):
        if out is None:
            out = torch.full((self.q.shape[0], self.H * self.hd), float("nan"), dtype=self.dtype, device="cuda")
        w = self.workspace() if isinstance(workspace, str) else workspace
        scale = self.hd ** -0.5 if scale is None else scale
        s = stream if stream is not None else torch.cuda.current_stream()
        if self.prefix is None:
            rc = pkv.pkv_attn_cross(self.q, self.ql, self.k, self.v, self.kl, self.H, self.KV, self.hd, scale, out,
                                    self.k_start, w, s)
        else:
            rc = pkv.pkv_attn_prefix(self.q, self.ql, self.kp, self.vp, self.k, self.v, self.kl, self.H, self.KV, self.hd,
                                     scale, out, self.k_start, w, s)
        pkv.check(rc)
        return out

    def plain(self, scale=None):
        """(outputs, tolerance) in 64 bits."""
        H, KV, hd, u = self.H, self.KV, self.hd, U[self.dtype]
        G, scale = H // KV, hd ** -0.5 if scale is None else scale
        T = sum(self.ql)
        out = torch.zeros(T, H, hd, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        at = 0
        for n, m, k0 in zip(self.ql, self.kl, self.start):
            K, V = (x[k0:k0 + m].double().view(m, KV, hd) for x in (self.k, self.v))
            seen = torch.full((n,), m, device="cuda")
            if self.prefix is not None:
                K, V = (torch.cat([p.double().view(-1, KV, hd), x]) for p, x in ((self.kp, K), (self.vp, V)))
                seen = self.prefix + m - n + 1 + torch.arange(n, device="cuda")
            s = slice(at, at + n)
            at += n
            if n == 0 or K.shape[0] == 0:
                continue
            hide = torch.arange(K.shape[0], device="cuda")[None, :] >= seen[:, None]
            for j in range(KV):
                g = slice(j * G, (j + 1) * G)
                Q = self.q[s].double().view(n, H, hd)[:, g]
                x = torch.einsum("igd,jd->gij", Q, K[:, j]) * scale
                w = (torch.einsum("igd,jd->gij", Q.abs(), K[:, j].abs()) * abs(scale)).masked_fill(hide, 0.0)
                p = torch.softmax(x.masked_fill(hide, -math.inf), dim=-1)
                out[s, g] = torch.einsum("gij,jd->igd", p, V[:, j])
                A = torch.einsum("gij,jd->igd", p, V[:, j].abs())
                es = (hd + 4) * 2.0 ** -23 * w.amax(-1).t()[:, :, None]
                tol[s, g] = A * (2 * u + 2 * es) + K.shape[0] * 2.0 ** -24 * V[:, j].abs().max()
        return out.view(T, H * hd), tol.view(T, H * hd)

    def check(self, got=None, scale=None, **kw):
        got = self.call(scale=scale, **kw) if got is None else got
        assert pkv.pkv_contiguous_sync_error(torch.cuda.current_stream()) == pkv.PKV_OK, pkv.pkv_last_error()
        exp, tol = self.plain(scale)
        T = sum(self.ql)
        err = (got[:T].double() - exp).abs()
        bad = ~(err <= tol)
        assert not bool(bad.any()), (int(bad.sum()), float(err.nan_to_num(9e9).max()), bad.nonzero()[:4].tolist())
        return got

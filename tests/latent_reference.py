"""Plain 64-bit forms of the cache, tree-attention and head-norm operators, on
the CPU, with the bands their results are held to.

Bands.  Every rounding to a type t is off by at most u(t) = finfo(t).eps / 2 of
the value.  A result that is rounded once from a value computed in fp32 is held
to u(t) |value| plus the fp32 arithmetic's share.  The bf16 attention rounds in
the middle of sums of hundreds of terms, where a worst case says nothing; its
roundings are independent of one another, uniform at best and so of variance at
most (u x)^2 / 3, and their first-order effect on each output value is a linear
form that is computed here from the exact values.  Results are held to eight
standard deviations of that form (a sum of bounded independent terms passes
that with probability below 2 exp(-32)), plus one final rounding.
"""
from __future__ import annotations

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SIGMAS = 8.0


def rows_of(cu_k, table, page, b, pos):
    """Cache rows of positions (a list) of sequence b; -1 where the table names no page."""
    out = []
    for s in pos:
        if table is None:
            out.append(cu_k[b] + s)
        else:
            e = int(table[b, s // page])
            out.append(e * page + s % page if e >= 0 else -1)
    return out


def quantise(x):
    """e4m3 codes (uint8) and power-of-two scales of fp64 rows [n, 128 g] that are fp32 or bf16 values."""
    blk = x.reshape(x.shape[0], -1, 128)
    amax = blk.abs().amax(-1)
    e = torch.zeros_like(amax)
    for i in torch.nonzero(amax).tolist():
        a = float(amax[tuple(i)])
        k = math.frexp(a / 448.0)[1] - 1
        while a > 448.0 * 2.0 ** k:
            k += 1
        while a <= 448.0 * 2.0 ** (k - 1):
            k -= 1
        e[tuple(i)] = max(-127, min(127, k))
    scale = 2.0 ** e
    codes = (blk / scale[..., None]).float().to(torch.float8_e4m3fn)  # exact in fp32, then one rounding
    return codes.reshape(x.shape).view(torch.uint8), scale.float()


def dequantise(codes, scale):
    v = codes.view(torch.float8_e4m3fn).double().reshape(codes.shape[0], -1, 128) * scale.double()[..., None]
    return v.reshape(codes.shape)


def visible(T, first, mask_rows):
    """[T, first + T] booleans; mask_rows: integers of node bits, or None for a chain."""
    see = torch.zeros(T, first + T, dtype=torch.bool)
    see[:, :first] = True
    for t in range(T):
        for j in range(T):
            see[t, first + j] = (j <= t) if mask_rows is None else bool(mask_rows[t] >> j & 1)
    return see


def tree_attention(q_nope, q_pe, lat, pe, see, W_UK, W_UV, scale, u, exchange=False):
    """One sequence: q_nope [T, H, d_n] ..., lat [n, d_c], pe [n, d_r], see [T, n] (all fp64 values of the stored
    types).  u: the unit rounding of the intermediate type.  exchange: the scores may be the sum of two halves of
    fp16, each half of the latent and rotary columns.  Returns out, its band, lse, its band."""
    T, H, _ = q_nope.shape
    d_c = lat.shape[1]
    lat = torch.where(see.any(0)[:, None], lat, torch.zeros(()).double())  # what nobody sees holds anything
    pe = torch.where(see.any(0)[:, None], pe, torch.zeros(()).double())
    out = torch.zeros(T, H, W_UV.shape[2], dtype=torch.float64)
    tol, lse, ltol = torch.zeros_like(out), torch.full((T, H), -math.inf).double(), torch.zeros(T, H).double()
    v = u / math.sqrt(3.0)
    acc = 2.0 ** -24 * math.sqrt(d_c + pe.shape[1] + lat.shape[0])  # fp32 sums of that many terms
    for h in range(H):
        qt = q_nope[:, h] @ W_UK[h]
        for t in range(T):
            vis = see[t].nonzero()[:, 0]
            if not len(vis):
                continue
            # a row must not depend on what it does not see, so only what it sees is looked at
            c, r = lat[vis], pe[vis]
            z = (c @ qt[t] + r @ q_pe[t, h]) * scale
            m = z.max()
            p = torch.exp(z - m)
            lse[t, h] = m + p.sum().log()
            p = p / p.sum()
            o = p @ c
            out[t, h] = o @ W_UV[h]
            d = c @ W_UV[h] - out[t, h]                      # value of each token against the mean
            lin = (p[:, None] * c).T @ d                     # effect of each q~ column's rounding
            absz = (c.abs() @ qt[t].abs() + r.abs() @ q_pe[t, h].abs()) * scale
            var_z = (acc * absz) ** 2
            if exchange:
                hc, hr = d_c // 2, r.shape[1] // 2
                for cs, rs in ((slice(0, hc), slice(0, hr)), (slice(hc, None), slice(hr, None))):
                    half = (c[:, cs] @ qt[t, cs] + r[:, rs] @ q_pe[t, h, rs]) * scale
                    var_z += (U[torch.float16] * half) ** 2 / 3
            var = (v * scale) ** 2 * (qt[t] ** 2) @ lin ** 2
            var += (p ** 2 * (var_z + v ** 2 + acc ** 2)) @ d ** 2
            var += v ** 2 * (o ** 2) @ W_UV[h] ** 2
            small = acc * (o.abs() @ W_UV[h].abs())          # fp32 sums of the last product
            tol[t, h] = SIGMAS * var.sqrt() + SIGMAS * small
            lvar = (v * scale) ** 2 * ((qt[t] * o) ** 2).sum() + (p ** 2 * (var_z + v ** 2)).sum()
            ltol[t, h] = SIGMAS * lvar.sqrt() + 2.0 ** -20 * (1 + lse[t, h].abs())
    return out, tol, lse, ltol


def norm_rope(x, norm, gain, bias, eps, cos, sin, pos, rope, rope_first):
    """x [N, n, D] fp64; cos, sin [n_pos, d_r / 2]; pos [N] (outside the tables: unrotated)."""
    D, d_r = x.shape[2], 2 * cos.shape[1]
    y = x
    if norm == "rms":
        y = x / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    elif norm == "layer":
        y = (x - x.mean(-1, keepdim=True)) / (x.var(-1, unbiased=False, keepdim=True) + eps).sqrt()
    if norm != "none":
        y = y * (1.0 if gain is None else gain) + (0.0 if bias is None or norm != "layer" else bias)
    at = 0 if rope_first else D - d_r
    keep = torch.cat([y[..., :at], y[..., at + d_r:]], -1)
    t = y[..., at:at + d_r]
    a, b = (t[..., ::2], t[..., 1::2]) if rope == "pairs" else (t[..., :d_r // 2], t[..., d_r // 2:])
    ok = [0 <= p < cos.shape[0] for p in pos]
    at_p = [p if o else 0 for p, o in zip(pos, ok)]
    here = torch.tensor(ok)[:, None, None]
    c = torch.where(here, cos[at_p][:, None], torch.ones(()).double())
    s = torch.where(here, sin[at_p][:, None], torch.zeros(()).double())
    return keep, torch.cat([a * c - b * s, a * s + b * c], -1)


class Batch:
    """Sequences of T new tokens on P cached ones (slack rows behind them), laid out contiguously (page 0) or in pages
    in random order with unused pages between."""

    def __init__(self, T, P, page, seed=0, slack=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.P, self.page = list(T), list(P), page
        self.S = [t + p + slack for t, p in zip(T, P)]
        self.cu_q, self.cu_k = [0], [0]
        for t, s in zip(self.T, self.S):
            self.cu_q.append(self.cu_q[-1] + t)
            self.cu_k.append(self.cu_k[-1] + s)
        self.N, self.table, self.n_pages = self.cu_q[-1], None, 0
        self.rows = self.cu_k[-1] + 3
        if page:
            per = [-(-s // page) for s in self.S]
            self.n_pages = sum(per) + 2
            order = torch.randperm(self.n_pages, generator=g).int()
            self.table = torch.full((len(T), max(per + [1])), -1, dtype=torch.int32)
            at = 0
            for b, k in enumerate(per):
                self.table[b, :k] = order[at:at + k]
                at += k
            self.rows = self.n_pages * page + 5

    def rows_at(self, b, pos):
        return rows_of(self.cu_k, self.table, self.page, b, pos)

    def seqs(self):
        import sparse_latent_attention_indexer_gb300 as dsa
        return dsa.Seqs(self.cu_q, self.cu_k, self.P)

    def pages(self):
        import sparse_latent_attention_indexer_gb300 as dsa
        return None if self.table is None else dsa.Pages(self.table.cuda(), self.page, self.n_pages)

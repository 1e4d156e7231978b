"""A paged KV cache on the CPU with 64-bit references of the attention operators.

Every cell of the pool that no token owns holds NaN, so whatever reads past a
sequence shows.  Tolerances are counted from the roundings (u = half a step of a type:
bf16 2^-8, e4m3 2^-4, fp32 2^-24 of a value) and written where they are used.
"""
from __future__ import annotations

import math

import torch

BF, F8 = torch.bfloat16, torch.float8_e4m3fn
U_BF, U_F8, U_32 = 2.0 ** -8, 2.0 ** -4, 2.0 ** -24
KINDS = {"bf16": BF, "e4m3": F8}


class Cache:
    """lens: (new tokens, tokens before them) a sequence; the new tokens' cells are filled too."""

    def __init__(self, lens, *, H_q, H_kv, d, page=16, kind="bf16", seed=0, extra_rows=1, spare=3, width=None,
                 q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H_q, self.H_kv, self.d, self.page, self.kind = lens, H_q, H_kv, d, page, kind
        self.B, self.T = len(lens), sum(n for n, _ in lens)
        need = [-(-(n + p) // page) for n, p in lens]
        self.N = 1 + sum(need) + spare
        ids = (1 + torch.randperm(self.N - 1, generator=g)).tolist()
        self.R = 1 + self.B + extra_rows
        self.width = width or max(need + [1]) + 1
        self.table = torch.zeros(self.R, self.width, dtype=torch.int32)
        self.kv_len = torch.zeros(self.R, dtype=torch.int32)
        rows = (1 + torch.randperm(self.R - 1, generator=g))[:self.B]
        self.row = rows.to(torch.int32)
        shape = (self.N, H_kv, page, d)
        k = torch.full(shape, math.nan, dtype=torch.float64)
        v = torch.full(shape, math.nan, dtype=torch.float64)
        self.refs = torch.zeros(self.N, dtype=torch.int32)
        for (n, past), r, m in zip(lens, rows.tolist(), need):
            mine, ids = ids[:m], ids[m:]
            self.table[r, :m] = torch.tensor(mine, dtype=torch.int32)
            self.kv_len[r] = n + past
            for i, p in enumerate(mine):
                self.refs[p] = 1
                c = min(page, n + past - i * page)
                k[p, :, :c] = torch.randn(H_kv, c, d, generator=g, dtype=torch.float64)
                v[p, :, :c] = torch.randn(H_kv, c, d, generator=g, dtype=torch.float64)
        self.k = k.to(torch.float32).to(KINDS[kind])
        self.v = v.to(torch.float32).to(KINDS[kind])
        self.k_scale = self.v_scale = None
        if kind == "e4m3":
            self.k_scale = 0.5 + torch.rand(H_kv, generator=g)
            self.v_scale = 0.5 + torch.rand(H_kv, generator=g)
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        self.cu = torch.tensor(cu, dtype=torch.int32)
        self.q = (q_scale * torch.randn(self.T, H_q, d, generator=g)).to(BF)
        self.gen = g

    def gather(self, b, h, which):
        """[L][d] of sequence b's kv head h, in 64 bits."""
        r = int(self.row[b])
        L = int(self.kv_len[r])
        pages, scale = (self.k, self.k_scale) if which == "k" else (self.v, self.v_scale)
        ids = self.table[r, :-(-L // self.page)].long()
        x = pages.to(torch.float32)[ids, h].reshape(-1, self.d)[:L].double()
        return x * scale[h].double() if scale is not None else x

    def cuda(self, **over):
        """The tensors of a call on the GPU, as keyword arguments."""
        t = dict(k_pages=self.k, v_pages=self.v, page_table=self.table, kv_len=self.kv_len, row=self.row,
                 cu_seqlens=self.cu, k_scale=self.k_scale, v_scale=self.v_scale)
        t.update(over)
        return {n: (x.cuda() if x is not None else None) for n, x in t.items()}


def attention(c: Cache, scale, window=0):
    """o, lse, and a bound of the kernel's error in each, in 64 bits.

    The kernel rounds each weight to bf16 once (u_bf of sum p|v|), o once (u_bf |o|), and works in fp32
    otherwise: a score is a sum of d products (off by at most d u_32 sum|q k| scale, plus two roundings of the
    score), which moves each weight by that much relatively, numerator and denominator alike."""
    o = torch.zeros(c.T, c.H_q, c.d, dtype=torch.float64)
    lse = torch.full((c.T, c.H_q), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(o)
    tol_lse = torch.zeros_like(lse)
    G = c.H_q // c.H_kv
    for b in range(c.B):
        a, e = int(c.cu[b]), int(c.cu[b + 1])
        L = int(c.kv_len[int(c.row[b])])
        pos = torch.arange(L - (e - a), L)[:, None]
        key = torch.arange(L)[None]
        seen = key <= pos
        if window:
            seen &= key > pos - window
        if L == 0 or e == a:
            continue
        for h in range(c.H_q):
            k, v = c.gather(b, h // G, "k"), c.gather(b, h // G, "v")
            q = c.q[a:e, h].double()
            s = torch.where(seen, q @ k.T * scale, -math.inf)
            some = seen.any(1)
            big = torch.where(seen, q.abs() @ k.abs().T * abs(scale), 0.0)
            ds = (c.d * U_32 * big + 4 * U_32 * s.abs().nan_to_num(posinf=0.0)).amax(1, keepdim=True) + 8 * U_32
            p = torch.where(some[:, None], torch.softmax(s, 1), 0.0)
            # a weight of 0 belongs to a cell that the token does not see, whatever stands there
            o[a:e, h] = sum_products(p, v)
            mass = sum_products(p, v.abs())
            lse[a:e, h] = torch.where(some, torch.logsumexp(s, 1), -math.inf)
            tol[a:e, h] = U_BF * o[a:e, h].abs() + (U_BF + 4 * ds + L * U_32) * mass + 1e-30
            tol_lse[a:e, h] = (2 * ds[:, 0] + (L + 8) * U_32 + 8 * U_32 * lse[a:e, h].abs().nan_to_num(posinf=0.0))
    return o, lse, tol, tol_lse


def sum_products(p, v):
    """p @ v where a weight of 0 takes nothing, not even from a NaN."""
    odd = ~torch.isfinite(v)
    o = p @ torch.where(odd, 0.0, v)
    for j in odd.any(1).nonzero()[:, 0].tolist():
        o += torch.where((p[:, j:j + 1] > 0) & odd[j], v[j], 0.0)
    return o


def check(got, want, tol, what):
    got = got.double().cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, 0.0, (got - want).abs())
    bad = ~(same | (off <= tol))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0]} for {want[bad][0]}, allowed {tol[bad][0]}")


def prologue(c: Cache, x, freqs, *, interleaved=False, scale=1.0, weight=None, eps=1e-6, add=0.0, positions=None):
    """Normed and rotated heads [T][H][d] in 64 bits, and what fp32 work may take from them (before rounding).

    The norm is a sum of d squares (its root: (d + 8) u_32 relatively); the rotation's angle is exact to 1e-9, its
    sine and cosine to 4 u_32, and two products meet in a sum."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (add + weight.double())
    rel = (c.d + 16) * U_32 if weight is not None else 0.0
    y, size = x.clone(), x.abs()
    rot = 2 * len(freqs)
    for b in range(c.B):
        for t in range(int(c.cu[b]), int(c.cu[b + 1])):
            pos = int(c.kv_len[int(c.row[b])]) - (int(c.cu[b + 1]) - t)
            if positions is not None:
                pos = int(positions[t])
            a = pos * freqs
            cos, sin = scale * torch.cos(a), scale * torch.sin(a)
            i, j = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved else
                    (slice(0, rot // 2), slice(rot // 2, rot)))
            u, w = x[t][:, i], x[t][:, j]
            y[t][:, i], y[t][:, j] = u * cos - w * sin, w * cos + u * sin
            size[t][:, i] = size[t][:, j] = abs(scale) * (u.abs() + w.abs())
    return y, size * (rel + 12 * U_32)

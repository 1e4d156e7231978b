"""Attention in 64 bits on any device, with a bound per (token, head), and how the kernels deal out work.

``attn_helpers.attention`` bounds each value by what its roundings could add up to in one direction, 2^-8 sum p |v|.
Over thousands of keys that is a good part of the value itself, for o shrinks as they cancel, so a lost block of
keys passes.  Here the error is bounded as a vector:

  the rounding of o            at most 2^-8 |o|, value by value;
  the rounding of the weights  sum_j p_j e_j v_j with |e_j| <= 2^-8 of either sign: keys' values point in directions
                               of their own (the caches are random), so the terms add as sqrt(sum p_j^2 |v_j|^2), with a
                               quarter more for the angles of a few keys that carry the weight (64 values or more a head);
  fp32 sums over the keys      L 2^-24 |o|;
  a score's sum of d products  sqrt(d) 2^-24 sum |q k| scale, four times over, and its own roundings: relative in a
                               weight, so these too add as sqrt(sum p_j^2 |v_j|^2).

A block of m of L keys that is lost takes about sqrt(m / L) |o|: 0.04 of it for 32 of 20 thousand keys, against a
bound of 0.01 |o|.
"""
from __future__ import annotations

import math

import torch

from tests.attn_helpers import U_32, U_BF


def cells(c, b, pages, scales, device):
    """[H_kv][L][d] of sequence b, in 64 bits; only its own pages are converted."""
    r = int(c.row[b])
    L = int(c.kv_len[r])
    bits = torch.uint8 if pages.element_size() == 1 else torch.int16
    x = pages.view(bits)[c.table[r, :-(-L // c.page)].long()].to(device).view(pages.dtype).double()
    x = x.transpose(0, 1).flatten(1, 2)[:, :L]
    return x * scales.double().to(device)[:, None, None] if scales is not None else x


def attention(c, scale, window=0, device="cpu"):
    """o, lse [T][H_q] and bounds of |got - o| and |lse - got| per (token, head), in 64 bits on the CPU."""
    G = c.H_q // c.H_kv
    o = torch.zeros(c.T, c.H_q, c.d, dtype=torch.float64)
    lse = torch.full((c.T, c.H_q), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(lse), torch.zeros_like(lse)
    for b in range(c.B):
        a, e = int(c.cu[b]), int(c.cu[b + 1])
        L = int(c.kv_len[int(c.row[b])])
        if L == 0 or e == a:
            continue
        pos = torch.arange(L - (e - a), L, device=device)[:, None]
        key = torch.arange(L, device=device)[None]
        seen = key <= pos
        if window:
            seen &= key > pos - window
        some = seen.any(1)
        ks, vs = cells(c, b, c.k, c.k_scale, device), cells(c, b, c.v, c.v_scale, device)
        for h in range(c.H_kv):
            k, v = ks[h], vs[h]
            odd = ~torch.isfinite(v)
            fine = torch.where(odd, 0.0, v)
            kt, ka = k.T.contiguous(), k.abs().T.contiguous()
            v2 = fine.square().sum(1)
            for g in range(h * G, h * G + G):
                q = c.q[a:e, g].double().to(device)
                s = torch.where(seen, q @ kt * scale, -math.inf)
                big = torch.where(seen, q.abs() @ ka * abs(scale), 0.0)
                ds = ((4 * c.d ** 0.5 * big).amax(1) + 4 * torch.where(seen, s.abs(), 0.0).amax(1) + 8) * U_32
                p = torch.where(some[:, None], torch.softmax(s, 1), 0.0)
                x = p @ fine
                spread = (p.square() @ v2).sqrt()
                size = x.norm(dim=1)
                for j in odd.any(1).nonzero()[:, 0].tolist():
                    x += torch.where((p[:, j:j + 1] > 0) & odd[j], v[j], 0.0)
                o[a:e, g] = x.cpu()
                top = torch.where(some, torch.logsumexp(s, 1), -math.inf)
                lse[a:e, g] = top.cpu()
                tol[a:e, g] = (U_BF * size + (1.25 * U_BF + 8 * ds) * spread + L * U_32 * size + 1e-30).cpu()
                tol_lse[a:e, g] = (2 * ds + (L + 8) * U_32 + 8 * U_32 * top.abs().nan_to_num(posinf=0.0)).cpu()
    return o, lse, tol, tol_lse


def check_norms(got, want, tol, what):
    """Per (token, head): the same values that are not finite, and the rest within tol of `want` as a vector."""
    got = got.double().cpu()
    odd = ~(torch.isfinite(want) & torch.isfinite(got))
    assert ((got == want) | (got.isnan() & want.isnan()))[odd].all(), f"{what}: other values are not finite"
    off = torch.where(odd, 0.0, got - want).norm(dim=-1)
    bad = ~(off <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} heads off, first {bad.nonzero()[0].tolist()} by "
                           f"{off[bad][0]}, allowed {tol[bad][0]}, size {want.nan_to_num(0, 0, 0).norm(dim=-1)[bad][0]}")


ROW_TILE, ROW_UNIT = 16, 128  # the kernel of few rows: rows of a tile, keys of a unit
TILE = 256                    # the other: rows of a tile


def deal(c, window, workgroups, few):
    """[(entry, first block, last block + 1, blocks of the entry, slot)] a piece: what each workgroup does of the
    (sequence, kv head, tile) entries, one list a workgroup.  few: the kernel of few rows (workgroups 2 a CU),
    otherwise the one of 256-row tiles (1 a CU)."""
    G = c.H_q // c.H_kv
    block = ROW_UNIT if few else (32 if c.d == 256 else 128)
    sizes = []
    for b, (n, past) in enumerate(c.lens):
        L, rows = n + past, n * G
        for h in range(c.H_kv):
            for t in range(-(-rows // (ROW_TILE if few else TILE))):
                if few:
                    lo = max(0, L - n - window + 1) & ~31 if window else 0
                    sizes.append(max(1, -(-(L - lo) // block)))
                else:
                    last = min(rows, (t + 1) * TILE) - 1
                    hi = L - n + last // G + 1
                    lo = max(0, L - n + t * TILE // G - window + 1) // block * block if window else 0
                    sizes.append(-(-(hi - lo) // block))
    total = sum(sizes)
    pieces = min(total, workgroups)
    at = [0]
    for s in sizes:
        at.append(at[-1] + s)
    out, e = [], 0
    for w in range(pieces):
        u, end = total * w // pieces, total * (w + 1) // pieces
        mine = []
        while u < end:
            while at[e + 1] <= u:
                e += 1
            stop = min(at[e + 1], end)
            mine.append((e, u - at[e], stop - at[e], sizes[e], min(1, len(mine))))
            u = stop
        out.append(mine)
    return out

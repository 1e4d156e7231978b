"""Linear attention with a decay for each head, token by token in 64 bits on the CPU, with bounds of what the
kernels may be off by.

A state's error grows along the recurrence: every token scales what is there by a decay that fp32 work is off by
about |g| steps (its logarithm's products and sums) and a few more (the exponential, products and sums), and adds a
product that is off by a few steps itself.  With A the recurrence of the absolute values and u = 2^-24:
  err_t = e^g (err_(t-1) + (3 |g| + 8) u A_(t-1)) + 8 u |k v|.
A read-out sums d_k products (d_k + 40 steps of |q| A, the chunk's sums among them) and, in the chunked form, takes
the state and the weights of a chunk as two bf16 numbers each, which leave at most 2^-15 of each: 2^-14 of |q| A
together.  Its own rounding is half a step of bf16, 2^-8.
"""
from __future__ import annotations

import torch

BF = torch.bfloat16
U_BF, U_32 = 2.0 ** -8, 2.0 ** -24


def recurrence(q, k, v, g, S0, scale):
    """q, k [T][H_k][d_k], v [T][H_v][d_v] (bf16), g [T][H_v], S0 [H_v][d_k][d_v]: o, its bound, and a list of
    (state, bound) after each token, S0's first.  All in 64 bits."""
    r = v.shape[1] // q.shape[1]
    q, k = (x.double().repeat_interleave(r, 1) for x in (q, k))
    v, g, S = v.double(), g.double(), S0.double()
    A, err = S.abs(), torch.zeros_like(S)
    o, tol, states = torch.zeros_like(v), torch.zeros_like(v), [(S, err)]
    for t in range(v.shape[0]):
        e = torch.exp(g[t])[:, None, None]
        kv = k[t][:, :, None] * v[t][:, None]
        S = e * S + kv
        err = e * (err + (3 * g[t].abs().clamp_max(200.0)[:, None, None] + 8) * U_32 * A) + 8 * U_32 * kv.abs()
        A = e * A + kv.abs()
        states.append((S, err + 1e-37))
        o[t] = scale * (q[t][:, :, None] * S).sum(1)
        mass = (q[t].abs()[:, :, None] * A).sum(1)
        tol[t] = (U_BF * o[t].abs() + abs(scale) * ((q[t].abs()[:, :, None] * err).sum(1) +
                                                    ((q.shape[2] + 40) * U_32 + 2.0 ** -14) * mass) + 1e-37)
    return o, tol, states


def close(got, want, tol, what):
    got = got.double().cpu()
    off = (got - want).abs()
    bad = ~((off <= tol) | (got == want))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0]} for {want[bad][0]}, allowed {tol[bad][0]}")


class Layer:
    """Inputs of packed tokens with q, k and v as views of one projection, and a pool whose slots hold states."""

    def __init__(self, T, *, H_k=2, H_v=2, d_k=64, d_v=64, N=9, per_token=True, seed=0, spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.H_k, self.H_v, self.d_k, self.d_v, self.N = T, H_k, H_v, d_k, d_v, N
        x = torch.randn(T, 2 * H_k * d_k + H_v * d_v, generator=gen).to(BF)
        self.qkv = x
        slope = -spread * torch.exp2(-6.0 * torch.rand(H_v, generator=gen))
        self.per_token = per_token
        self.g = slope * torch.rand(T, H_v, generator=gen) * 2 if per_token else slope
        self.state = torch.randn(N, H_v, d_k, d_v, generator=gen)
        self.state[0] = 0
        self.scale = d_k ** -0.5

    def heads(self, x):
        a, b = self.H_k * self.d_k, 2 * self.H_k * self.d_k
        return (x[:, :a].unflatten(1, (self.H_k, self.d_k)), x[:, a:b].unflatten(1, (self.H_k, self.d_k)),
                x[:, b:].unflatten(1, (self.H_v, self.d_v)))

    def reference(self, a, e, S0):
        q, k, v = self.heads(self.qkv)
        g = self.g[a:e] if self.per_token else self.g.expand(e - a, self.H_v)
        return recurrence(q[a:e], k[a:e], v[a:e], g, S0, self.scale)

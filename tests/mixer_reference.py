"""Plain fp64 forms of the mixers of include/carve_mixers.h, written from their definitions (token
by token, full score matrices) on the CPU; gradients by torch.autograd.  Used by the tests alone."""
from __future__ import annotations

import math

import torch


def delta(q, k, v, g, w, A_dec=None, tau=None, S0=None):
    """q, k [T, Hk, dk], v [T, Hv, dv], g, w [T, Hv] (fp64): outputs [T, Hv, dv], last state."""
    T, Hv, dv = v.shape
    share = Hv // k.shape[1]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    x = g if tau is None else g + tau
    la = -torch.nn.functional.softplus(x, threshold=1e9)
    a = torch.exp(la if A_dec is None else torch.exp(A_dec) * la)
    w = torch.sigmoid(w)
    S = torch.zeros(Hv, dv, k.shape[2], dtype=torch.float64) if S0 is None else S0
    o = []
    for t in range(T):
        S = S * a[t][:, None, None]
        u = w[t][:, None] * (v[t] - (S * k[t][:, None, :]).sum(-1))
        S = S + u[:, :, None] * k[t][:, None, :]
        o.append((S * q[t][:, None, :]).sum(-1))
    return (torch.stack(o) if o else v.new_zeros(0, Hv, dv)), S


def visible(T, window, sinks):
    i, j = torch.arange(T)[:, None], torch.arange(T)
    return (j <= i) & ((i - j < window) | (j < sinks))


def window(q, k, v, win, sinks, scale=None):
    """q [T, Hq, d], k, v [T, Hkv, d] (fp64): outputs [T, Hq, d] and log-sum-exp [T, Hq]."""
    T, Hq, d = q.shape
    share = Hq // k.shape[1]
    k, v = k.repeat_interleave(share, 1), v.repeat_interleave(share, 1)
    s = torch.einsum("ihd,jhd->hij", q, k) * (d ** -0.5 if scale is None else scale)
    s = s.masked_fill(~visible(T, win, sinks), -math.inf)
    return torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), v), torch.logsumexp(s, -1).T


def window_masses(q, k, v, dO, win, sinks, scale=None):
    """What the absolute values of each result's terms add up to: the size that a rounding of the
    terms is relative to.  o: sum p |v|; dv: sum p |dO|; dq, dk: sum of |scale| p (|dO|.|v| +
    |dO|.|o|) times |k|, |q|."""
    T, Hq, d = q.shape
    share = Hq // k.shape[1]
    sc = d ** -0.5 if scale is None else scale
    kk, vv = k.repeat_interleave(share, 1), v.repeat_interleave(share, 1)
    s = torch.einsum("ihd,jhd->hij", q, kk) * sc
    p = torch.softmax(s.masked_fill(~visible(T, win, sinks), -math.inf), -1)
    o = torch.einsum("hij,jhd->ihd", p, vv)
    ds = abs(sc) * p * (torch.einsum("ihd,jhd->hij", dO.abs(), vv.abs()) + (dO.abs() * o.abs()).sum(-1).T[:, :, None])

    def shared(x):   # [T, Hq, d] -> [T, Hkv, d]
        return x.unflatten(1, (-1, share)).sum(2)

    return dict(o=torch.einsum("hij,jhd->ihd", p, vv.abs()), dq=torch.einsum("hij,jhd->ihd", ds, kk.abs()),
                dk=shared(torch.einsum("hij,ihd->jhd", ds, q.abs())),
                dv=shared(torch.einsum("hij,ihd->jhd", p, dO.abs())))


def grads(f, inputs, cotangents):
    """Gradients of sum_n <cotangents[n], f(**inputs)[n]> with respect to every input (None: not
    given)."""
    leaves = {n: x.detach().clone().requires_grad_() for n, x in inputs.items() if x is not None}
    outs = f(**{n: leaves.get(n) for n in inputs})
    total = sum((c * o).sum() for c, o in zip(cotangents, outs) if c is not None)
    return dict(zip(leaves, torch.autograd.grad(total, list(leaves.values()), allow_unused=True,
                                                materialize_grads=True)))

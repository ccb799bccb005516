"""Plain 64-bit implementations of the gated delta rule and of the projection,
on the CPU, and the comparison that their GPU tests share."""
from __future__ import annotations

import math

import torch


def unit(x, eps):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)


def rule(q, k, v, log_alpha, beta, S0=None, *, l2norm_qk=True, beta_is_logit=False,
         decay_from_logit=False, decay_scale=None, decay_bias=None, q_scale=1.0, eps_l2=1e-6):
    """One sequence, token by token: q, k [T, H_k, d_k], v [T, H_v, d_v], log_alpha and
    beta [T, H_v], S0 [H_v, d_k, d_v] or None.  Returns (o, the states after each token)."""
    q, k, v, g, b = (x.detach().cpu().double() for x in (q, k, v, log_alpha, beta))
    G = v.shape[1] // q.shape[1]
    if l2norm_qk:
        q, k = unit(q, eps_l2), unit(k, eps_l2)
    if beta_is_logit:
        b = torch.sigmoid(b)
    if decay_from_logit:
        A = 1.0 if decay_scale is None else decay_scale.detach().cpu().double()
        c = 0.0 if decay_bias is None else decay_bias.detach().cpu().double()
        g = -A * torch.log1p(torch.exp(g + c))
    a = torch.exp(torch.clamp(g, max=0.0))
    S = (torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if S0 is None
         else S0.detach().cpu().double().clone())
    o = torch.zeros_like(v)
    states = []
    for t in range(q.shape[0]):
        for h in range(v.shape[1]):
            kt, qt = k[t, h // G], q[t, h // G]
            fade = a[t, h] * S[h]
            S[h] = fade + b[t, h] * torch.outer(kt, v[t, h] - fade.T @ kt)
            o[t, h] = q_scale * (S[h].T @ qt)
        states.append(S.clone())
    return o, states


def last_state(states, S0, shape):
    if states:
        return states[-1]
    return torch.zeros(shape, dtype=torch.float64) if S0 is None else S0.detach().cpu().double()


def activation(z, act):
    return {"none": lambda: z, "relu": lambda: torch.clamp(z, min=0.0),
            "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2.0)),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi)
                                                           * (z + 0.044715 * z ** 3))),
            "sigmoid": lambda: torch.sigmoid(z)}[act]()


# No activation is steeper than this (silu' <= 1.0999, gelu' <= 1.1290 in both forms).
STEEPEST = 1.13


def linear(x, w, bias=None, residual=None, act="none"):
    """(y, how far an fp32 evaluation may be from it before its last rounding).

    A sum of K products in fp32, in any order and with every addition cut rather than
    rounded (2^-23 each), is off by at most (K + 2) 2^-23 sum |x||w|; the bias adds one rounding of
    |z|; the activation multiplies that by its steepest slope and adds its own few roundings
    (16 half-steps of 2^-24 of the value, which covers an exponential of an argument of up to 40
    whose own rounding it magnifies, and 16 of the argument where the value is far below it);
    the residual adds one."""
    x, w = x.detach().cpu().double(), w.detach().cpu().double()
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z = z + bias.detach().cpu().double()
        mag = mag + bias.detach().cpu().double().abs()
    off = (x.shape[1] + 2) * 2.0 ** -23 * mag
    y = activation(z, act)
    if act != "none":
        off = STEEPEST * off + 16 * 2.0 ** -24 * (y.abs() + z.abs())
    if residual is not None:
        y = y + residual.detach().cpu().double()
        off = off + 2.0 ** -24 * y.abs()
    return y, off


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def excess(x, ref):
    """|x - ref| beyond the rounding of x to its own type (half a step of the value)."""
    assert torch.isfinite(x).all()
    x64 = x.detach().cpu().double()
    return torch.clamp((x64 - ref).abs() - half_step(x.dtype) * ref.abs(), min=0.0)


def rel(x, ref):
    """2-norm of the excess over the 2-norm of the reference."""
    if ref.numel() == 0:
        return 0.0
    n = float(ref.norm())
    e = float(excess(x, ref).norm())
    return e / n if n > 0 else e

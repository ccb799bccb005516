"""The gated linear recurrence and its gradient in 64 bits on the CPU, token by token, with
how far an fp32 evaluation may be from them before its last rounding.

The allowances, in units of E = 2^-24 (half a step of fp32):
* a decay's distance from one, the factor c and a gate are each off by at most REL of
  themselves: the exponential of an argument of up to 20 by an approximate instruction is off by
  (2 + 1.2 * 20) * 2, a quotient by 4, the series and the products behind it by 16 more.
  (A decay far from one: a |g| <= 1.3 (1 - a), so that it is covered as well, with the
  factor 2 below.)
* a state is off by what its predecessor was, faded, by 2 REL (1 - a) of the largest size that
  the predecessor's terms can have, and by 4 roundings of its own terms' size; `size` is the same
  recurrence of magnitudes, which bounds every partial result of a scan in pieces.
* the gradient of a state runs the same recurrence backwards.
"""
import torch

E = 2.0 ** -24
REL = 72


def _d(t):
    return None if t is None else t.detach().cpu().double()


class Form:
    """What a call's tokens give: decays, factors and slopes of [T, D]."""

    def __init__(self, x, la, *, decay_from="log", decay_scale=None, decay_bias=None,
                 input_scale="none", input_gate=None):
        self.x, la = _d(x), _d(la)
        A = 1.0 if decay_scale is None else _d(decay_scale)
        v = la if decay_bias is None else la + _d(decay_bias)
        if decay_from == "log":
            v = la
            g, self.dv, self.val = v.clamp(max=0.0), (v <= 0).double(), None
        elif decay_from == "softplus":
            self.val = torch.logaddexp(v, torch.zeros((), dtype=v.dtype))
            g, self.dv = -A * self.val, -A * torch.sigmoid(v)
        else:
            self.val = torch.sigmoid(v)
            g, self.dv = -A * self.val, -A * self.val * torch.sigmoid(-v)
        self.a = torch.exp(g)
        self.near = -torch.expm1(g)  # 1 - a
        if input_scale == "none":
            self.c, self.dc = torch.ones_like(g), torch.zeros_like(g)
        elif input_scale == "complement":
            self.c, self.dc = self.near, -self.a
        else:
            self.c = torch.sqrt(-torch.expm1(2 * g))
            self.dc = torch.where(self.c > 0, -self.a ** 2 / self.c, torch.zeros_like(g))
        if input_gate is None:
            self.s, self.rest = torch.ones_like(g), torch.zeros_like(g)
        else:
            self.s, self.rest = torch.sigmoid(_d(input_gate)), torch.sigmoid(-_d(input_gate))


def scan(f, h0, lens):
    """(y, h_T, their allowances, states before each token, allowances and sizes of those)."""
    T, D = f.x.shape
    h0 = torch.zeros(len(lens), D, dtype=torch.float64) if h0 is None else _d(h0)
    u = f.c * f.s * f.x
    y, off_y = torch.zeros(T, D, dtype=torch.float64), torch.zeros(T, D, dtype=torch.float64)
    before, off_b, size_b = (torch.zeros(T, D, dtype=torch.float64) for _ in range(3))
    end, off_end = h0.clone(), torch.zeros_like(h0)
    at = 0
    for n, L in enumerate(lens):
        h, off, size = h0[n], torch.zeros(D, dtype=torch.float64), h0[n].abs()
        for t in range(at, at + L):
            before[t], off_b[t], size_b[t] = h, off, size
            off = f.a[t] * off + E * (2 * REL * f.near[t] * size + 2 * REL * u[t].abs())
            h = f.a[t] * h + u[t]
            size = f.a[t] * size + u[t].abs()
            off = off + 4 * E * size
            y[t], off_y[t] = h, off
        end[n], off_end[n] = h, off
        at += L
    return y, end, off_y, off_end, (before, off_b, size_b)


def backward(f, h0, lens, dy, dh_T):
    """{name: (gradient, allowance)} of dx, dla, dgate, dh0, dA, db."""
    T, D = f.x.shape
    dy = torch.zeros(T, D, dtype=torch.float64) if dy is None else _d(dy)
    dh = torch.zeros(len(lens), D, dtype=torch.float64) if dh_T is None else _d(dh_T)
    _, _, _, _, (hb, off_hb, size_hb) = scan(f, h0, lens)
    G, off_G, size_G = (torch.zeros(T, D, dtype=torch.float64) for _ in range(3))
    dh0, off_dh0 = dh.clone(), torch.zeros_like(dh)
    at = 0
    for n, L in enumerate(lens):
        back, off, size = dh[n], torch.zeros(D, dtype=torch.float64), dh[n].abs()
        for t in reversed(range(at, at + L)):
            G[t], size_G[t] = dy[t] + back, dy[t].abs() + size
            off_G[t] = off + E * size_G[t]
            back = f.a[t] * G[t]
            off = f.a[t] * off_G[t] + E * (2 * REL * f.near[t] + 4) * size_G[t]
            size = f.a[t] * size_G[t]
        dh0[n], off_dh0[n] = back, off
        at += L
    cs = f.c * f.s
    dx = G * cs
    off_dx = off_G * cs + 2 * REL * E * size_G * cs
    dgate = dx * f.x * f.rest
    off_dgate = (off_dx + REL * E * size_G * cs) * (f.x * f.rest).abs()
    inner = f.a * hb + f.dc * f.s * f.x
    terms = f.a * size_hb + (f.dc * f.s * f.x).abs()
    off_inner = f.a * off_hb + E * (2 * REL * f.near * size_hb + 2 * REL * terms)
    dg = G * inner
    off_dg = off_G * terms + size_G * off_inner + 2 * E * size_G * terms
    dla = f.dv * dg
    off_dla = f.dv.abs() * (off_dg + 2 * REL * E * size_G * terms)
    out = {"dx": (dx, off_dx), "dla": (dla, off_dla), "dgate": (dgate, off_dgate), "dh0": (dh0, off_dh0)}
    if f.val is not None:
        total = sum(lens)
        dA, db = -(f.val * dg)[:total], dla[:total]
        off_A = f.val[:total] * (off_dg + REL * E * size_G * terms)[:total]
        # sums of eight terms each, then compensated ones
        out["dA"] = dA.sum(0), off_A.sum(0) + 8 * E * dA.abs().sum(0)
        out["db"] = db.sum(0), off_dla[:total].sum(0) + 8 * E * db.abs().sum(0)
    return out

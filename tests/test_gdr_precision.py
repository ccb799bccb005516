"""How exactly the chunked rule holds its operands: every fp32 operand enters the
tensor cores as the sum of three bf16 parts, each rounded to nearest.

Bounds (2-norm of the error over the 2-norm of the result; for o beyond its own
rounding):

* final states.  Three parts hold all of fp32's 24 bits, and the products of parts
  that are left out are below 2^-24.  What remains is the sums: an instruction adds
  16 products to its fp32 sum and cuts the result, by half a unit, 2^-24, on average
  and always toward zero.  The smaller parts' products go first, so the cuts that
  count are those at a sum's full size: on the way through a chunk of d_k = 128,
  8 for S k, 4 + 24 for the solve and 4 for the update, ``TCGEN05`` = 40 2^-24 =
  2.4e-6.  The walk on mma.sync adds part by part: 12 + 24 + 12 for d_k = 64.
  Operands of two parts, off by 2^-17 of their value, would exceed both.
* o, where it is small beside the state: q S and P U cancel, so the error is that of
  the state's read-out, of which two parts are used.  They leave a third of at most
  2^-17 of each element, of either sign: 2^-17 / sqrt(3) as a root mean square, for a
  state of entries of size s and |q| = 1 that is s 2^-17 / sqrt(3); the sums' cuts, 8 at
  the read-out's and 24 at P U's size, come on top (plus 8 for mma.sync's order).
* o as it is rounded.  An error e of the value moves its rounding by a whole step u with
  probability |e| / u, so the distance of o from the right value's rounding is, squared,
  the mean of |e| u, and u <= 2^-7 of the value: at most 2^-7 e, with e the error's size.
  From a state of zeros, one chunk: 4 cuts at full size for the solve and 4 for P U, and 16
  roundings of 2^-24 for the solve itself (24 2^-24): 1.06e-4.  Kernels with U and P in two
  parts were at 1.1e-4 to 1.5e-4.
"""
import math

import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import plain64
from tests.test_gdr import BF16, check, draw, expect_prefill, pool

gpu = pytest.mark.gpu
TCGEN05, MMA_SYNC = 40 * 2.0 ** -24, 48 * 2.0 ** -24
READ_OUT = 2.0 ** -17 / math.sqrt(3) + 40 * 2.0 ** -24
ROUNDED = math.sqrt(2.0 ** -7 * 24 * 2.0 ** -24)
HUGE = 2.0 ** 14  # entries of the state beside values of 1


# ------------------------------------------------------------------ on the CPU
def parts(x, n, cut=False):
    """x [float64, of fp32 values] as n bf16 parts."""
    out, rest = [], x.float()
    for _ in range(n):
        p = ((rest.view(torch.int32) & -65536).view(torch.float32) if cut
             else rest.to(torch.bfloat16).float())
        out.append(p.double())
        rest = rest - p
    return out, rest


def test_three_parts_are_exact():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(100000, generator=g) * torch.exp(8 * torch.randn(100000, generator=g))
    _, two = parts(x, 2)
    _, three = parts(x, 3)
    assert (three == 0).all()
    assert (two.abs() <= 2.0 ** -17 * x.abs()).all()


def product(a, b, n):
    """a b with both operands in n parts, the products of parts of order n and more left out."""
    pa, pb = parts(a, n)[0], parts(b, n)[0]
    return sum(pa[i] @ pb[j] for i in range(n) for j in range(n - i))


def chunk(k, v, S, n=3, n_out=3, n_read=2, cut=False, q=None):
    """One chunk with beta = 1 and no decay of one head (q = k if not given), in 64 bits apart
    from the parts of the state's way, of P U and of the read-out: (o, the state behind it)."""
    q = k if q is None else q
    A = torch.tril(k @ k.T, -1)
    T, P = torch.linalg.inv(torch.eye(len(k), dtype=torch.float64) + A), torch.tril(q @ k.T)
    X = sum(k @ p for p in parts(S, n)[0])
    U = product(T, v - X, n)
    Y = sum(q @ p for p in parts(S, n_read, cut)[0])
    return Y + product(P, U, n_out), S + sum(k.T @ p for p in parts(U, n)[0])


def test_what_fewer_parts_would_cost():
    """The bounds tell three parts from two, and rounded parts from parts cut off."""
    g = torch.Generator().manual_seed(9)
    k = plain64.unit(torch.randn(64, 128, generator=g).to(BF16).double(), 0.0)
    v = torch.randn(64, 128, generator=g).to(BF16).double()
    S = torch.randn(128, 128, generator=g).double()

    def off(x, y):
        return float(torch.linalg.norm(x - y) / torch.linalg.norm(y))

    # beta = 1, q = k: v is what is read back
    assert off(chunk(k, v, HUGE * S, n_read=3)[0], v) < HUGE * 2.0 ** -20
    assert off(chunk(k, v, HUGE * S)[0], v) < HUGE * READ_OUT / 2
    assert off(chunk(k, v, HUGE * S, n_out=2, cut=True)[0], v) > HUGE * READ_OUT
    exact = S + k.T @ torch.linalg.solve(torch.eye(64, dtype=torch.float64) + torch.tril(k @ k.T, -1), v - k @ S)
    assert off(chunk(k, v, S)[1], exact) < 2.0 ** -22
    assert off(chunk(k, v, S, n=2)[1], exact) > MMA_SYNC
    # as rounded, from a state of zeros
    q, zero = plain64.unit(torch.randn(64, 128, generator=g).to(BF16).double(), 0.0), torch.zeros_like(S)
    right = (torch.tril(q @ k.T) @ torch.linalg.solve(torch.eye(64, dtype=torch.float64)
                                                      + torch.tril(k @ k.T, -1), v)).to(BF16)
    assert off(chunk(k, v, zero, q=q)[0].to(BF16).double(), right.double()) < ROUNDED / 2


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("dk, dv, tol", [(128, 128, TCGEN05), (64, 256, TCGEN05), (64, 64, MMA_SYNC),
                                         (32, 256, MMA_SYNC)])
@pytest.mark.parametrize("decay", ["mixed", "none"])
def test_states(dk, dv, tol, decay):
    T, Hk, Hv = 333, 1, 3
    args = draw((T,), Hk, Hv, dk, dv, BF16, decay=decay, seed=21)
    S0 = pool(1, Hv, dk, dv)
    o, S = kda.kda_gdr_prefill(*args, S0, impl="tc")
    _, S_ref = expect_prefill(args, [T], S0)
    check(S, S_ref, tol, "S_T")


@gpu
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 128), (128, 64), (64, 64), (32, 32)])
def test_small_o_beside_a_large_state(dk, dv):
    """Each key's old value is replaced and read back: o is v, what it is read from is 2^14 v."""
    T, H = 64, 2
    _, k, v, la, beta = draw((T,), H, H, dk, dv, BF16, decay="none", seed=22)
    beta = torch.ones_like(beta)
    S0 = torch.randn(1, H, dk, dv, generator=torch.Generator().manual_seed(23)).cuda() * HUGE
    o, _ = kda.kda_gdr_prefill(k, k, v, la, beta, S0, impl="tc")
    o_ref, _ = expect_prefill((k, k, v, la, beta), [T], S0)
    check(o, o_ref, HUGE * READ_OUT / float(o_ref.pow(2).mean().sqrt()), "o")


@gpu
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 128), (128, 64), (32, 32)])
def test_o_as_rounded(dk, dv):
    N, H = 8, 4
    args = draw((64 * N,), H, H, dk, dv, BF16, seed=24)
    o, _ = kda.kda_gdr_prefill(*args, None, N=N, impl="tc")
    o_ref, _ = expect_prefill(args, [64] * N, None)
    right = o_ref.to(BF16).double()
    off = float((o.cpu().double() - right).norm() / right.norm())
    assert off <= ROUNDED, f"{off:.3e} from the rounded value, allowed {ROUNDED:.3e}"

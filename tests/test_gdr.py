"""The gated delta rule: the chunked prefill and the recurrent step against the
64-bit recurrence, their refusals, and sequences that are left out.

Tolerances (2-norm of the error beyond the output's own rounding, over the
2-norm of the result), from the roundings on the way:

* token by token in fp32 (``simt``, the step): every token multiplies the state
  by its decay and adds one product, two roundings of at most 2^-24; the map
  from state to state contracts (|I - beta k k^T| <= 1, e^g <= 1), so errors of
  different tokens add like independent ones: at most 2^-24 sqrt(2 T), plus the
  sqrt(d_k) of the reductions.  For T <= 1000, d_k = 128: 2^-24 (45 + 12) < 2^-18.
* chunks on the tensor cores (``tc``): an operand that is not exact in bf16 is
  the sum of two bf16 parts, off by at most 2^-16 of its value (2^-8 twice); the
  state, the chunk's solve and the products before it each bring one such error
  of random sign, of which 2^-16 is a bound on the root mean square (at most
  2^-18 each, of up to 16 independent ones).
"""
import ctypes

import pytest
import torch

import oracle
from linear_attention_recurrence_prefill_gb300 import kda
from tests import plain64

gpu = pytest.mark.gpu
TOL = {"simt": 2.0 ** -18, "tc": 2.0 ** -16}
BF16, F32 = torch.bfloat16, torch.float32


def draw(rows, Hk, Hv, dk, dv, dtype, seed=0, device="cuda", decay="mixed"):
    """Inputs with token rows `rows` (a tuple)."""
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(*rows, Hk, dk, generator=g) for _ in range(2))
    v = torch.randn(*rows, Hv, dv, generator=g)
    la = -torch.exp(torch.randn(*rows, Hv, generator=g) * 2 - 3)  # from 1e-4 to 10
    if decay == "none":
        la = torch.zeros_like(la)
    beta = torch.sigmoid(torch.randn(*rows, Hv, generator=g))
    to = lambda x: x.to(dtype).to(device)  # noqa: E731
    return to(q), to(k), to(v), la.to(device), to(beta)


def pool(n, Hv, dk, dv, seed=1, device="cuda"):
    return (torch.randn(n, Hv, dk, dv, generator=torch.Generator().manual_seed(seed)) * 0.3).to(device)


def cu_of(lens, device="cuda"):
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int32, device=device)


def check(x, ref, tol, what):
    r = plain64.rel(x, ref)
    assert r <= tol, f"{what}: {r:.3e} beyond rounding, allowed {tol:.3e}"


def expect_prefill(args, lens, S0, **form):
    """o [T, ...] and the final states of packed sequences, S0 [N, ...] or None."""
    o, S, at = [], [], 0
    q, k, v, la, beta = args
    for n, L in enumerate(lens):
        s0 = None if S0 is None else S0[n]
        on, states = plain64.rule(*(x[at:at + L] for x in args), s0, **form)
        o.append(on)
        S.append(plain64.last_state(states, s0, (v.shape[1], q.shape[2], v.shape[2])))
        at += L
    return torch.cat(o), torch.stack(S)


# ------------------------------------------------------------------ on the CPU
def test_plain_rule_is_the_oracles_rule():
    """With as many query heads as value heads and decays above the floor, the plain
    recurrence is the oracle's with its decay broadcast over the channels."""
    q, k, v, la, beta = draw((40,), 3, 3, 32, 32, F32, device="cpu")
    la = la.clamp(min=-4.9)
    S0 = pool(1, 3, 32, 32, device="cpu")
    o, states = plain64.rule(q, k, v, la, beta, S0[0])
    o_ref, S_ref = oracle.prefill(q, k, v, la[..., None].expand(40, 3, 32).contiguous(), beta, S0)
    assert abs(o.numpy() - o_ref).max() < 1e-11
    assert abs(states[-1].numpy() - S_ref[0]).max() < 1e-11


def test_options_defaults():
    o = kda.kda_gdr_options_init()
    assert (o.l2norm_qk, o.beta_is_logit, o.decay_from_logit, o.impl) == (1, 0, 0, 0)
    assert o.q_scale == 1.0 and abs(o.eps_l2 - 1e-6) < 1e-12
    assert not o.slots and not o.snapshots and not o.workspace
    assert (o.ldq, o.ldk, o.ldv, o.n_slots, o.max_seqlen) == (0, 0, 0, 0, 0)
    # on LP64: 3 ints and padding, 2 pointers, 2 floats, 3 long longs, a pointer, an int and
    # padding, a pointer, 2 ints, a pointer, a size_t
    assert ctypes.sizeof(kda.kda_gdr_options) == 16 + 16 + 8 + 24 + 8 + 8 + 8 + 8 + 8 + 8


A = 0x10000  # a 16-byte aligned stand-in address, never dereferenced
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="refusals use stand-in addresses: only where nothing can launch")


def _prefill(opt=None, **kw):
    a = dict(q=A, k=A, v=A, la=A, beta=A, S0=None, cu=None, N=1, o=A, S=A, T=64, Hk=2, Hv=4, dk=64,
             dv=128, dtype=kda.KDA_BF16) | kw
    opt = opt or kda.kda_gdr_options_init()
    return kda.load().kda_gdr_prefill(a["q"], a["k"], a["v"], a["la"], a["beta"], a["S0"], a["cu"],
                                      a["N"], a["o"], a["S"], a["T"], a["Hk"], a["Hv"], a["dk"],
                                      a["dv"], a["dtype"], ctypes.byref(opt), None)


def _step(opt=None, **kw):
    a = dict(q=A, k=A, v=A, la=A, beta=A, S=A, o=A, N=2, L=1, Hk=2, Hv=4, dk=64, dv=128,
             dtype=kda.KDA_BF16) | kw
    opt = opt or kda.kda_gdr_options_init()
    return kda.load().kda_gdr_decode_step(a["q"], a["k"], a["v"], a["la"], a["beta"], a["S"], a["o"],
                                          a["N"], a["L"], a["Hk"], a["Hv"], a["dk"], a["dv"],
                                          a["dtype"], ctypes.byref(opt), None)


SHARED = [
    (dict(q=None), {}, kda.KDA_ERR_ARG), (dict(k=None), {}, kda.KDA_ERR_ARG),
    (dict(v=None), {}, kda.KDA_ERR_ARG), (dict(la=None), {}, kda.KDA_ERR_ARG),
    (dict(beta=None), {}, kda.KDA_ERR_ARG), (dict(o=None), {}, kda.KDA_ERR_ARG),
    (dict(S=None), {}, kda.KDA_ERR_ARG),
    (dict(N=0), {}, kda.KDA_ERR_SHAPE), (dict(Hk=0), {}, kda.KDA_ERR_SHAPE),
    (dict(Hk=3), {}, kda.KDA_ERR_SHAPE), (dict(Hv=0), {}, kda.KDA_ERR_SHAPE),
    (dict(Hk=65536, Hv=65536), {}, kda.KDA_ERR_SHAPE),
    (dict(dk=256), {}, kda.KDA_ERR_UNSUPPORTED), (dict(dk=48), {}, kda.KDA_ERR_UNSUPPORTED),
    (dict(dv=96), {}, kda.KDA_ERR_UNSUPPORTED), (dict(dtype=7), {}, kda.KDA_ERR_DTYPE),
    (dict(q=A + 8), {}, kda.KDA_ERR_ALIGN), (dict(v=A + 2), {}, kda.KDA_ERR_ALIGN),
    (dict(S=A + 4), {}, kda.KDA_ERR_ALIGN), (dict(o=A + 8), {}, kda.KDA_ERR_ALIGN),
    (dict(la=A + 2), {}, kda.KDA_ERR_ALIGN), (dict(beta=A + 1), {}, kda.KDA_ERR_ALIGN),
    ({}, dict(l2norm_qk=2), kda.KDA_ERR_ARG), ({}, dict(beta_is_logit=-1), kda.KDA_ERR_ARG),
    ({}, dict(decay_from_logit=5), kda.KDA_ERR_ARG), ({}, dict(eps_l2=-1.0), kda.KDA_ERR_ARG),
    ({}, dict(q_scale=float("nan")), kda.KDA_ERR_ARG),
    ({}, dict(ldq=64), kda.KDA_ERR_SHAPE), ({}, dict(ldk=129), kda.KDA_ERR_ALIGN),
    ({}, dict(ldv=516), kda.KDA_ERR_ALIGN), ({}, dict(ldv=-512), kda.KDA_ERR_SHAPE),
    ({}, dict(slots=A), kda.KDA_ERR_SHAPE), ({}, dict(slots=A + 2, n_slots=4), kda.KDA_ERR_ALIGN),
    ({}, dict(decay_scale=A + 2), kda.KDA_ERR_ALIGN), ({}, dict(decay_bias=A + 1), kda.KDA_ERR_ALIGN),
]


@no_gpu
@pytest.mark.parametrize("kw, opt, status", SHARED)
def test_refusals_shared(kw, opt, status):
    assert _prefill(kda.kda_gdr_options_init(**opt), **kw) == status
    assert _step(kda.kda_gdr_options_init(**opt), **kw) == status


@no_gpu
def test_refusals_of_one():
    assert _prefill(T=-1) == kda.KDA_ERR_SHAPE
    assert _prefill(T=65, N=2) == kda.KDA_ERR_SHAPE
    assert _prefill(cu=A + 2) == kda.KDA_ERR_ALIGN
    assert _prefill(S0=A + 8) == kda.KDA_ERR_ALIGN
    assert _prefill(kda.kda_gdr_options_init(max_seqlen=65)) == kda.KDA_ERR_SHAPE
    assert _prefill(kda.kda_gdr_options_init(max_seqlen=-1)) == kda.KDA_ERR_SHAPE
    assert _prefill(kda.kda_gdr_options_init(impl=9)) == kda.KDA_ERR_UNSUPPORTED
    assert _prefill(kda.kda_gdr_options_init(snapshots=A)) == kda.KDA_ERR_UNSUPPORTED
    assert _prefill(kda.kda_gdr_options_init(impl="tc"), dtype=kda.KDA_F32) == kda.KDA_ERR_UNSUPPORTED
    assert _step(L=0) == kda.KDA_ERR_SHAPE
    assert _step(N=1 << 20, L=1 << 12) == kda.KDA_ERR_SHAPE
    assert _step(kda.kda_gdr_options_init(snapshots=A + 8)) == kda.KDA_ERR_ALIGN


def test_path():
    """Chunks on the tensor cores for bf16 from 17 tokens on (49 with small heads)."""
    path = kda.kda_gdr_prefill_path
    o = kda.kda_gdr_options_init
    assert path(17, 1, 2, 4, 128, 128) == "tc" and path(16, 1, 2, 4, 128, 128) == "simt"
    assert path(49, 1, 2, 4, 64, 64) == "tc" and path(48, 1, 2, 4, 64, 64) == "simt"
    assert path(4096, 256, 2, 4, 128, 128, kda.KDA_BF16, o(max_seqlen=16)) == "simt"
    assert path(4096, 256, 2, 4, 128, 128, kda.KDA_F32) == "simt"
    assert path(4096, 1, 2, 4, 128, 128, kda.KDA_BF16, o(impl="simt")) == "simt"
    assert path(1, 1, 2, 4, 128, 128, kda.KDA_BF16, o(impl="tc")) == "tc"
    size = kda.kda_gdr_prefill_workspace_size
    assert size(16, 1, 2, 4, 128, 128) == 0
    # a block of 41 KB per value head and chunk, 4096 / 64 + 3 chunks at most
    assert size(4096, 3, 2, 4, 128, 128) == 67 * 4 * 41 * 1024
    assert size(4096, 3, 2, 4, 128, 128, kda.KDA_F32) == 0


def test_binding_refuses():
    q, k, v, la, beta = draw((8,), 2, 4, 32, 32, BF16, device="cpu")
    with pytest.raises(ValueError):  # not on a GPU
        kda.kda_gdr_prefill(q, k, v, la, beta)
    with pytest.raises(ValueError):
        kda._token_stride(torch.zeros(4, 2, 32)[:, :, ::2], "q")
    with pytest.raises(ValueError):
        kda._token_stride(torch.zeros(4, 2, 32).transpose(0, 1), "q")
    with pytest.raises(ValueError):  # [N, L] rows that are not evenly spaced
        kda._token_stride(torch.zeros(3, 8, 2, 32)[:, :4], "q")
    for x in (torch.zeros(1, 2, 32).expand(4, 2, 32), torch.zeros(3, 1, 2, 32).expand(3, 4, 2, 32)):
        with pytest.raises(ValueError):  # one token broadcast
            kda._token_stride(x, "q")
    assert kda._token_stride(torch.zeros(9, 6, 32)[:, 2:4], "q") == 6 * 32
    assert kda._token_stride(torch.zeros(3, 4, 6, 32)[..., :2, :], "q") == 6 * 32
    assert kda._token_stride(torch.zeros(3, 1, 6, 32)[:, :, 1:3], "q") == 6 * 32
    assert kda._token_stride(torch.zeros(3, 1, 2, 32), "q") == 0
    with pytest.raises(ValueError):
        kda._expect(torch.zeros(3, 2), "x", (3, 3), F32)
    with pytest.raises(TypeError):
        kda._expect(torch.zeros(3, 2), "x", (3, 2), BF16)
    with pytest.raises(ValueError):
        kda._expect(torch.zeros(2, 3).T, "x", (3, 2), F32)


# ------------------------------------------------------------------ prefill on the GPU
IMPL = [("simt", F32), ("simt", BF16), ("tc", BF16)]


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
@pytest.mark.parametrize("Hk, Hv, dk, dv, lens", [
    (2, 4, 128, 128, [1]), (1, 1, 128, 128, [63, 64, 65]), (2, 6, 128, 128, [0, 130, 2, 0]),
    (1, 2, 64, 64, [200, 16]), (2, 2, 32, 32, [77]), (1, 4, 64, 256, [70]), (1, 2, 128, 256, [100]),
    (2, 2, 32, 128, [129]), (1, 1, 128, 32, [65]), (1, 3, 128, 64, [150]), (4, 4, 64, 32, [17, 17])])
def test_prefill(impl, dtype, Hk, Hv, dk, dv, lens):
    args = draw((sum(lens),), Hk, Hv, dk, dv, dtype)
    S0 = pool(len(lens), Hv, dk, dv)
    o, S = kda.kda_gdr_prefill(*args, S0, cu_of(lens), impl=impl)
    o_ref, S_ref = expect_prefill(args, lens, S0)
    assert kda.kda_get_last_error() == kda.KDA_OK
    check(o, o_ref, TOL[impl], "o")
    check(S, S_ref, TOL[impl], "S_T")


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_forms(impl, dtype):
    """Logits of beta and of the decay, no norms, a read-out scale, no initial state,
    sequences of one length."""
    q, k, v, la, beta = draw((3 * 90,), 2, 4, 128, 128, dtype, seed=3)
    k = (k * 0.08).to(dtype)
    z = torch.randn_like(la) * 3
    lb = torch.randn(beta.shape, device="cuda").to(dtype)
    A, b = torch.rand(4, device="cuda") * 8, torch.randn(4, device="cuda")
    for form in (dict(l2norm_qk=False, q_scale=0.25),
                 dict(decay_from_logit=True, decay_scale=A, decay_bias=b),
                 dict(decay_from_logit=True, beta_is_logit=True, eps_l2=0.5),
                 dict(decay_from_logit=True, decay_bias=b)):
        args = (q, k, v, z if form.get("decay_from_logit") else la,
                lb if form.get("beta_is_logit") else beta)
        o, S = kda.kda_gdr_prefill(*args, N=3, impl=impl, **form)
        o_ref, S_ref = expect_prefill(args, [90] * 3, None, **form)
        check(o, o_ref, TOL[impl], f"o {form}")
        check(S, S_ref, TOL[impl], f"S_T {form}")


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_decays_at_the_ends(impl, dtype):
    """No decay at all, positive log decays (taken as 0), minus infinity (a forgotten
    past), decays far below fp32's range followed by mild ones; beta 0 and 1."""
    q, k, v, la, beta = draw((140,), 1, 2, 128, 128, dtype, seed=4)
    S0 = pool(1, 2, 128, 128)
    la = -torch.rand_like(la) * 0.01
    la[:20] = 0.0
    la[20:30] = 3.0
    la[50] = -float("inf")
    la[70:75] = -1e30
    la[75:80] = -150.0
    la[130] = -float("inf")
    beta[90:100] = 0.0
    beta[100:110] = 1.0
    o, S = kda.kda_gdr_prefill(q, k, v, la, beta, S0, impl=impl)
    o_ref, S_ref = expect_prefill((q, k, v, la, beta), [140], S0)
    check(o, o_ref, TOL[impl], "o")
    check(S, S_ref, TOL[impl], "S_T")


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_magnitudes(impl, dtype):
    """Values of 1e6 and of 1e-6, keys and queries of 1e4, equal keys, a zero key."""
    for scale in (1e6, 1e-6):
        q, k, v, la, beta = draw((100,), 1, 1, 128, 128, dtype, seed=5)
        q, k, v = (q * 1e4).to(dtype), (k * 1e4).to(dtype), (v * scale).to(dtype)
        k[30:60] = k[30]
        k[70] = 0
        la = la * 0.1
        o, S = kda.kda_gdr_prefill(q, k, v, la, beta, impl=impl)
        o_ref, S_ref = expect_prefill((q, k, v, la, beta), [100], None)
        check(o, o_ref, TOL[impl], f"o {scale}")
        check(S, S_ref, TOL[impl], f"S_T {scale}")


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_in_a_projection_and_a_pool(impl, dtype):
    """q, k and v are slices of one projection's rows; the states sit in a pool, updated
    in place; one sequence is left out."""
    Hk, Hv, d, lens = 2, 4, 128, [33, 64, 0, 100]
    T = sum(lens)
    wide = (torch.randn(T, (2 * Hk + Hv) * d + 64, generator=torch.Generator().manual_seed(6))
            .to(dtype).cuda())
    q = wide[:, 64:64 + Hk * d].view(T, Hk, d)
    k = wide[:, 64 + Hk * d:64 + 2 * Hk * d].view(T, Hk, d)
    v = wide[:, 64 + 2 * Hk * d:].view(T, Hv, d)
    _, _, _, la, beta = draw((T,), Hk, Hv, d, d, dtype)
    P = pool(7, Hv, d, d)
    before = P.clone()
    slots = torch.tensor([5, -1, 0, 3], dtype=torch.int32, device="cuda")
    o = torch.full((T, Hv, d), 7.0, dtype=dtype, device="cuda")
    kda.kda_gdr_prefill(q, k, v, la, beta, P, cu_of(lens), o=o, S_T=P, slots=slots, impl=impl)
    assert kda.kda_get_last_error() == kda.KDA_OK
    S0 = before[torch.tensor([5, 0, 0, 3])]
    o_ref, S_ref = expect_prefill((q, k, v, la, beta), lens, S0)
    out = torch.zeros(T, dtype=torch.bool)
    out[33:97] = True
    assert (o[out] == 7).all()
    check(o[~out], o_ref[~out], TOL[impl], "o")
    check(P[[5, 0, 3]], S_ref[[0, 2, 3]], TOL[impl], "pool")
    assert torch.equal(P[[1, 2, 4, 6]], before[[1, 2, 4, 6]])


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_leaves_out_what_is_out_of_range(impl, dtype):
    """A slot out of range, a slot taken twice, token offsets out of range: those sequences
    are left out and reported, the others are right."""
    Hk, Hv, d, lens = 1, 2, 128, [20, 70, 30]
    args = draw((120,), Hk, Hv, d, d, dtype)
    for slots, good in (([1, 4, 0], [0, 2]), ([2, 2, 0], [0, 2]), ([0, 1, 1 << 30], [0, 1])):
        P = pool(4, Hv, d, d)
        before = P.clone()
        kda.kda_gdr_prefill(*args, P, cu_of(lens), S_T=P, impl=impl,
                            slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE
        assert kda.kda_get_last_error() == kda.KDA_OK
        _, S_ref = expect_prefill(args, lens, torch.stack([before[s % 4] for s in slots]))
        for n in good:
            check(P[slots[n]], S_ref[n], TOL[impl], f"state {n}")
        rest = [i for i in range(4) if i not in [slots[n] for n in good]]
        assert torch.equal(P[rest], before[rest])
    for cu, good in (([0, 20, 10, 120], [0]), ([0, 20, 90, 121], [0, 1]), ([-1, 20, 90, 120], [1, 2])):
        S0 = pool(3, Hv, d, d)
        S = torch.full_like(S0, 5.0)
        kda.kda_gdr_prefill(*args, S0, torch.tensor(cu, dtype=torch.int32, device="cuda"), S_T=S,
                            impl=impl)
        assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE
        for n in good:
            _, S_ref = expect_prefill([x[cu[n]:cu[n + 1]] for x in args], [cu[n + 1] - cu[n]], S0[n:n + 1])
            check(S[n], S_ref[0], TOL[impl], f"state {n}")


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_keeps_what_is_not_finite_to_itself(impl, dtype):
    """NaN and infinity in one sequence, and in the rows behind the last one: the neighbours on
    either side, whose chunks end inside the same 64 rows, do not see them; nor do other columns
    see one of v."""
    lens = [70, 40, 90]
    q, k, v, la, beta = draw((230,), 1, 2, 128, 128, dtype, seed=40)  # 30 rows of no sequence
    S0 = pool(3, 2, 128, 128)
    clean = [x[:200].clone() for x in (q, k, v, la, beta)]
    for x in (q, k, v, la, beta):
        x[200:] = float("nan")
    q[70] = float("inf")
    k[75] = float("nan")
    la[80] = float("nan")
    args = [x[:200] for x in (q, k, v, la, beta)]
    o, S = kda.kda_gdr_prefill(*args, S0, cu_of(lens), impl=impl)
    o_ref, S_ref = expect_prefill(clean, lens, S0)
    keep = torch.ones(200, dtype=torch.bool)
    keep[70:110] = False
    check(o[keep], o_ref[keep], TOL[impl], "o")
    check(S[[0, 2]], S_ref[[0, 2]], TOL[impl], "states")
    assert S[1].isnan().any()
    args = [x.clone() for x in clean]
    args[2][20, 1, 5] = float("inf")
    o, S = kda.kda_gdr_prefill(*args, S0, cu_of(lens), impl=impl)
    cols = [i for i in range(128) if i != 5]
    check(o[:, 1][:, cols], o_ref[:, 1][:, cols], TOL[impl], "o")
    check(S[..., cols], S_ref[..., cols], TOL[impl], "states")
    check(o[:, 0], o_ref[:, 0], TOL[impl], "o of the other head")
    assert not torch.isfinite(S[0, 1, :, 5]).all()


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_of_many_sequences(impl, dtype):
    """More sequences than a warp has lanes, some empty, some left out, states in a pool."""
    g = torch.Generator().manual_seed(41)
    lens = torch.randint(0, 40, (70,), generator=g).tolist()
    lens[3] = 0
    lens[50] = 130
    args = draw((sum(lens),), 1, 2, 64, 64, dtype, seed=42)
    slots = torch.randperm(80, generator=g)[:70].to(torch.int32)
    slots[7] = -1
    slots[60] = slots[2]
    slots[61] = 80
    P = pool(80, 2, 64, 64)
    before = P.clone()
    o = torch.full_like(args[2], 9.0)
    kda.kda_gdr_prefill(*args, P, cu_of(lens), o=o, S_T=P, slots=slots.cuda(), impl=impl)
    assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE
    out = (7, 60, 61)
    o_ref, S_ref = expect_prefill(args, lens, before[[s % 80 if s >= 0 else 0 for s in slots.tolist()]])
    used, at = [], 0
    for n, L in enumerate(lens):
        if n in out:
            assert (o[at:at + L] == 9).all()
        else:
            if L:
                check(o[at:at + L], o_ref[at:at + L], TOL[impl], f"o {n}")
            check(P[slots[n]], S_ref[n], TOL[impl], f"state {n}")
            used.append(int(slots[n]))
        at += L
    rest = [i for i in range(80) if i not in used]
    assert torch.equal(P[rest], before[rest])


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_split_equals_whole(impl, dtype):
    args = draw((150,), 1, 2, 128, 128, dtype, seed=8)
    _, whole = kda.kda_gdr_prefill(*args, impl=impl)
    _, S = kda.kda_gdr_prefill(*(x[:75].contiguous() for x in args), impl=impl)
    _, S = kda.kda_gdr_prefill(*(x[75:].contiguous() for x in args), S, S_T=S, impl=impl)
    check(S, whole.cpu().double(), 2 * TOL[impl], "S_T")


@gpu
def test_prefill_without_tokens():
    S0 = pool(2, 2, 64, 64)
    q = torch.zeros(0, 1, 64, dtype=BF16, device="cuda")
    v = torch.zeros(0, 2, 64, dtype=BF16, device="cuda")
    la = torch.zeros(0, 2, device="cuda")
    o, S = kda.kda_gdr_prefill(q, q, v, la, la.to(BF16), S0, N=2)
    assert o.numel() == 0 and torch.equal(S, S0)
    _, S = kda.kda_gdr_prefill(q, q, v, la, la.to(BF16), None, N=2)
    assert (S == 0).all()


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_repeats_to_the_bit(impl, dtype):
    lens = [65, 300, 1, 40]
    args = draw((sum(lens),), 2, 4, 128, 128, dtype, seed=9)
    a = kda.kda_gdr_prefill(*args, None, cu_of(lens), impl=impl)
    b = kda.kda_gdr_prefill(*args, None, cu_of(lens), impl=impl)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
@pytest.mark.parametrize("impl, dtype", IMPL)
def test_prefill_captured_and_on_two_streams(impl, dtype):
    """Two captured graphs with a workspace each, replayed side by side on inputs written
    after the capture."""
    n = 200
    sets = []
    for i in range(2):
        args = draw((n,), 1, 2, 128, 128, dtype, seed=20 + i)
        o = torch.empty(n, 2, 128, dtype=dtype, device="cuda")
        S = torch.empty(1, 2, 128, 128, device="cuda")
        opt = kda.kda_gdr_options_init(impl=impl)
        need = kda.kda_gdr_prefill_workspace_size(n, 1, 1, 2, 128, 128, kda._dtype_code(o), opt)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        kda.kda_gdr_prefill(*args, o=o, S_T=S, workspace=ws, impl=impl)  # loads the kernels
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_gdr_prefill(*args, o=o, S_T=S, workspace=ws, impl=impl)
        sets.append((args, o, S, ws, g))
    new = [draw((n,), 1, 2, 128, 128, dtype, seed=30 + i) for i in range(2)]
    for (args, o, S, _, _), x in zip(sets, new):
        for dst, src in zip(args, x):
            dst.copy_(src)
        o.zero_()
        S.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for (_, _, _, _, g), st in zip(sets, streams):
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for (_, o, S, _, _), x in zip(sets, new):
        o_ref, S_ref = expect_prefill(x, [n], None)
        check(o, o_ref, TOL[impl], "o")
        check(S, S_ref, TOL[impl], "S_T")


# ------------------------------------------------------------------ the step on the GPU
@gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N, L, Hk, Hv, dk, dv", [
    (1, 1, 1, 1, 128, 128), (3, 1, 2, 6, 128, 128), (2, 5, 1, 2, 64, 256), (5, 2, 2, 2, 32, 32),
    (1, 9, 1, 4, 128, 64), (70, 1, 1, 2, 32, 128)])
def test_step(dtype, N, L, Hk, Hv, dk, dv):
    args = draw((N, L), Hk, Hv, dk, dv, dtype, seed=11)
    S = pool(N, Hv, dk, dv)
    before = S.clone()
    o, snaps = kda.kda_gdr_decode_step(*args, S, snapshots=True)
    assert kda.kda_get_last_error() == kda.KDA_OK
    for n in range(N):
        o_ref, states = plain64.rule(*(x[n] for x in args), before[n])
        check(o[n], o_ref, TOL["simt"], f"o {n}")
        check(snaps[n], torch.stack(states), TOL["simt"], f"states {n}")
    assert torch.equal(S, snaps[:, -1])


@gpu
def test_step_one_token_rows_and_slots():
    """[N, H, d] rows inside a wider projection, a pool, padding rows (slot -1), a slot
    taken twice."""
    N, Hk, Hv, d = 6, 2, 4, 128
    wide = torch.randn(N, (2 * Hk + Hv) * d, device="cuda").to(BF16)
    q = wide[:, :Hk * d].view(N, Hk, d)
    k = wide[:, Hk * d:2 * Hk * d].view(N, Hk, d)
    v = wide[:, 2 * Hk * d:].view(N, Hv, d)
    _, _, _, la, beta = draw((N,), Hk, Hv, d, d, BF16)
    P = pool(9, Hv, d, d)
    before = P.clone()
    slots = [8, -1, 2, 8, -1, 0]
    o = torch.full((N, Hv, d), 3.0, dtype=BF16, device="cuda")
    kda.kda_gdr_decode_step(q, k, v, la, beta, P, o, slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE
    for n in (0, 2, 5):
        o_ref, states = plain64.rule(*(x[n:n + 1] for x in (q, k, v, la, beta)), before[slots[n]])
        check(o[n], o_ref[0], TOL["simt"], f"o {n}")
        check(P[slots[n]], states[0], TOL["simt"], f"state {n}")
    assert (o[[1, 3, 4]] == 3).all()
    assert torch.equal(P[[1, 3, 4, 5, 6, 7]], before[[1, 3, 4, 5, 6, 7]])


@gpu
def test_step_far_into_a_pool():
    """A slot whose offset passes 2^31 elements, and 2^32."""
    Hv, d = 96, 128
    n = 2800  # 2800 * 96 * 128 * 128 = 4.4e9 elements, 17.6 GB
    P = torch.empty(n, Hv, d, d, device="cuda")
    args = draw((2,), 48, Hv, d, d, BF16, seed=13)
    at = [1400, 2799]
    before = [pool(1, Hv, d, d, seed=i)[0] for i in at]
    for i, b in zip(at, before):
        P[i] = b
    slots = torch.tensor(at, dtype=torch.int32, device="cuda")
    o = kda.kda_gdr_decode_step(*args, P, slots=slots)
    for j in range(2):
        o_ref, states = plain64.rule(*(x[j:j + 1] for x in args), before[j])
        check(o[j], o_ref[0], TOL["simt"], "o")
        check(P[at[j]], states[0], TOL["simt"], "state")
    _, S = kda.kda_gdr_prefill(*args, P, N=2, S_T=P, slots=slots)
    assert kda.kda_get_last_error() == kda.KDA_OK


@gpu
def test_steps_equal_prefill():
    args = draw((2 * 70,), 2, 4, 128, 128, BF16, seed=14)
    o, S = kda.kda_gdr_prefill(*args, N=2)
    step = torch.zeros_like(S)
    got = []
    rows = [x.view(2, 70, *x.shape[1:]) for x in args]
    for t in range(0, 70, 7):
        got.append(kda.kda_gdr_decode_step(*(x[:, t:t + 7].contiguous() for x in rows), step))
    check(step, S.cpu().double(), 2 * TOL["tc"], "S")
    check(torch.cat(got, 1).view_as(o), o.cpu().double(), 2.0 ** -8 + 2 * TOL["tc"], "o")


@gpu
def test_step_captured():
    """A decode loop as a graph: the state moves on with every replay."""
    args = draw((4,), 2, 4, 128, 128, BF16, seed=15)
    S = pool(4, 4, 128, 128)
    start = S.clone()
    o = torch.empty(4, 4, 128, dtype=BF16, device="cuda")
    kda.kda_gdr_decode_step(*args, S, o)
    S.copy_(start)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_gdr_decode_step(*args, S, o)
    S.copy_(start)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for n in range(4):
        tokens = [x[n:n + 1].expand(3, *x.shape[1:]) for x in args]
        o_ref, states = plain64.rule(*tokens, start[n])
        check(S[n], states[-1], TOL["simt"], "state")
        check(o[n], o_ref[-1], TOL["simt"], "o")


@gpu
def test_refuses_a_broadcast_workspace():
    """One byte repeated has the size that is asked for, and not the memory."""
    args = draw((200,), 2, 4, 128, 128, BF16)
    need = kda.kda_gdr_prefill_workspace_size(200, 1, 2, 4, 128, 128)
    with pytest.raises(ValueError):
        kda.kda_gdr_prefill(*args, workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(need))


@gpu
def test_a_stream_owns_what_its_calls_allocate(monkeypatch):
    """With ``stream``, workspace and results come from that stream's memory: the workspace is
    given back on return, while the kernels still use it."""
    args = draw((200,), 2, 4, 128, 128, BF16)
    want, S_want = kda.kda_gdr_prefill(*args, impl="tc")
    host, st, seen = kda._host(), torch.cuda.Stream(), []

    def empty(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return torch.empty(*a, **kw)

    def empty_like(x):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return torch.empty_like(x)

    monkeypatch.setattr(host, "empty", empty)
    monkeypatch.setattr(host, "empty_like", empty_like)
    torch.cuda.synchronize()
    before = torch.cuda.current_stream().cuda_stream
    for stream in (st, st.cuda_stream):
        o, S_T = kda.kda_gdr_prefill(*args, impl="tc", stream=stream)
        st.synchronize()
        assert torch.equal(o, want) and torch.equal(S_T, S_want)
    x = torch.randn(8, 64, device="cuda").to(BF16)
    torch.cuda.synchronize()
    y = kda.kda_linear(x, x, stream=st)
    st.synchronize()
    assert torch.equal(y, kda.kda_linear(x, x))
    assert len(seen) == 8 and seen[:7] == [st.cuda_stream] * 7 and seen[7] == before
    assert torch.cuda.current_stream().cuda_stream == before


@gpu
def test_refuses_a_stream_of_another_device():
    class Other:
        device = torch.device("cuda", torch.cuda.current_device() + 1)
    args = draw((8,), 2, 4, 32, 32, BF16)
    with pytest.raises(ValueError):
        kda.kda_gdr_prefill(*args, stream=Other())


def apart():
    return {x: A * (i + 1) for i, x in enumerate(("q", "k", "v", "la", "beta", "o", "S"))}


@no_gpu
@pytest.mark.parametrize("out, other", [(a, b) for a in "oS" for b in ("q", "k", "v", "la", "beta")]
                         + [("o", "S")])
def test_refuses_an_output_on_an_input(out, other):
    at = apart()
    at[out] = at[other]
    assert _step(**at) == kda.KDA_ERR_ARG
    assert _prefill(kda.kda_gdr_options_init(impl="simt"), **at) == kda.KDA_ERR_ARG


@no_gpu
def test_refuses_shared_states_and_scratch():
    at = apart()
    for x in ("S", "q", "o"):
        assert _step(kda.kda_gdr_options_init(snapshots=at[x]), **at) == kda.KDA_ERR_ARG
    assert _prefill(kda.kda_gdr_options_init(impl="simt"), **at | {"S0": at["o"]}) == kda.KDA_ERR_ARG
    for x in ("S", "o"):
        opt = kda.kda_gdr_options_init(impl="tc", workspace=at[x], workspace_bytes=1 << 30)
        assert _prefill(opt, **at) == kda.KDA_ERR_ARG


def test_path_without_tokens():
    opt = kda.kda_gdr_options_init(impl="tc")
    assert kda.kda_gdr_prefill_path(0, 2, 2, 4, 128, 128, kda.KDA_BF16, opt) == "simt"
    assert kda.kda_gdr_prefill_workspace_size(0, 2, 2, 4, 128, 128, kda.KDA_BF16, opt) == 0


@gpu
@pytest.mark.parametrize("impl", ["auto", "simt", "tc"])
def test_no_tokens_hand_the_states_on(impl):
    args = draw((0,), 2, 4, 128, 128, BF16)
    S0 = pool(2, 4, 128, 128)
    o, S_T = kda.kda_gdr_prefill(*args, S0, cu_of([0, 0]), impl=impl)
    assert o.shape == (0, 4, 128) and torch.equal(S_T, S0)
    assert kda.kda_get_last_error() == kda.KDA_OK


@no_gpu
def test_refuses_tokens_near_two_to_the_31():
    assert _prefill(T=2 ** 31 - 256) == kda.KDA_ERR_SHAPE
    assert _step(N=2 ** 31 - 256, Hk=1, Hv=1, dk=32, dv=32) == kda.KDA_ERR_SHAPE

"""kda_linear against the 64-bit product, its refusals, and a layer's run of the
operators together.  Tolerances: ``plain64.linear`` bounds what an fp32 evaluation
may be off, the output's own rounding comes on top."""
import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import plain64

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(M, K, N, dtype, seed=0, bias=True, residual=True, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    to = lambda x: x.to(dtype).to(device)  # noqa: E731
    x, w = to(torch.randn(M, K, generator=g)), to(torch.randn(N, K, generator=g) * max(K, 1) ** -0.5)
    b = to(torch.randn(N, generator=g)) if bias else None
    r = to(torch.randn(M, N, generator=g)) if residual else None
    return x, w, b, r


def check(y, ref, off):
    e = plain64.excess(y, ref)
    # the rounding to y's type applies to a value that is itself off
    allowed = off * (1 + plain64.half_step(y.dtype))
    worst = (e - allowed).max() if e.numel() else torch.tensor(0.0)
    assert worst <= 0, f"{float(worst):.3e} over the allowed error"


# ------------------------------------------------------------------ on the CPU
A = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="refusals use stand-in addresses: only where nothing can launch")


def _linear(**kw):
    a = dict(x=A, ldx=0, w=A, ldw=0, b=None, r=None, ldr=0, y=A, ldy=0, M=8, N=16, K=32, act=0,
             dtype=kda.KDA_BF16) | kw
    return kda.load().kda_linear(a["x"], a["ldx"], a["w"], a["ldw"], a["b"], a["r"], a["ldr"], a["y"],
                                 a["ldy"], a["M"], a["N"], a["K"], a["act"], a["dtype"], None)


@no_gpu
@pytest.mark.parametrize("kw, status", [
    (dict(M=-1), kda.KDA_ERR_SHAPE), (dict(N=-1), kda.KDA_ERR_SHAPE), (dict(K=-1), kda.KDA_ERR_SHAPE),
    (dict(dtype=2), kda.KDA_ERR_DTYPE), (dict(act=6), kda.KDA_ERR_ARG), (dict(act=-1), kda.KDA_ERR_ARG),
    (dict(ldx=31), kda.KDA_ERR_SHAPE), (dict(ldw=16), kda.KDA_ERR_SHAPE),
    (dict(r=A, ldr=15), kda.KDA_ERR_SHAPE), (dict(ldy=8), kda.KDA_ERR_SHAPE),
    (dict(ldx=-32), kda.KDA_ERR_SHAPE),
    (dict(x=None), kda.KDA_ERR_ARG), (dict(w=None), kda.KDA_ERR_ARG), (dict(y=None), kda.KDA_ERR_ARG),
    (dict(x=A + 1), kda.KDA_ERR_ALIGN), (dict(y=A + 1), kda.KDA_ERR_ALIGN),
    (dict(b=A + 1), kda.KDA_ERR_ALIGN), (dict(dtype=kda.KDA_F32, w=A + 2), kda.KDA_ERR_ALIGN),
    (dict(r=A, y=A, ldr=32, ldy=16), kda.KDA_ERR_ARG),
    (dict(M=0), kda.KDA_OK), (dict(N=0), kda.KDA_OK)])
def test_refusals(kw, status):
    assert _linear(**kw) == status


def test_binding_refuses():
    x, w, b, r = make(4, 8, 6, F32, device="cpu")
    with pytest.raises(ValueError):
        kda.kda_linear(x, w)
    with pytest.raises(ValueError):
        kda._rows(x.T, "x", 8, 4)
    with pytest.raises(ValueError):
        kda._rows(x, "x", 4, 9)
    with pytest.raises(ValueError):
        kda._rows(x[:1].expand(4, 8), "x", 4, 8)
    assert kda._rows(torch.zeros(5, 20)[:, 4:12], "x", 5, 8) == 20
    assert kda._rows(x, "x", 4, 8) == 0


def test_plain_bound_holds_for_fp32():
    """The bound of the plain form holds for an fp32 evaluation by torch."""
    for act in kda.ACTS:
        x, w, b, r = make(20, 300, 30, F32, device="cpu")
        ref, off = plain64.linear(x, w, b, r, act)
        z = x @ w.T + b
        y = plain64.activation(z, act) + r
        check(y, ref, off)


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", [
    (1, 1, 1), (1, 64, 128), (1, 4096, 264), (2, 72, 40), (3, 200, 33), (5, 77, 129), (8, 512, 512), (15, 512, 1000),
    (17, 1024, 384), (31, 8, 8), (33, 136, 72), (64, 256, 520), (65, 1000, 136), (100, 2000, 264),
    (127, 333, 511), (128, 128, 128), (129, 64, 257), (200, 96, 1499), (256, 256, 256), (300, 1304, 777),
    (513, 192, 300), (1000, 40, 130)])
def test_linear(dtype, M, K, N):
    x, w, b, r = make(M, K, N, dtype)
    y = kda.kda_linear(x, w, b, r)
    check(y, *plain64.linear(x, w, b, r))
    y = kda.kda_linear(x, w)
    check(y, *plain64.linear(x, w))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", list(kda.ACTS))
@pytest.mark.parametrize("M", [1, 20, 150])
def test_activations(dtype, act, M):
    x, w, b, r = make(M, 128, 144, dtype, seed=2)
    x = (x * 6).to(dtype)  # arguments out to where the activations are flat
    for bias, res in ((b, r), (None, r), (b, None)):
        y = kda.kda_linear(x, w, bias, res, act=act)
        check(y, *plain64.linear(x, w, bias, res, act))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N, ldx, ldw, ldr, ldy, off", [
    (40, 96, 64, 160, 96, 64, 64, 0), (40, 96, 64, 96, 200, 72, 80, 0), (130, 96, 70, 104, 104, 71, 73, 0),
    (40, 96, 64, 97, 99, 65, 67, 0), (40, 96, 64, 128, 128, 128, 128, 1), (3, 520, 136, 1040, 520, 136, 272, 8)])
def test_strides(dtype, M, K, N, ldx, ldw, ldr, ldy, off):
    """Rows inside wider arrays, at any distance and offset; what lies between them stays."""
    g = torch.Generator().manual_seed(3)

    def part(rows, width, ld, value=None):
        size = (rows, ld + off)
        whole = (torch.randn(size, generator=g) if value is None else torch.full(size, value)).to(dtype).cuda()
        return whole, whole[:, off:off + width]

    _, x = part(M, K, ldx)
    _, w = part(N, K, ldw)
    _, r = part(M, N, ldr)
    whole, y = part(M, N, ldy, 5.0)
    b = torch.randn(N, generator=g).to(dtype).cuda()
    kda.kda_linear(x, w, b, r, y, act="silu")
    check(y, *plain64.linear(x, w, b, r, "silu"))
    outside = torch.ones_like(whole, dtype=torch.bool)
    outside[:, off:off + N] = False
    assert (whole[outside] == 5).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N, off, pad", [
    (1, 77, 50, 1, 3), (2, 333, 130, 3, 0), (40, 1003, 515, 1, 0), (300, 65, 130, 5, 2), (17, 9, 300, 7, 7),
    (600, 1023, 1030, 1, 0)])
def test_unaligned_rows_between_nan(dtype, M, K, N, off, pad):
    """Rows at odd addresses and distances with NaN before, between and behind them."""
    g = torch.Generator().manual_seed(12)

    def part(rows, width, scale):
        flat = torch.full((off + rows * (width + pad) + 16,), float("nan"))
        view = flat[off:off + rows * (width + pad)].view(rows, width + pad)[:, :width]
        view.copy_(torch.randn(rows, width, generator=g) * scale)
        return flat.to(dtype).cuda()[off:off + rows * (width + pad)].view(rows, width + pad)[:, :width]

    x, w, r = part(M, K, 1.0), part(N, K, K ** -0.5), part(M, N, 1.0)
    y = kda.kda_linear(x, w, None, r, act="gelu")
    check(y, *plain64.linear(x, w, None, r, "gelu"))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", [(1, 64, 96), (70, 200, 136), (300, 64, 384)])
def test_residual_in_place(dtype, M, K, N):
    x, w, b, r = make(M, K, N, dtype, seed=4)
    ref, off = plain64.linear(x, w, b, r, "gelu")
    kda.kda_linear(x, w, b, r, r, act="gelu")
    check(r, ref, off)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_empty_sizes(dtype):
    x, w, b, r = make(5, 0, 24, dtype)
    y = kda.kda_linear(x, w, b, r, act="relu")
    check(y, *plain64.linear(x, w, b, r, "relu"))
    assert kda.kda_linear(x[:0], w).shape == (0, 24)
    assert kda.kda_linear(x, w[:0]).shape == (5, 0)


@gpu
@pytest.mark.parametrize("M, K, N", [(1, 128, 128), (40, 256, 200), (300, 256, 300)])
def test_infinities_and_nan_stay_in_their_rows(M, K, N):
    x, w, b, _ = make(M, K, N, BF16, seed=5, residual=False)
    ref, off = plain64.linear(x, w, b)
    x[M // 2, 3] = float("inf")
    w[:, 3] = w[:, 3].abs() + 0.01
    ref, off = plain64.linear(x, w, b)
    y = kda.kda_linear(x, w, b)
    assert (y[M // 2] == float("inf")).all()
    keep = [i for i in range(M) if i != M // 2]
    check(y[keep], ref[keep], off[keep])
    x[M // 2, 5] = float("nan")
    y = kda.kda_linear(x, w, b)
    assert y[M // 2].isnan().all() and torch.isfinite(y[keep]).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", [(1, 4096, 256), (48, 4096, 256), (400, 512, 640)])
def test_repeats_to_the_bit_and_on_streams(dtype, M, K, N):
    x, w, b, r = make(M, K, N, dtype, seed=6)
    y = kda.kda_linear(x, w, b, r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append([kda.kda_linear(x, w, b, r) for _ in range(4)])
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(y, z) for z in o)


@gpu
@pytest.mark.parametrize("M", [1, 64, 300])
def test_captured(M):
    x, w, b, r = make(M, 1024, 512, BF16, seed=7)
    y = kda.kda_linear(x, w, b, r)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_linear(x, w, b, r, y)
    x2 = make(M, 1024, 512, BF16, seed=8)[0]
    x.copy_(x2)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(y, *plain64.linear(x, w, b, r))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_each_reads_what_the_last_wrote(dtype):
    """Products in a row on one stream, each of the forms, every one reading the y of the one before
    and writing over the x of the one before that: as calls and as a replayed graph, against the
    same with the device idle between them."""
    g = torch.Generator().manual_seed(18)
    shapes = []  # (M, D): x [M, D] -> y [M, D]
    for M, D in ((1, 2048), (3, 1024), (64, 2048), (600, 2048), (2, 1001), (40, 515)):
        w = [(torch.randn(D, D, generator=g) * D ** -0.5).to(dtype).cuda() for _ in range(3)]
        shapes.append((torch.randn(M, D, generator=g).to(dtype).cuda(), w))

    def chain(x, ws, bufs, wait):
        for i in range(9):
            kda.kda_linear(x if i == 0 else bufs[(i - 1) % 2], ws[i % 3], None,
                           bufs[i % 2] if i > 1 else None, bufs[i % 2], act="silu" if i % 2 else "none")
            if wait:
                torch.cuda.synchronize()

    for x, ws in shapes:
        want = [torch.zeros_like(x) for _ in range(2)]
        chain(x, ws, want, True)
        got = [torch.zeros_like(x) for _ in range(2)]
        chain(x, ws, got, False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain(x, ws, got, False)
        for b in got:
            b.zero_()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        # a replay starts from buffers that it then overwrites: the same each time
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@gpu
def test_rows_past_two_to_the_31():
    """x and y of more than 2^31 elements: the last rows, at offsets past 32 bits."""
    M, K, N = 270_000, 8192, 8192
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    x[-300:].normal_(generator=torch.Generator("cuda").manual_seed(9))
    x[:-300] = 0
    w = make(1, K, N, BF16, seed=9)[1]
    y = kda.kda_linear(x, w)
    ref, off = plain64.linear(x[-300:], w[:64])
    check(y[-300:, :64], ref, off)
    assert (y[: M - 300: 997] == 0).all()


# ------------------------------------------------------------------ together, as a layer runs them
def _layer(x, p, pool, slots, cu, step):
    """One gated-delta-rule layer on packed tokens x [T, D]: projections, the rule, the gated
    norm, the output projection onto the residual stream."""
    Hk, Hv, d = p["Hk"], p["Hv"], p["d"]
    T = x.shape[0]
    qkv = kda.kda_linear(x, p["w_qkv"], act="silu")
    beta = kda.kda_linear(x, p["w_beta"], act="sigmoid")
    z = kda.kda_linear(x.float(), p["w_decay"])
    gate = kda.kda_linear(x, p["w_gate"], p["b_gate"])
    q, k, v = (qkv[:, a:b].view(T, -1, d) for a, b in
               ((0, Hk * d), (Hk * d, 2 * Hk * d), (2 * Hk * d, (2 * Hk + Hv) * d)))
    form = dict(slots=slots, decay_from_logit=True, decay_scale=p["A"], decay_bias=p["bias"])
    if step:
        o = kda.kda_gdr_decode_step(q, k, v, z, beta, pool, **form)
    else:
        o, _ = kda.kda_gdr_prefill(q, k, v, z, beta, pool, cu, S_T=pool, **form)
    y = kda.kda_gated_rmsnorm(o, gate.view(T, Hv, d))
    return kda.kda_linear(y.view(T, Hv * d), p["w_out"], None, x)


def _layer_plain(x, p, states, lens):
    """The same in 64 bits, each array that the layer stores rounded to its type; the states
    after each sequence's last token."""
    Hk, Hv, d = p["Hk"], p["Hv"], p["d"]
    c = {k: v.cpu() if torch.is_tensor(v) else v for k, v in p.items()}
    x = x.cpu()
    st = lambda y: y.to(BF16)  # noqa: E731
    qkv = st(plain64.linear(x, c["w_qkv"], act="silu")[0])
    beta = st(plain64.linear(x, c["w_beta"], act="sigmoid")[0])
    z = plain64.linear(x.float(), c["w_decay"])[0].float()
    gate = st(plain64.linear(x, c["w_gate"], c["b_gate"])[0]).double()
    T = x.shape[0]
    q, k, v = (qkv[:, a:b].reshape(T, -1, d) for a, b in
               ((0, Hk * d), (Hk * d, 2 * Hk * d), (2 * Hk * d, (2 * Hk + Hv) * d)))
    o, last, at = [], [], 0
    for n, L in enumerate(lens):
        s = slice(at, at + L)
        on, sn = plain64.rule(q[s], k[s], v[s], z[s], beta[s], states[n], decay_from_logit=True,
                              decay_scale=c["A"], decay_bias=c["bias"])
        o.append(on)
        last.append(plain64.last_state(sn, states[n], None))
        at += L
    o = st(torch.cat(o)).double()
    y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + 1e-6) * torch.sigmoid(gate.view(T, Hv, d))
    return plain64.linear(st(y).view(T, Hv * d), c["w_out"], None, x)[0], torch.stack(last)


@gpu
def test_layer_prefill_then_decode():
    """Prompts of ragged lengths, then two decode steps, the states in one pool throughout.

    Each stored array (qkv, beta, gate, o, y) may fall on the other side of a rounding
    boundary than the plain form's, a step of 2^-7 of its value; five such independent
    roundings, each met by a small share of the elements, stay below 2^-7 in the 2-norm.
    The output itself is held to its own rounding on top of that."""
    D, Hk, Hv, d = 256, 2, 4, 64
    g = torch.Generator().manual_seed(17)

    def w(n, k, dtype=BF16):
        return (torch.randn(n, k, generator=g) * k ** -0.5).to(dtype).cuda()

    p = dict(Hk=Hk, Hv=Hv, d=d, w_qkv=w((2 * Hk + Hv) * d, D), w_beta=w(Hv, D), w_decay=w(Hv, D, F32),
             w_gate=w(Hv * d, D), b_gate=w(1, Hv * d)[0], w_out=w(D, Hv * d),
             A=(torch.rand(Hv, generator=g) * 4).cuda(), bias=torch.randn(Hv, generator=g).cuda() - 2)
    lens = [70, 1, 130]
    x = torch.randn(sum(lens), D, generator=g).to(BF16).cuda()
    P = (torch.randn(5, Hv, d, d, generator=g) * 0.1).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    states = P[slots.long()].cpu().double()
    cu = torch.tensor([0, 70, 71, 201], dtype=torch.int32, device="cuda")
    out = _layer(x, p, P, slots, cu, False)
    ref, states = _layer_plain(x, p, states, lens)
    assert plain64.rel(out, ref) <= 2.0 ** -7
    assert plain64.rel(P[slots.long()], states) <= 2.0 ** -7
    for i in range(2):
        x = torch.randn(3, D, generator=g).to(BF16).cuda()
        out = _layer(x, p, P, slots, None, True)
        ref, states = _layer_plain(x, p, states, [1, 1, 1])
        assert plain64.rel(out, ref) <= 2.0 ** -7
        assert plain64.rel(P[slots.long()], states) <= 2.0 ** -7
    assert kda.kda_get_last_error() == kda.KDA_OK


@no_gpu
def test_refuses_an_output_on_an_input():
    at = dict(x=A, w=2 * A, b=3 * A, r=4 * A, y=5 * A)
    for name in ("x", "w", "b"):
        assert _linear(**at | {"y": at[name]}) == kda.KDA_ERR_ARG


@no_gpu
@pytest.mark.parametrize("size", ["M", "N", "K"])
def test_refuses_sizes_near_two_to_the_31(size):
    at = dict(x=A, w=2 * A, y=5 * A)
    assert _linear(**at | {size: 2 ** 31 - 256}) == kda.KDA_ERR_SHAPE

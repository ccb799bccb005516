"""kda_rmsnorm, kda_rmsnorm_i8 and kda_quantize_i8 against 64 bits, and their refusals.

Allowances before the output's own rounding, E = 2^-24: s is one rounded addition (E |s|); the
sum of squares, all of one sign, is off by at most one rounding per addition on an element's way
through it (at most 64 where D is at most 65536: at most 50 of a thread's own, five of a warp, the
rest between warps) and two per square; 1 / sqrt halves that and adds four; two products follow.
So |n| is off by at most (64 + 2) / 2 + 8 = 41 E of itself, and a scale by 40 E.  The integers are
those nearest to the exact quotients: equal."""
import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import plain64

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def make(M, D, dtype, seed=0, residual=True, weight=True, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    to = lambda t, dt=dtype: t.to(dt).to(device)  # noqa: E731
    return (to(torch.randn(M, D, generator=g)), to(1 + 0.2 * torch.randn(D, generator=g), F32) if weight else None,
            to(3 * torch.randn(M, D, generator=g)) if residual else None)


def plain(x, w, res, eps=1e-6, norm=True):
    """(s, n, q, scale) in 64 bits."""
    s = x.cpu().double()
    if res is not None:
        s = s + res.cpu().double()
    p = s if w is None else s * w.cpu().double()
    r = 1 / torch.sqrt((s * s).mean(1, keepdim=True) + eps) if norm else torch.ones(x.shape[0], 1, dtype=torch.float64)
    big = p.abs().amax(1, keepdim=True)
    q = torch.where(big > 0, torch.round(127 * p / torch.where(big > 0, big, torch.ones_like(big))), torch.zeros_like(p))
    return s, p * r, q, (big * r / 127)[:, 0]


def check(got, ref, units):
    e = plain64.excess(got, ref)
    assert (e <= units * E * ref.abs() * (1 + plain64.half_step(got.dtype))).all()


# ------------------------------------------------------------------ on the CPU
A = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="refusals use stand-in addresses: only where nothing can launch")


def _norm(**kw):
    a = dict(x=A, ldx=0, r=None, ldr=0, w=None, s=None, lds=0, y=2 * A, ldy=0, q=None, ldq=0, scale=None, M=8, D=32,
             eps=1e-6, dtype=kda.KDA_BF16) | kw
    return kda.load().kda_rmsnorm(a["x"], a["ldx"], a["r"], a["ldr"], a["w"], a["s"], a["lds"], a["y"], a["ldy"],
                                  a["q"], a["ldq"], a["scale"], a["M"], a["D"], a["eps"], a["dtype"], None)


def _quant(**kw):
    a = dict(x=A, ldx=0, q=2 * A, ldq=0, scale=3 * A, M=8, D=32, dtype=kda.KDA_BF16) | kw
    return kda.load().kda_quantize_i8(a["x"], a["ldx"], a["q"], a["ldq"], a["scale"], a["M"], a["D"], a["dtype"], None)


I8 = dict(q=5 * A, scale=6 * A)


@no_gpu
@pytest.mark.parametrize("kw, status", [
    (dict(M=-1), kda.KDA_ERR_SHAPE), (dict(D=0), kda.KDA_ERR_SHAPE), (dict(D=-4), kda.KDA_ERR_SHAPE),
    (dict(M=2 ** 31 - 256), kda.KDA_ERR_SHAPE), (dict(D=2 ** 31 - 256), kda.KDA_ERR_SHAPE),
    (dict(dtype=2), kda.KDA_ERR_DTYPE), (dict(eps=-1.0), kda.KDA_ERR_ARG), (dict(eps=float("nan")), kda.KDA_ERR_ARG),
    (dict(ldx=31), kda.KDA_ERR_SHAPE), (dict(ldr=31), kda.KDA_ERR_SHAPE), (dict(lds=31), kda.KDA_ERR_SHAPE),
    (dict(ldy=-32), kda.KDA_ERR_SHAPE), (dict(ldq=31), kda.KDA_ERR_SHAPE),
    (dict(x=None), kda.KDA_ERR_ARG), (dict(y=None), kda.KDA_ERR_ARG), (dict(q=5 * A), kda.KDA_ERR_ARG),
    (dict(scale=5 * A), kda.KDA_ERR_ARG), (dict(x=A + 1), kda.KDA_ERR_ALIGN), (dict(r=A + 1), kda.KDA_ERR_ALIGN),
    (dict(s=A + 1), kda.KDA_ERR_ALIGN), (dict(y=A + 1), kda.KDA_ERR_ALIGN), (dict(w=A + 2), kda.KDA_ERR_ALIGN),
    (dict(q=5 * A, scale=6 * A + 2), kda.KDA_ERR_ALIGN), (dict(y=A), kda.KDA_ERR_ARG),
    (dict(r=3 * A, y=3 * A), kda.KDA_ERR_ARG), (dict(s=2 * A), kda.KDA_ERR_ARG), (dict(w=2 * A), kda.KDA_ERR_ARG),
    (dict(I8, s=5 * A), kda.KDA_ERR_ARG), (dict(I8, x=5 * A), kda.KDA_ERR_ARG), (dict(I8, y=5 * A), kda.KDA_ERR_ARG),
    (dict(I8, y=6 * A), kda.KDA_ERR_ARG), (dict(q=5 * A, scale=5 * A), kda.KDA_ERR_ARG),
    (dict(I8, x=6 * A), kda.KDA_ERR_ARG), (dict(I8, s=6 * A), kda.KDA_ERR_ARG), (dict(s=7 * A, w=7 * A), kda.KDA_ERR_ARG),
    (dict(s=A, lds=40), kda.KDA_ERR_ARG), (dict(r=3 * A, s=3 * A, ldr=40), kda.KDA_ERR_ARG),
    (dict(M=0), kda.KDA_OK)])
def test_refusals(kw, status):
    assert _norm(**kw) == status


@no_gpu
@pytest.mark.parametrize("kw, status", [
    (dict(M=-1), kda.KDA_ERR_SHAPE), (dict(D=0), kda.KDA_ERR_SHAPE), (dict(dtype=3), kda.KDA_ERR_DTYPE),
    (dict(ldx=8), kda.KDA_ERR_SHAPE), (dict(ldq=8), kda.KDA_ERR_SHAPE), (dict(x=None), kda.KDA_ERR_ARG),
    (dict(q=None), kda.KDA_ERR_ARG), (dict(scale=None), kda.KDA_ERR_ARG), (dict(x=A + 1), kda.KDA_ERR_ALIGN),
    (dict(scale=3 * A + 1), kda.KDA_ERR_ALIGN), (dict(q=A), kda.KDA_ERR_ARG), (dict(scale=A), kda.KDA_ERR_ARG),
    (dict(scale=2 * A), kda.KDA_ERR_ARG), (dict(M=0), kda.KDA_OK)])
def test_quantize_refusals(kw, status):
    assert _quant(**kw) == status


def test_binding_refuses():
    x, w, r = make(4, 8, F32, device="cpu")
    for call in (kda.kda_rmsnorm, kda.kda_rmsnorm_i8, kda.kda_quantize_i8):
        with pytest.raises(ValueError):
            call(x)


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, D", [(1, 1), (1, 4096), (2, 7), (3, 32), (5, 33), (4, 64), (9, 255), (7, 256), (6, 264),
                                  (33, 520), (3, 1000), (70, 1024), (3, 2047), (2, 2048), (5, 5000), (2, 8192),
                                  (3, 16384), (2, 16392), (2, 33000), (1, 40001), (400, 128), (1000, 4096), (1000, 96)])
def test_norm(dtype, M, D):
    for residual, weight in ((True, True), (False, True), (True, False), (False, False)):
        x, w, res = make(M, D, dtype, D, residual, weight)
        s, n, q, scale = plain(x, w, res)
        got = kda.kda_rmsnorm(x, w, res)
        y, total = got if residual else (got, None)
        check(y, n, 41)
        if residual:
            check(total, s, 1)
        both = torch.empty_like(x)
        qs, sc, *total = kda.kda_rmsnorm_i8(x, w, res, y=both)
        assert torch.equal(qs.cpu().double(), q)
        check(sc, scale, 40)
        assert torch.equal(both, y) and len(total) == residual
        if residual:
            check(total[0], s, 1)
        if not weight and not residual:
            qs, sc = kda.kda_quantize_i8(x)
            _, _, q, scale = plain(x, None, None, norm=False)
            assert torch.equal(qs.cpu().double(), q)
            check(sc, scale, 2)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, D", [(50, 96), (20, 4096)])
def test_quotients_between_two_integers(dtype, M, D):
    """Values whose quotients lie on, or as near as fp32 gets to, the middle between two integers."""
    g = torch.Generator().manual_seed(1)
    half = torch.randint(-127, 127, (M, D), generator=g) + 0.5
    x = half / 127 * torch.exp(torch.randn(M, 1, generator=g))
    x[:, 0] = torch.exp(torch.randn(M, generator=g)) + x.abs().amax(1)
    big = x[:, :1].to(dtype).float()
    x = (half / 127 * big).to(dtype)
    x[:, 0] = big[:, 0].to(dtype)
    x[:, 1] = x[:, 0] / 2  # exactly 63.5
    x = x.cuda()
    q, _ = kda.kda_quantize_i8(x)
    assert torch.equal(q.cpu().double(), plain(x, None, None, norm=False)[2])
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    q, _ = kda.kda_rmsnorm_i8(x, w)
    assert torch.equal(q.cpu().double(), plain(x, w, None)[2])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, D, ldx, ldr, lds, ldy, ldq, off", [
    (9, 96, 128, 96, 104, 200, 112, 0), (9, 96, 97, 99, 101, 103, 105, 1), (5, 1000, 1001, 1008, 1000, 1016, 1003, 3),
    (17, 40, 48, 48, 48, 48, 48, 8), (4, 4096, 4104, 4096, 4100, 4098, 4097, 2)])
def test_strides(dtype, M, D, ldx, ldr, lds, ldy, ldq, off):
    g = torch.Generator().manual_seed(3)

    def part(ld, dt=dtype, value=None):
        whole = (torch.full((M, ld + off), float("nan")) if value is None else torch.full((M, ld + off), value)).to(dt).cuda()
        view = whole[:, off:off + D]
        if value is None:
            view.copy_(torch.randn(M, D, generator=g))
        return whole, view

    _, x = part(ldx)
    _, res = part(ldr)
    w = torch.randn(D, generator=g).cuda()
    outs = [part(lds, value=5.0), part(ldy, value=5.0), part(ldq, torch.int8, 5.0)]
    s, n, q, scale = plain(x, w, res)
    _, sc, _ = kda.kda_rmsnorm_i8(x, w, res, outs[2][1], total=outs[0][1], y=outs[1][1])
    check(outs[0][1], s, 1)
    check(outs[1][1], n, 41)
    assert torch.equal(outs[2][1].cpu().double(), q)
    check(sc, scale, 40)
    for whole, view in outs:
        outside = torch.ones_like(whole, dtype=torch.bool)
        outside[:, off:off + D] = False
        assert (whole[outside] == 5).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, D", [(3, 64), (40, 4096), (2, 50000)])
def test_sum_in_place(dtype, M, D):
    for which in (0, 2):
        x, w, res = make(M, D, dtype, 5)
        s, n, q, scale = plain(x, w, res)
        into = (x, w, res)[which]
        qs, sc, total = kda.kda_rmsnorm_i8(x, w, res, total=into)
        assert total is into and torch.equal(qs.cpu().double(), q)
        check(into, s, 1)
        x, w, res = make(M, D, dtype, 5)
        into = (x, w, res)[which]
        y, total = kda.kda_rmsnorm(x, w, res, total=into)
        check(y, n, 41)
        check(into, s, 1)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [40, 4096, 40000])
def test_rows_that_are_not_ordinary(dtype, D):
    x, w, _ = make(8, D, dtype, 2, residual=False)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 3] = float("inf")
    x[4] = 0
    x[4, D - 1] = 1e-38  # the only one, and 127 / it overflows
    x[5] = torch.finfo(dtype).tiny * torch.arange(D, device="cuda") / D
    x[6] *= 1e15
    y = kda.kda_rmsnorm(x, w)
    q, scale = kda.kda_rmsnorm_i8(x, w)
    s, n, want, sc = plain(x, w, None)
    ordinary = [0, 1, 4, 5, 6, 7]
    check(scale[[0, 1, 6, 7]], sc[[0, 1, 6, 7]], 40)
    check(y[[0, 1, 6, 7]], n[[0, 1, 6, 7]], 41)
    assert torch.equal(q[ordinary].cpu().double(), want[ordinary])
    assert (q[2:4] == 0).all() and not torch.isfinite(scale[2:4]).any()
    assert y[2].isnan().all() and y[3, 3].isnan()
    q, scale = kda.kda_quantize_i8(x)
    _, _, want, sc = plain(x, None, None, norm=False)
    assert torch.equal(q[ordinary].cpu().double(), want[ordinary])
    assert (q[2:4] == 0).all() and scale[2].isnan() and scale[3] == float("inf")
    assert (kda.kda_rmsnorm(x[1:2], w, eps=0.0) == 0).all()


@gpu
def test_empty_and_captured_and_streams():
    x, w, res = make(0, 64, BF16)
    assert kda.kda_rmsnorm(x, w).shape == (0, 64) and kda.kda_quantize_i8(x)[1].shape == (0,)
    x, w, res = make(100, 1000, BF16)
    first = kda.kda_rmsnorm_i8(x, w, res)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = kda.kda_rmsnorm_i8(x, w, res, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_rmsnorm_i8(x, w, res)
    x.copy_(make(100, 1000, BF16, 7)[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kda.kda_rmsnorm_i8(x, w, res), got))


@gpu
def test_rows_past_two_to_the_31():
    M, D = 530_000, 4096 + 8
    x = torch.zeros(M, D, dtype=BF16, device="cuda")
    x[-5:].normal_(generator=torch.Generator("cuda").manual_seed(9))
    y = kda.kda_rmsnorm(x)
    q, scale = kda.kda_rmsnorm_i8(x)
    s, n, want, sc = plain(x[-5:], None, None)
    check(y[-5:], n, 41)
    check(scale[-5:], sc, 40)
    assert torch.equal(q[-5:].cpu().double(), want) and (q[:-5:1009] == 0).all() and (scale[:-5:1009] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [40, 4096, 20000])
def test_small_rows_without_eps(dtype, D):
    """Squares down to a mean of 2^-100: what is lost of one below 2^-126 is 2^-24 of the mean at most."""
    x, w, _ = make(4, D, dtype, 5, residual=False)
    x *= 2.0 ** -50 * 1.5  # (the mean of the squares of normal numbers is one, and 2.25 here)
    y = kda.kda_rmsnorm(x, w, eps=0.0)
    q, scale = kda.kda_rmsnorm_i8(x, w, eps=0.0)
    s, n, want, sc = plain(x, w, None, eps=0.0)
    assert (s * s).mean(1).min() >= 2.0 ** -100
    check(y, n, 42)
    check(scale, sc, 41)
    assert torch.equal(q.cpu().double(), want)
    x[1:3] = 1e-30  # squares that vanish
    x[2] *= -1
    y = kda.kda_rmsnorm(x, w, eps=0.0)
    q, scale = kda.kda_rmsnorm_i8(x, w, eps=0.0)
    for t in (y, q, scale):
        assert (t[1:3] == 0).all() and (t[[0, 3]] != 0).any()


@gpu
@pytest.mark.parametrize("M, D", [(40, 520), (8, 8192), (3, 20000)])
def test_products_between_two_integers(M, D):
    """Products of a rounded sum and a weight whose quotients lie a few steps of fp32 on either side of
    the middle between two integers: every rounding that the fp32 quotient has counts."""
    g = torch.Generator().manual_seed(11)
    w = 1 + torch.rand(D, generator=g)
    res = torch.randn(M, D, generator=g)
    big = 1 + torch.rand(M, 1, generator=g)
    half = torch.randint(-126, 126, (M, D), generator=g) + 0.5
    s = half.double() / 127 * big.double() / w.double() * (1 + torch.randint(-6, 7, (M, D), generator=g) * 2.0 ** -24)
    s[:, 0] = big[:, 0].double() / w[0].double()
    x = (s - res.double()).float()
    x, w, res = x.cuda(), w.cuda(), res.cuda()
    q, _, _ = kda.kda_rmsnorm_i8(x, w, res)
    assert torch.equal(q.cpu().double(), plain(x, w, res)[2])

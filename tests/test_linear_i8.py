"""kda_linear_i8 against the 64-bit product, its refusals, and a recurrent layer's run of the
operators together.

Allowance before the output's own rounding, E = 2^-24: the integer sum is exact below 2^24, and
beyond it each of at most K / 16 additions of a tensor core's group cuts off at most 2 E of the largest
partial sum (and one conversion rounds); two products with the scales, the bias's addition; then as in
``plain64.linear``."""
import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import glr64, plain64
from tests.test_linear import check

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -24


def make(M, K, N, dtype, seed=0, bias=True, residual=True, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    to = lambda t, dt=dtype: t.to(dt).to(device)  # noqa: E731
    x, w = (to(torch.randint(-128, 128, s, generator=g), torch.int8) for s in ((M, K), (N, K)))
    sx = to(torch.exp(torch.randn(M, generator=g)) / 100, F32)
    sw = to(torch.exp(torch.randn(N, generator=g)) / 100 * max(K, 1) ** -0.5, F32)
    return (x, sx, w, sw, to(torch.randn(N, generator=g)) if bias else None,
            to(torch.randn(M, N, generator=g)) if residual else None)


def plain(x, sx, w, sw, bias=None, residual=None, act="none"):
    x, w, sx, sw = (t.cpu().double() for t in (x, w, sx, sw))
    scales = sx[:, None] * sw
    z, mag = x @ w.T, x.abs() @ w.abs().T
    off = torch.where(mag < 2 ** 24, 2 * E * z.abs(), (x.shape[1] / 8 + 3) * E * mag) * scales
    z = z * scales
    if bias is not None:
        z = z + bias.cpu().double()
        off = off + 2 * E * z.abs()
    y = plain64.activation(z, act)
    if act != "none":
        off = plain64.STEEPEST * off + 16 * E * (y.abs() + z.abs())
    if residual is not None:
        y = y + residual.cpu().double()
        off = off + E * y.abs()
    return y, off


# ------------------------------------------------------------------ on the CPU
A = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="refusals use stand-in addresses: only where nothing can launch")


def _linear(**kw):
    a = dict(x=A, ldx=0, sx=2 * A, w=3 * A, ldw=0, sw=4 * A, b=None, r=None, ldr=0, y=5 * A, ldy=0, M=8, N=16, K=32,
             act=0, dtype=kda.KDA_BF16, ws=6 * A, size=1 << 40) | kw
    return kda.load().kda_linear_i8(a["x"], a["ldx"], a["sx"], a["w"], a["ldw"], a["sw"], a["b"], a["r"], a["ldr"],
                                    a["y"], a["ldy"], a["M"], a["N"], a["K"], a["act"], a["dtype"], a["ws"], a["size"],
                                    None)


@no_gpu
@pytest.mark.parametrize("kw, status", [
    (dict(M=-1), kda.KDA_ERR_SHAPE), (dict(N=-1), kda.KDA_ERR_SHAPE), (dict(K=-1), kda.KDA_ERR_SHAPE),
    (dict(M=2 ** 31 - 256), kda.KDA_ERR_SHAPE), (dict(N=2 ** 31 - 256), kda.KDA_ERR_SHAPE),
    (dict(K=2 ** 31 - 256), kda.KDA_ERR_SHAPE), (dict(dtype=2), kda.KDA_ERR_DTYPE), (dict(act=6), kda.KDA_ERR_ARG),
    (dict(act=-1), kda.KDA_ERR_ARG), (dict(ldx=31), kda.KDA_ERR_SHAPE), (dict(ldw=16), kda.KDA_ERR_SHAPE),
    (dict(r=7 * A, ldr=15), kda.KDA_ERR_SHAPE), (dict(ldy=8), kda.KDA_ERR_SHAPE), (dict(x=None), kda.KDA_ERR_ARG),
    (dict(w=None), kda.KDA_ERR_ARG), (dict(y=None), kda.KDA_ERR_ARG), (dict(sx=None), kda.KDA_ERR_ARG),
    (dict(sw=None), kda.KDA_ERR_ARG), (dict(y=A + 1), kda.KDA_ERR_ALIGN), (dict(b=A + 1), kda.KDA_ERR_ALIGN),
    (dict(r=A + 1), kda.KDA_ERR_ALIGN), (dict(sx=A + 2), kda.KDA_ERR_ALIGN), (dict(sw=A + 1), kda.KDA_ERR_ALIGN),
    (dict(dtype=kda.KDA_F32, y=A + 2), kda.KDA_ERR_ALIGN), (dict(r=5 * A, ldr=32, ldy=16), kda.KDA_ERR_ARG),
    (dict(y=A), kda.KDA_ERR_ARG), (dict(y=2 * A), kda.KDA_ERR_ARG), (dict(y=3 * A), kda.KDA_ERR_ARG),
    (dict(y=4 * A), kda.KDA_ERR_ARG), (dict(b=5 * A), kda.KDA_ERR_ARG), (dict(M=0), kda.KDA_OK),
    (dict(N=0), kda.KDA_OK)])
def test_refusals(kw, status):
    assert _linear(**kw) == status


def test_binding_refuses():
    x, sx, w, sw, b, r = make(4, 8, 6, F32, device="cpu")
    with pytest.raises(ValueError):
        kda.kda_linear_i8(x, sx, w, sw)


# ------------------------------------------------------------------ on the GPU
SIZES = [(1, 1, 1), (1, 64, 128), (1, 4096, 264), (2, 72, 40), (3, 200, 33), (4, 1024, 136), (5, 77, 129), (8, 512, 512),
         (15, 512, 1000), (16, 128, 128), (17, 1024, 384), (31, 8, 8), (33, 136, 72), (64, 256, 520), (65, 1008, 136),
         (100, 2000, 264), (127, 333, 511), (128, 128, 128), (129, 64, 257), (200, 96, 1499), (256, 256, 256),
         (300, 1304, 777), (333, 1000, 1499), (513, 192, 300), (1000, 48, 130), (700, 512, 5000), (2500, 272, 2100),
         (400, 4095, 200)]


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", SIZES)
def test_linear_i8(dtype, M, K, N):
    a = make(M, K, N, dtype)
    check(kda.kda_linear_i8(*a), *plain(*a))
    check(kda.kda_linear_i8(*a[:4], dtype=dtype), *plain(*a[:4]))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", list(kda.ACTS))
@pytest.mark.parametrize("M", [1, 20, 150, 1200])
def test_activations(dtype, act, M):
    a = make(M, 128, 2500 if M > 1000 else 144, dtype, seed=2)
    for bias, res in ((a[4], a[5]), (None, a[5]), (a[4], None)):
        check(kda.kda_linear_i8(*a[:4], bias, res, act=act, dtype=dtype), *plain(*a[:4], bias, res, act))


@gpu
@pytest.mark.parametrize("M, K, N", [(1, 12288, 40), (3, 5000, 64), (64, 12288, 130), (200, 9000, 260), (1500, 4112, 2600)])
def test_largest_integers(M, K, N):
    """Sums beyond 2^24, of either sign, in rows and columns of equal integers at both ends."""
    _, sx, _, sw, *_ = make(M, K, N, F32)
    x = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    x[::2], w[::3], x[:, 5::7] = -128, -128, 126
    y, off = plain(x, sx, w, sw)
    check(kda.kda_linear_i8(x, sx, w, sw, dtype=F32), y, off)
    check(kda.kda_linear_i8(x, sx, w, sw), y, off)


@gpu
@pytest.mark.parametrize("M, K, N", [(1, 1024, 500), (7, 1000, 300), (60, 1024, 300), (400, 1016, 300), (1500, 1024, 2600)])
def test_exact_below_two_to_the_24(M, K, N):
    """K up to 1024: no sum exceeds 2^24, and with scales of one the result is the integer."""
    x, _, w, *_ = make(M, K, N, F32, seed=4)
    x[0], w[0] = -128, -128
    one = torch.ones(max(M, N), device="cuda")
    y = kda.kda_linear_i8(x, one[:M], w, one[:N], dtype=F32)
    assert torch.equal(y.double(), (x.double() @ w.double().T))


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N, ldx, ldw, ldr, ldy, off", [
    (40, 96, 64, 160, 96, 64, 64, 0), (40, 96, 64, 96, 208, 72, 80, 0), (130, 96, 70, 112, 128, 71, 73, 0),
    (40, 96, 64, 97, 99, 65, 67, 0), (40, 96, 64, 128, 128, 128, 128, 1), (3, 520, 136, 1040, 528, 136, 272, 16),
    (1, 1000, 50, 1000, 1001, 50, 50, 3), (1200, 100, 2600, 101, 112, 2601, 2608, 5)])
def test_strides(dtype, M, K, N, ldx, ldw, ldr, ldy, off):
    """Rows inside wider arrays, at any distance and offset; what lies between them stays."""
    x0, sx, w0, sw, b, r0 = make(M, K, N, dtype, seed=3)

    def part(t, ld, value):
        whole = torch.full((t.shape[0], ld + off), value, dtype=t.dtype, device="cuda")
        view = whole[:, off:off + t.shape[1]]
        view.copy_(t)
        return whole, view

    x, w, r = part(x0, ldx, 77)[1], part(w0, ldw, -77)[1], part(r0, ldr, float("nan"))[1]
    whole, y = part(r0, ldy, 5.0)
    kda.kda_linear_i8(x, sx, w, sw, b, r, y, act="silu")
    check(y, *plain(x0, sx, w0, sw, b, r0, "silu"))
    outside = torch.ones_like(whole, dtype=torch.bool)
    outside[:, off:off + N] = False
    assert (whole[outside] == 5).all()


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", [(1, 64, 96), (70, 208, 136), (300, 64, 384), (1300, 64, 2500)])
def test_residual_in_place(dtype, M, K, N):
    a = make(M, K, N, dtype, seed=4)
    ref, off = plain(*a, "gelu")
    kda.kda_linear_i8(*a, a[5], act="gelu")
    check(a[5], ref, off)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_empty_sizes(dtype):
    a = make(5, 0, 24, dtype)
    check(kda.kda_linear_i8(*a, act="relu"), *plain(*a, "relu"))
    x, sx, w, sw, *_ = a
    assert kda.kda_linear_i8(x[:0], sx[:0], w, sw).shape == (0, 24)
    assert kda.kda_linear_i8(x, sx, w[:0], sw[:0]).shape == (5, 0)


@gpu
@pytest.mark.parametrize("M", [1, 40, 300, 1500])
def test_scales_that_are_not_finite_stay_in_their_rows(M):
    x, sx, w, sw, *_ = make(M, 256, 2300, BF16, seed=5)
    sx[M // 2], sw[7] = float("nan"), float("inf")
    y = kda.kda_linear_i8(x, sx, w, sw)
    assert y[M // 2].isnan().all() and not torch.isfinite(y[:, 7]).any()
    keep = [i for i in range(M) if i != M // 2]
    cols = [i for i in range(2300) if i != 7]
    ref, off = plain(x[keep], sx[keep], w[cols], sw[cols])
    check(y[keep][:, cols], ref, off)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", [(1, 4096, 256), (48, 4096, 256), (400, 512, 640), (1500, 512, 2600)])
def test_repeats_to_the_bit_on_streams_and_in_graphs(dtype, M, K, N):
    a = make(M, K, N, dtype, seed=6)
    y = kda.kda_linear_i8(*a)
    torch.cuda.synchronize()
    outs = []
    for st in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(st):
            outs += [kda.kda_linear_i8(*a) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, z) for z in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = kda.kda_linear_i8(*a)
    a[0].copy_(make(M, K, N, dtype, seed=8)[0])
    graph.replay()
    torch.cuda.synchronize()
    check(z, *plain(*a))


@gpu
def test_rows_past_two_to_the_31():
    """x and y of more than 2^31 elements: the last rows, at offsets past 32 bits."""
    M, K, N = 270_000, 8192, 8192
    x = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    last, _, w, sw, *_ = make(300, K, N, BF16, seed=9)
    x[-300:] = last
    sx = torch.full((M,), 0.01, device="cuda")
    y = kda.kda_linear_i8(x, sx, w, sw)
    check(y[-300:, :64], *plain(x[-300:], sx[-300:], w[:64], sw[:64]))
    assert (y[: M - 300: 997] == 0).all()


# ------------------------------------------------------------------ together, as a layer runs them
def _layer(x, res, p, pool, slots, cu, step):
    """A recurrent layer in 8 bits on packed tokens: the norm with the residual stream, one projection
    to the recurrence's input, decay and gate, the recurrence, the projection back onto the stream."""
    D, R = p["D"], p["R"]
    q, scale, res = kda.kda_rmsnorm_i8(x, p["w_norm"], res)
    z = kda.kda_linear_i8(q, scale, p["w_in"], p["s_in"], p["b_in"])
    u, la, gate = (z[:, i * R:(i + 1) * R] for i in range(3))
    form = dict(slots=slots, decay_from="sigmoid", decay_scale=p["A"], input_scale="normalized", input_gate=gate)
    if step:
        h = kda.kda_glr_step(u, la, pool, **form)
    else:
        h, _ = kda.kda_glr_scan(u, la, pool, cu, h_T=pool, **form)
    q, scale = kda.kda_quantize_i8(h)
    return kda.kda_linear_i8(q, scale, p["w_out"], p["s_out"]), res


def _layer_plain(x, res, p, h0, lens):
    c = {k: v.cpu() if torch.is_tensor(v) else v for k, v in p.items()}
    R = c["R"]
    st = lambda t: t.to(BF16).double()  # noqa: E731

    def quantized(t):
        scale = t.abs().amax(1, keepdim=True) / 127
        return torch.round(t / scale) * scale

    s = x.cpu().double() + res.cpu().double()
    n = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * c["w_norm"].double()
    z = st(quantized(n) @ (c["w_in"].double() * c["s_in"].double()[:, None]).T + c["b_in"].double())
    f = glr64.Form(z[:, :R], z[:, R:2 * R], decay_from="sigmoid", decay_scale=c["A"], input_scale="normalized",
                   input_gate=z[:, 2 * R:])
    y, end, *_ = glr64.scan(f, h0, lens)
    return quantized(st(y)) @ (c["w_out"].double() * c["s_out"].double()[:, None]).T, st(s), end


@gpu
def test_layer_prefill_then_decode():
    """Prompts of ragged lengths, then two tokens each, the states in one pool throughout.

    Where a stored array falls on the other side of a rounding boundary than the plain form's it
    is a step off: 2^-8 of its value in z and h, 1 / 127 of the row's largest in what is
    quantized from them, both met by a small share of the elements; the outputs stay within 2^-6 in
    the 2-norm, and the states, behind one such array, within 2^-7."""
    D, R = 256, 192
    g = torch.Generator().manual_seed(17)

    def w(n, k):
        t = torch.randn(n, k, generator=g) * k ** -0.5
        scale = t.abs().amax(1) / 127
        return torch.round(t / scale[:, None]).to(torch.int8).cuda(), scale.cuda()

    p = dict(D=D, R=R, w_norm=(1 + 0.1 * torch.randn(D, generator=g)).cuda(),
             b_in=torch.randn(3 * R, generator=g).to(BF16).cuda(), A=torch.rand(R, generator=g).cuda())
    p["w_in"], p["s_in"] = w(3 * R, D)
    p["w_out"], p["s_out"] = w(D, R)
    lens = [70, 1, 130]
    pool = torch.randn(5, R, generator=g).cuda()
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    h = pool[slots.long()].cpu().double()
    cu = torch.tensor([0, 70, 71, 201], dtype=torch.int32, device="cuda")
    for step in (False, True, True):
        T = 3 if step else 201
        x, res = (torch.randn(T, D, generator=g).to(BF16).cuda() for _ in range(2))
        out, total = _layer(x, res, p, pool, slots, None if step else cu, step)
        ref, s, h = _layer_plain(x, res, p, h, [1, 1, 1] if step else lens)
        assert plain64.rel(out, ref) <= 2.0 ** -6
        assert torch.equal(total.cpu().double(), s)
        assert plain64.rel(pool[slots.long()], h) <= 2.0 ** -7
    assert kda.kda_get_last_error() == kda.KDA_OK


@gpu
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 6, 7, 8, 9])
@pytest.mark.parametrize("K, N", [(16, 3), (1040, 67), (4100, 130), (131088, 5)])
def test_few_rows(M, K, N):
    """Each number of rows that is taken as a stream of w, and the next; K beyond a 32-bit sum."""
    a = make(M, K, N, F32, seed=M)
    check(kda.kda_linear_i8(*a, act="silu"), *plain(*a, "silu"))


@gpu
@pytest.mark.parametrize("M, K, N", [(640, 512, 4096), (700, 100, 5000), (330, 77, 19000), (3000, 1, 700), (150, 4095, 4100)])
def test_widened_first(M, K, N):
    """Sizes whose integers are widened into the workspace, with one that is given and holds NaN."""
    a = make(M, K, N, F32, seed=3)
    need = kda.load().kda_linear_i8_workspace_size(M, N, K)
    assert need > 0
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    y = kda.kda_linear_i8(*a, workspace=ws)
    check(y, *plain(*a))
    with pytest.raises(kda.KdaError):
        kda.kda_linear_i8(*a, workspace=ws[:need // 8])


@gpu
@pytest.mark.parametrize("K", [1040, 4096, 12288, 40000])
@pytest.mark.parametrize("M, N", [(1, 300), (8, 300), (9, 300), (64, 300), (200, 300), (1500, 2600)])
def test_bound_of_sums_beyond_two_to_the_24(M, N, K):
    """Integers of one sign: up to eight rows the sum itself, rounded once; beyond, low by at most
    K / 16 additions' 2^-23 of it (and a rounding of each of up to eight parts of K, and the last one).
    Integers of either sign: the sum, which stays below 2^24 at these K."""
    g = torch.Generator().manual_seed(K)
    one = torch.ones(max(M, N), device="cuda")
    for low in (100, -128):
        x, w = (torch.randint(low, 128, (rows, K), generator=g).to(torch.int8).cuda() for rows in (M, N))
        y = kda.kda_linear_i8(x, one[:M], w, one[:N], dtype=F32).double()
        z = x.double() @ w.double().T  # (exact: below 2^53)
        if M <= 8:
            assert torch.equal(y, z.float().double())
        elif low < 0:
            assert z.abs().max() < 2 ** 24 and torch.equal(y, z)
        else:
            assert ((y - z) <= 9 * E * z).all() and ((z - y) <= (K * 2.0 ** -27 + 9 * E) * z).all()


@gpu
def test_a_token_alone_and_in_a_batch():
    """Up to K = 1024 a token's row does not depend on how many others are in the batch, or on the kernel."""
    x, sx, w, sw, b, r = make(1500, 1024, 2600, F32, seed=12)
    x[0] = w[0] = -128
    whole = kda.kda_linear_i8(x, sx, w, sw, b, r)
    for M in (1, 8, 9, 40, 200):
        assert torch.equal(kda.kda_linear_i8(x[:M], sx[:M], w, sw, b, r[:M]), whole[:M])


@no_gpu
@pytest.mark.parametrize("M, N, K, ldx, need", [
    (8, 12288, 4096, 0, False), (64, 12288, 4095, 0, False), (65, 12288, 4095, 0, True), (65, 12288, 4096, 0, False),
    (65, 12288, 4096, 4100, True), (400, 2 ** 20, 4096, 0, False), (384, 12288, 4096, 0, False), (512, 12288, 4096, 0, True),
    (512, 4096, 4096, 0, False), (640, 4096, 4096, 0, True), (128, 4096, 1000, 0, False), (129, 4096, 1000, 0, True),
    (20000, 100, 1000, 0, True), (20000, 100, 1024, 0, False), (5, 12288, 4095, 0, False), (640, 4096, 0, 0, False)])
def test_which_products_need_a_workspace(M, N, K, ldx, need):
    """Arrays at 16 bytes go by another rule than others, and bring a workspace only where it is used."""
    kw = dict(M=M, N=N, K=K, ldx=ldx)
    size = kda.load().kda_linear_i8_workspace_size(M, N, K)
    assert (_linear(**kw, ws=None, size=0) == kda.KDA_ERR_WORKSPACE) == need
    assert _linear(**kw, ws=6 * A, size=size) != kda.KDA_ERR_WORKSPACE
    if need:
        assert size == (M + N) * (-(-K // 16) * 16) * 2
        assert _linear(**kw, ws=6 * A, size=size - 1) == kda.KDA_ERR_WORKSPACE
        assert _linear(**kw, ws=6 * A + 8, size=size) == kda.KDA_ERR_ALIGN


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M, K, N", [(65, 100, 9800), (96, 333, 12288), (5000, 77, 65), (512, 128, 12288), (384, 128, 12288),
                                     (70, 96, 10000)])
def test_either_side_of_the_rule(dtype, M, K, N):
    """Few rows of many channels, many rows of few; a second wave of tiles; with and without a workspace."""
    a = make(M, K, N, dtype, seed=13)
    want = plain(*a, "silu")
    check(kda.kda_linear_i8(*a, act="silu"), *want)
    ws = torch.full((kda.load().kda_linear_i8_workspace_size(M, N, K),), 255, dtype=torch.uint8, device="cuda")
    check(kda.kda_linear_i8(*a, act="silu", workspace=ws if len(ws) else None), *want)

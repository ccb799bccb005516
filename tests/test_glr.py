"""The gated linear recurrence, its gradient and its step against 64 bits, and its refusals.
Allowances: tests/glr64.py, and on top of them the output's own rounding."""
import ctypes

import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import glr64, plain64

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
DECAYS, SCALES = list(kda.DECAY_FROM), list(kda.INPUT_SCALES)
FORMS = [(d, s, g) for d in DECAYS for s in SCALES for g in (False, True)]


def make(T, D, dtype, decay, scale, gate, seed=0, device="cuda"):
    """Inputs of a layer: decays of a few to some thousand tokens."""
    g = torch.Generator().manual_seed(seed)
    to = lambda t, dt=dtype: t.to(dt).to(device)  # noqa: E731
    x = to(torch.randn(T, D, generator=g))
    form = dict(decay_from=decay, input_scale=scale,
                input_gate=to(torch.randn(T, D, generator=g)) if gate else None)
    if decay == "log":
        la = -torch.exp(torch.randn(T, D, generator=g) * 2 - 3)
        la = torch.where(torch.rand(T, D, generator=g) < 0.05, la.abs(), la)  # some above 0
    else:
        la = torch.randn(T, D, generator=g) * 2
        form["decay_scale"] = to(torch.exp(torch.randn(D, generator=g) * 2 - 3), F32)
        form["decay_bias"] = to(torch.randn(D, generator=g), F32)
    return x, to(la), form


def check(got, ref, off):
    """Within the allowance.  Below the smallest normal number the spacing of a type falls no
    further: rounding to it is then off by up to half of the smallest subnormal number, whatever the
    value.  Decays, gates and factors below 2^-126 act as 0 (the header says so): a state or a
    gradient of up to 16 in size is then off by 16 * 2^-126, once for each of at most four factors
    of a product, and what follows such a decay has forgotten what was before it."""
    e = plain64.excess(got, ref)
    info = torch.finfo(got.dtype)
    allowed = off * (1 + plain64.half_step(got.dtype)) + info.tiny * info.eps / 2 + 64 * 2.0 ** -126
    worst = (e - allowed).max() if e.numel() else torch.tensor(0.0)
    assert worst <= 0, f"{float(worst):.3e} over the allowed error"


def offsets(lens, device="cuda"):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)


def states(N, D, seed=9, device="cuda"):
    return torch.randn(N, D, generator=torch.Generator().manual_seed(seed)).to(device)


# ------------------------------------------------------------------ on the CPU
A = 0x10000
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="refusals use stand-in addresses: only where nothing can launch")


def _scan(opt=None, **kw):
    a = dict(x=A, la=2 * A, h0=None, cu=None, N=1, y=3 * A, h=4 * A, T=64, D=32, dtype=kda.KDA_BF16) | kw
    o = kda.kda_glr_options_init(**(opt or {}))
    return kda.load().kda_glr_scan(a["x"], a["la"], a["h0"], a["cu"], a["N"], a["y"], a["h"], a["T"],
                                   a["D"], a["dtype"], ctypes.byref(o), None)


def _back(opt=None, **kw):
    a = dict(dy=A, dh=None, x=2 * A, la=3 * A, cu=None, N=1, dx=4 * A, dla=5 * A, dg=None, dh0=None, dA=None,
             db=None, T=64, D=32, dtype=kda.KDA_BF16) | kw
    o = kda.kda_glr_options_init(**(dict(checkpoints=9 * A) | (opt or {})))
    return kda.load().kda_glr_scan_backward(
        a["dy"], a["dh"], a["x"], a["la"], a["cu"], a["N"], a["dx"], a["dla"], a["dg"], a["dh0"], a["dA"],
        a["db"], a["T"], a["D"], a["dtype"], ctypes.byref(o), None)


def _step(opt=None, **kw):
    a = dict(x=A, la=2 * A, h=3 * A, y=4 * A, N=2, L=1, D=32, dtype=kda.KDA_BF16) | kw
    o = kda.kda_glr_options_init(**(opt or {}))
    return kda.load().kda_glr_step(a["x"], a["la"], a["h"], a["y"], a["N"], a["L"], a["D"], a["dtype"],
                                   ctypes.byref(o), None)


BAD_OPTIONS = [
    (dict(decay_from=3), kda.KDA_ERR_ARG), (dict(decay_from=-1), kda.KDA_ERR_ARG),
    (dict(input_scale=3), kda.KDA_ERR_ARG), (dict(input_scale=-1), kda.KDA_ERR_ARG),
    (dict(ldx=31), kda.KDA_ERR_SHAPE), (dict(ldla=-32), kda.KDA_ERR_SHAPE), (dict(ldg=8), kda.KDA_ERR_SHAPE),
    (dict(input_gate=A + 1), kda.KDA_ERR_ALIGN), (dict(decay_scale=A + 2), kda.KDA_ERR_ALIGN),
    (dict(decay_bias=A + 1), kda.KDA_ERR_ALIGN), (dict(checkpoints=A + 2), kda.KDA_ERR_ALIGN),
    (dict(slots=A + 2, n_slots=4), kda.KDA_ERR_ALIGN), (dict(slots=A, n_slots=0), kda.KDA_ERR_SHAPE),
    (dict(max_seqlen=-1), kda.KDA_ERR_SHAPE), (dict(max_seqlen=65), kda.KDA_ERR_SHAPE)]
BAD_SIZES = [
    (dict(D=0), kda.KDA_ERR_SHAPE), (dict(N=0), kda.KDA_ERR_SHAPE), (dict(D=2 ** 31 - 256), kda.KDA_ERR_SHAPE),
    (dict(dtype=2), kda.KDA_ERR_DTYPE), (dict(x=None), kda.KDA_ERR_ARG), (dict(la=None), kda.KDA_ERR_ARG),
    (dict(x=A + 1), kda.KDA_ERR_ALIGN), (dict(la=A + 1), kda.KDA_ERR_ALIGN),
    (dict(D=2 ** 30, N=2 ** 10, T=2 ** 10), kda.KDA_ERR_SHAPE)]


@no_gpu
@pytest.mark.parametrize("opt, status", BAD_OPTIONS)
def test_options_refused(opt, status):
    assert _scan(opt) == status
    if "slots" not in opt and "checkpoints" not in opt and "max_seqlen" not in opt:
        assert _back(opt) == status and _step(opt) == status


@no_gpu
@pytest.mark.parametrize("kw, status", BAD_SIZES)
def test_sizes_refused(kw, status):
    assert _scan(**kw) == status
    assert _back(**kw) == status
    kw = {k: v for k, v in kw.items() if k != "T"}
    assert _step(**kw) == status


@no_gpu
def test_scan_refuses():
    assert _scan(T=-1) == kda.KDA_ERR_SHAPE
    assert _scan(T=2 ** 31 - 1024) == kda.KDA_ERR_SHAPE
    assert _scan(T=65, N=2) == kda.KDA_ERR_SHAPE
    assert _scan(y=None) == kda.KDA_ERR_ARG and _scan(h=None) == kda.KDA_ERR_ARG
    assert _scan(y=A + 1) == kda.KDA_ERR_ALIGN and _scan(h=A + 2) == kda.KDA_ERR_ALIGN
    assert _scan(h0=A + 2) == kda.KDA_ERR_ALIGN and _scan(cu=A + 2) == kda.KDA_ERR_ALIGN
    for out in ("y", "h"):
        for at in (A, 2 * A):
            assert _scan(**{out: at}) == kda.KDA_ERR_ARG
    assert _scan(y=5 * A, h0=5 * A) == kda.KDA_ERR_ARG and _scan(y=5 * A, h=5 * A) == kda.KDA_ERR_ARG
    assert _scan(dict(input_gate=3 * A)) == kda.KDA_ERR_ARG
    for at in (A, 2 * A, 3 * A, 4 * A):
        assert _scan(dict(checkpoints=at)) == kda.KDA_ERR_ARG


@no_gpu
def test_step_refuses():
    assert _step(L=0) == kda.KDA_ERR_SHAPE and _step(N=2 ** 20, L=2 ** 12) == kda.KDA_ERR_SHAPE
    assert _step(h=None) == kda.KDA_ERR_ARG and _step(y=None) == kda.KDA_ERR_ARG
    assert _step(h=A + 1) == kda.KDA_ERR_ALIGN and _step(y=A + 1) == kda.KDA_ERR_ALIGN
    assert _step(dict(checkpoints=9 * A)) == kda.KDA_ERR_UNSUPPORTED
    for at in (A, 2 * A, 3 * A):
        assert _step(y=at) == kda.KDA_ERR_ARG
    for at in (A, 2 * A):
        assert _step(h=at) == kda.KDA_ERR_ARG


@no_gpu
def test_backward_refuses():
    logits = dict(decay_from=1, workspace=11 * A, workspace_bytes=1 << 30)
    assert _back(dict(checkpoints=None)) == kda.KDA_ERR_ARG
    assert _back(dx=None) == kda.KDA_ERR_ARG and _back(dla=None) == kda.KDA_ERR_ARG
    assert _back(dg=6 * A) == kda.KDA_ERR_ARG                      # no gate
    assert _back(dA=6 * A) == kda.KDA_ERR_ARG                      # no parameters
    assert _back(dict(slots=A, n_slots=3)) == kda.KDA_ERR_UNSUPPORTED
    assert _back(dict(decay_from=1), dA=6 * A) == kda.KDA_ERR_WORKSPACE
    assert _back(logits | dict(workspace_bytes=8), db=6 * A) == kda.KDA_ERR_WORKSPACE
    assert _back(logits | dict(workspace=11 * A + 8), db=6 * A) == kda.KDA_ERR_ALIGN
    for name in ("dy", "dx", "dla"):
        assert _back(**{name: 7 * A + 1}) == kda.KDA_ERR_ALIGN
    for name in ("dh", "dh0", "cu"):
        assert _back(**{name: 7 * A + 2}) == kda.KDA_ERR_ALIGN
    assert _back(logits, dA=7 * A + 2) == kda.KDA_ERR_ALIGN
    for at in (A, 2 * A, 3 * A, 9 * A):
        assert _back(dx=at) == kda.KDA_ERR_ARG and _back(dla=at) == kda.KDA_ERR_ARG
        assert _back(dh0=at) == kda.KDA_ERR_ARG
        assert _back(logits, db=at) == kda.KDA_ERR_ARG
    assert _back(dx=5 * A) == kda.KDA_ERR_ARG                      # two outputs
    assert _back(logits, dA=6 * A, db=6 * A) == kda.KDA_ERR_ARG
    assert _back(logits | dict(workspace=4 * A), dA=6 * A) == kda.KDA_ERR_ARG


def test_binding_refuses():
    x, la, form = make(4, 8, F32, "log", "none", False, device="cpu")
    with pytest.raises(ValueError):
        kda.kda_glr_scan(x, la)
    with pytest.raises(ValueError):
        kda._tokens(x, "x", (4, 9), F32)
    with pytest.raises(TypeError):
        kda._tokens(x, "x", (4, 8), BF16)
    with pytest.raises(ValueError):
        kda._tokens(x.T, "x", (8, 4), F32)
    with pytest.raises(ValueError):
        kda._tokens(x[:1].expand(4, 8), "x", (4, 8), F32)
    assert kda._tokens(torch.zeros(5, 20)[:, 4:12], "x", (5, 8), F32) == 20
    assert kda._tokens(torch.zeros(3, 2, 20)[..., 4:12], "x", (3, 2, 8), F32) == 20
    with pytest.raises(ValueError):
        kda._tokens(torch.zeros(3, 4, 8)[:, :2], "x", (3, 2, 8), F32)


@pytest.mark.parametrize("decay, scale, gate", FORMS)
def test_plain_gradient(decay, scale, gate):
    """The 64-bit formulas against differentiation of the definition."""
    lens = [3, 0, 5, 1]
    T, D = sum(lens), 3
    x, la, form = make(T, D, torch.float64, decay, scale, gate, device="cpu")
    h0, dh, dy = (torch.randn(*s, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
                  for s in ((4, D), (4, D), (T, D)))
    leaves = {"dx": x, "dla": la, "dh0": h0}
    if gate:
        leaves["dgate"] = form["input_gate"]
    if decay != "log":
        form["decay_scale"], form["decay_bias"] = form["decay_scale"].double(), form["decay_bias"].double()
        leaves |= {"dA": form["decay_scale"], "db": form["decay_bias"]}
    ref = glr64.backward(glr64.Form(x, la, **form), h0, lens, dy, dh)

    def value():
        y, end, *_ = glr64.scan(glr64.Form(x, la, **form), h0, lens)
        return float((y * dy).sum() + (end * dh).sum())

    for name, leaf in leaves.items():
        flat, grad = leaf.view(-1), ref[name][0].reshape(-1)
        for i in range(0, flat.numel(), 2):
            if name == "dla" and decay == "log" and abs(float(flat[i])) < 1e-4:
                continue  # the border at 0
            keep, step = float(flat[i]), 1e-6 * max(1e-2, min(1.0, abs(float(flat[i]))))
            flat[i] = keep + step
            up = value()
            flat[i] = keep - step
            down = value()
            flat[i] = keep
            # a difference of two values of size ~10: 10 * 2^-52 / step; its curvature step^2
            assert abs((up - down) / (2 * step) - float(grad[i])) <= 1e-4 * max(1.0, abs(float(grad[i])))


# ------------------------------------------------------------------ on the GPU
@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decay, scale, gate", FORMS)
def test_forms(dtype, decay, scale, gate):
    lens = [70, 0, 1, 200]
    T, D = sum(lens), 66
    x, la, form = make(T, D, dtype, decay, scale, gate)
    h0, dh, dy = states(4, D), states(4, D, 10), states(T, D, 11).to(dtype)
    f = glr64.Form(x, la, **form)
    y, h, saved = kda.kda_glr_scan(x, la, h0, offsets(lens), checkpoints=True, **form)
    ref = glr64.scan(f, h0, lens)
    check(y, ref[0], ref[2])
    check(h, ref[1], ref[3])
    got = kda.kda_glr_scan_backward(dy, dh, x, la, saved, offsets(lens), **form)
    want = glr64.backward(f, h0, lens, dy, dh)
    for name, t in zip(("dx", "dla", "dgate", "dh0", "dA", "db"), got):
        if t is not None:
            check(t, *want[name])
    assert (got[2] is None) == (not gate) and (got[4] is None) == (decay == "log")
    assert kda.kda_get_last_error() == kda.KDA_OK


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, D", [(1, 1), (1, 64), (2, 33), (7, 2), (8, 65), (9, 128), (16, 31), (17, 34), (63, 3),
                                  (64, 64), (65, 70), (127, 130), (128, 1), (129, 62), (300, 200), (511, 8),
                                  (513, 6), (1025, 4), (1500, 5)])
def test_lengths(dtype, T, D):
    x, la, form = make(T, D, dtype, "sigmoid", "normalized", True, seed=T)
    dy = states(T, D, 11).to(dtype)
    f = glr64.Form(x, la, **form)
    ref = glr64.scan(f, None, [T])
    y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True, **form)
    check(y, ref[0], ref[2])
    check(h, ref[1], ref[3])
    for t in range(0, T, 64):
        check(saved[t // 64], ref[4][0][t], ref[4][1][t])
    want = glr64.backward(f, None, [T], dy, None)
    for name, t in zip(("dx", "dla", "dgate", "dh0", "dA", "db"),
                       kda.kda_glr_scan_backward(dy, None, x, la, saved, **form)):
        check(t, *want[name])
    # the same sequence by its last state alone
    want = glr64.backward(f, None, [T], None, h)
    for name, t in zip(("dx", "dla", "dgate", "dh0", "dA", "db"),
                       kda.kda_glr_scan_backward(None, h, x, la, saved, **form)):
        check(t, *want[name])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N, lens, D", [(3, None, 40), (40, None, 66), (5, [0, 0, 0, 0, 0], 10),
                                        (36, [i % 7 for i in range(36)], 20), (3, [500, 3, 129], 1200),
                                        (33, [17] * 33, 2000)])
def test_sequences(dtype, N, lens, D):
    """Equal lengths without offsets; empty, short and many sequences, on one CTA and on clusters."""
    cu = None if lens is None else offsets(lens)
    lens = lens or [90] * N
    T = sum(lens)
    x, la, form = make(T, D, dtype, "softplus", "complement", False, seed=3)
    h0, dy, dh = states(N, D), states(T, D, 5).to(dtype), states(N, D, 6)
    f = glr64.Form(x, la, **form)
    ref = glr64.scan(f, h0, lens)
    want = glr64.backward(f, h0, lens, dy, dh)
    for hint in (0, max(lens)):
        y, h, saved = kda.kda_glr_scan(x, la, h0, cu, N, checkpoints=True, max_seqlen=hint, **form)
        check(y, ref[0], ref[2])
        check(h, ref[1], ref[3])
        got = kda.kda_glr_scan_backward(dy, dh, x, la, saved, cu, N, max_seqlen=hint, **form)
        for name, t in zip(("dx", "dla", "dgate", "dh0", "dA", "db"), got):
            if t is not None:
                check(t, *want[name])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("L", [None, 1, 3, 20])
def test_step(dtype, L):
    """Tokens of five sequences, states in a pool whose other rows stay; one left out."""
    N, D = 5, 130
    T = N * (L or 1)
    x, la, form = make(T, D, dtype, "sigmoid", "normalized", True, seed=1)
    pool = states(8, D)
    slots = torch.tensor([3, 7, -1, 0, 2], dtype=torch.int32, device="cuda")
    shape = (N, D) if L is None else (N, L, D)
    f = glr64.Form(x, la, **form)
    form["input_gate"] = form["input_gate"].view(shape)
    first = pool[slots.long().clamp(min=0)].clone()
    y, h, off_y, off_h, _ = glr64.scan(f, first, [L or 1] * N)
    was = pool.clone()
    out = torch.full(shape, 7.0, dtype=dtype, device="cuda")
    assert kda.kda_glr_step(x.view(shape), la.view(shape), pool, out, slots=slots, **form) is out
    for n in range(N):
        rows = slice(n * (L or 1), (n + 1) * (L or 1))
        if n == 2:
            assert (out[n] == 7).all()
            continue
        check(out[n].view(-1, D), y[rows], off_y[rows])
        check(pool[slots[n].item()], h[n], off_h[n])
        was[slots[n].item()] = pool[slots[n].item()]
    assert torch.equal(was, pool)
    # without a pool, and into a new output
    h1 = first.clone()
    y1 = kda.kda_glr_step(x.view(shape), la.view(shape), h1, **form)
    check(y1.view(-1, D), y, off_y)
    check(h1, h, off_h)


@gpu
@pytest.mark.parametrize("T", [10, 200])
def test_pool_and_bad_slots(T):
    D = 100
    x, la, form = make(3 * T, D, BF16, "log", "none", False)
    pool = states(6, D)
    was = pool.clone()
    slots = torch.tensor([4, -3, 1], dtype=torch.int32, device="cuda")
    y = torch.full((3 * T, D), 5.0, dtype=BF16, device="cuda")
    kda.kda_glr_scan(x, la, pool, None, 3, y, pool, slots=slots, **form)
    ref = glr64.scan(glr64.Form(x, la, **form), was[[4, 0, 1]], [T] * 3)
    assert (y[T:2 * T] == 5).all()
    for n in (0, 2):
        check(y[n * T:(n + 1) * T], ref[0][n * T:(n + 1) * T], ref[2][n * T:(n + 1) * T])
        check(pool[slots[n].item()], ref[1][n], ref[3][n])
    for i in (0, 2, 3, 5):
        assert torch.equal(pool[i], was[i])
    assert kda.kda_get_last_error() == kda.KDA_OK
    for bad in ([4, 6, 1], [4, 1, 4]):  # out of the pool; taken twice
        pool.copy_(was)
        y.fill_(5)
        kda.kda_glr_scan(x, la, pool, None, 3, y, pool, slots=torch.tensor(bad, dtype=torch.int32, device="cuda"),
                         **form)
        assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE
        left_out = 1 if bad[1] == 6 else 2
        assert (y[left_out * T:(left_out + 1) * T] == 5).all()
        check(y[:T], ref[0][:T], ref[2][:T])


@gpu
@pytest.mark.parametrize("long", [False, True])
def test_bad_offsets_and_rows_behind_the_last_sequence(long):
    T, D = (400 if long else 20), 64
    x, la, form = make(T, D, BF16, "sigmoid", "none", False)
    cu = torch.tensor([0, T // 2, T - 7], dtype=torch.int32, device="cuda")
    y = torch.full((T, D), 5.0, dtype=BF16, device="cuda")
    _, h, saved = kda.kda_glr_scan(x, la, None, cu, y=y, checkpoints=True, **form)
    ref = glr64.scan(glr64.Form(x, la, **form), None, [T // 2, T - 7 - T // 2])
    check(y[:T - 7], ref[0][:T - 7], ref[2][:T - 7])
    assert (y[T - 7:] == 5).all()
    dy = torch.full((T, D), float("nan"), dtype=BF16, device="cuda")
    dy[:T - 7] = 1
    got = kda.kda_glr_scan_backward(dy, None, x, la, saved, cu, **form)
    assert all(torch.isfinite(t).all() for t in (got[0][:T - 7], got[1][:T - 7], *got[3:]))
    assert kda.kda_get_last_error() == kda.KDA_OK
    for bad in ([0, T + 1, T], [0, 8, 4], [-1, 8, 16]):
        kda.kda_glr_scan(x, la, None, torch.tensor(bad, dtype=torch.int32, device="cuda"), **form)
        assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE
        got = kda.kda_glr_scan_backward(dy, None, x, la, saved, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                                        **form)
        assert kda.kda_get_last_error() == kda.KDA_ERR_SHAPE


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [9, 150])
def test_slices_of_one_projection(dtype, T):
    """x, log_alpha and the gate as slices, at odd and even offsets, with NaN between them."""
    D = 50
    for off, width in ((0, 3 * D), (1, 3 * D + 5), (2, 3 * D + 6)):
        whole = torch.full((T, off + width), float("nan"))
        whole[:, off:off + 3 * D] = torch.randn(T, 3 * D, generator=torch.Generator().manual_seed(2))
        whole = whole.to(dtype).cuda()
        x, la, gate = (whole[:, off + i * D:off + (i + 1) * D] for i in range(3))
        form = dict(decay_from="sigmoid", input_scale="normalized", input_gate=gate)
        f = glr64.Form(x, la, **form)
        y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True, **form)
        ref = glr64.scan(f, None, [T])
        check(y, ref[0], ref[2])
        check(h, ref[1], ref[3])
        dy = states(T, D).to(dtype)
        want = glr64.backward(f, None, [T], dy, None)
        for name, t in zip(("dx", "dla", "dgate", "dh0", "dA", "db"),
                           kda.kda_glr_scan_backward(dy, None, x, la, saved, **form)):
            check(t, *want[name])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [12, 1000])
@pytest.mark.parametrize("scale", SCALES)
def test_border_values(dtype, T, scale):
    """Decays of exactly 0 and 1, none in between; and logits at both ends."""
    D = 64
    x, la, form = make(T, D, dtype, "log", scale, False, seed=6)
    g = torch.Generator().manual_seed(7)
    kind = torch.randint(0, 4, (T, D), generator=g).cuda()
    la[kind == 0] = float("-inf")
    la[kind == 1] = 0
    la[kind == 2] = 3.0
    la[kind == 3] = -200
    f = glr64.Form(x, la, **form)
    ref = glr64.scan(f, None, [T])
    y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True, **form)
    check(y, ref[0], ref[2])
    dy = states(T, D).to(dtype)
    got = kda.kda_glr_scan_backward(dy, None, x, la, saved, **form)
    want = glr64.backward(f, None, [T], dy, None)
    check(got[0], *want["dx"])
    check(got[3], *want["dh0"])
    assert torch.isfinite(got[1]).all()
    for decay in ("softplus", "sigmoid"):
        la = torch.where(kind == 0, -1e30, torch.where(kind == 1, float("-inf"), torch.where(kind == 2, 1e30, 0.0)))
        la = la.to(dtype)
        form = dict(decay_from=decay, input_scale=scale)
        y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True, **form)
        ref = glr64.scan(glr64.Form(x, la, **form), None, [T])
        check(y, ref[0], ref[2])
        got = kda.kda_glr_scan_backward(dy, None, x, la, saved, **form)
        assert all(torch.isfinite(t).all() for t in got if t is not None)


@gpu
@pytest.mark.parametrize("T", [15, 700])
def test_nan_stays_behind_itself(T):
    D, at = 40, T // 2
    x, la, form = make(2 * T, D, BF16, "sigmoid", "normalized", True)
    y0, h0, saved0 = kda.kda_glr_scan(x, la, None, None, 2, checkpoints=True, **form)
    dy = states(2 * T, D).to(BF16)
    g0 = kda.kda_glr_scan_backward(dy, None, x, la, saved0, None, 2, **form)
    for what, value in (("x", float("nan")), ("x", float("inf")), ("la", float("nan")), ("gate", float("nan"))):
        bad = {"x": x.clone(), "la": la.clone(), "gate": form["input_gate"].clone()}
        bad[what][at, 5] = value
        f2 = form | dict(input_gate=bad["gate"])
        y, h, saved = kda.kda_glr_scan(bad["x"], bad["la"], None, None, 2, checkpoints=True, **f2)
        assert not torch.isfinite(y[at:T, 5]).any() and not torch.isfinite(h[0, 5])
        assert torch.equal(y[:at], y0[:at]) and torch.equal(y[T:], y0[T:]) and torch.equal(h[1], h0[1])
        others = [c for c in range(D) if c != 5]
        assert torch.equal(y[:, others], y0[:, others])
        g = kda.kda_glr_scan_backward(dy, None, bad["x"], bad["la"], saved, None, 2, **f2)
        for a, b in zip(g[:3], g0[:3]):
            assert torch.equal(a[T:], b[T:]) and torch.equal(a[:, others], b[:, others])
        assert torch.equal(g[3][1], g0[3][1]) and torch.equal(g[4][others], g0[4][others])


@gpu
def test_long_memories_are_exact():
    """Decays of 1 - 1e-5 to 1 - 1e-2 over 20,000 tokens: states and the parameters' gradients, sums
    of terms that nearly cancel, in the 2-norm.  Decays rounded to fp32 are off by up to 2^-25, a
    share of 2^-25 / (1 - a) of the state: 5e-6 and more here, and ten times that in the gradients.
    Held as a - 1, what is left are roundings of h, sqrt(1 / (1 - a)) of them of 2^-25 each: 1e-5 at
    the very worst channel's 300 roundings, 1e-6 in the norm over channels."""
    T, D = 20000, 48
    g = torch.Generator().manual_seed(5)
    x, la, dy = (torch.randn(T, D, generator=g).cuda() for _ in range(3))
    scale = torch.exp(-torch.linspace(4.6, 11.5, D)).cuda() * 2
    form = dict(decay_from="sigmoid", decay_scale=scale, input_scale="normalized")
    leaves = [t.double().requires_grad_() for t in (x, la, scale)]
    lg = -leaves[2] * torch.sigmoid(leaves[1])
    a, u, h, rows = torch.exp(lg), torch.sqrt(-torch.expm1(2 * lg)) * leaves[0], 0.0, []
    for t in range(T):
        h = a[t] * h + u[t]
        rows.append(h)
    ref = torch.stack(rows)
    want = torch.autograd.grad((ref * dy.double()).sum(), leaves)
    y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True, **form)
    got = kda.kda_glr_scan_backward(dy, None, x, la, saved, **form)
    ref = ref.detach()
    rel = lambda u, v: float((u.double() - v).norm() / v.norm())  # noqa: E731
    assert rel(y, ref) <= 1e-6 and rel(h[0], ref[-1]) <= 1e-6
    assert rel(got[0], want[0]) <= 1e-6 and rel(got[1], want[1]) <= 2e-6 and rel(got[4], want[2]) <= 5e-6


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T, D", [(5, 300), (900, 70), (300, 9000)])
def test_repeats_to_the_bit_on_streams_and_in_graphs(dtype, T, D):
    x, la, form = make(T, D, dtype, "softplus", "complement", True)
    dy = states(T, D).to(dtype)

    def run():
        y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True, **form)
        return [y, h, *kda.kda_glr_scan_backward(dy, h, x, la, saved, **form)]

    first = run()
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for st in streams:
        with torch.cuda.stream(st):
            outs += [run() for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(first, o))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run()
    x2, la2, form2 = make(T, D, dtype, "softplus", "complement", True, seed=8)
    x.copy_(x2)
    la.copy_(la2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(o, run()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = kda.kda_glr_scan(x, la, stream=side, **form)
    side.synchronize()
    assert torch.equal(y, o[0])


@gpu
@pytest.mark.parametrize("chunks", [[1000], [999, 1], [300, 64, 636], [10] * 100])
def test_a_sequence_in_parts(chunks):
    """A prompt in parts, the state handed on in place, gives what one call gives (up to roundings)."""
    T, D = 1000, 90
    x, la, form = make(T, D, F32, "log", "none", False)
    ref = glr64.scan(glr64.Form(x, la, **form), None, [T])
    h, at = torch.zeros(1, D, device="cuda"), 0
    for n in chunks:
        y, _ = kda.kda_glr_scan(x[at:at + n], la[at:at + n], h, h_T=h, **form)
        check(y, ref[0][at:at + n], 2 * ref[2][at:at + n])
        at += n


@gpu
def test_tokens_past_two_to_the_31():
    """Arrays of more than 2^31 elements: the last tokens, forward and backward, at offsets past 32 bits."""
    T, D = 530_000, 4096 + 64
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    la = torch.full((T, D), -1.0, dtype=BF16, device="cuda")
    tail, _, _ = make(300, D, BF16, "log", "none", False)
    x[-300:] = tail
    y, h, saved = kda.kda_glr_scan(x, la, checkpoints=True)
    cols = slice(0, None, 97)
    f = glr64.Form(tail[:, cols], la[-300:, cols])
    ref = glr64.scan(f, None, [300])
    check(y[-300:, cols], ref[0], ref[2])
    assert (y[:-300:1009] == 0).all()
    got = kda.kda_glr_scan_backward(y, None, x, la, saved)
    want = glr64.backward(f, None, [300], y[-300:, cols], None)
    check(got[0][-300:, cols], *want["dx"])
    check(got[1][-300:, cols], *want["dla"])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 50])
def test_neighbours_of_a_sequence_do_not_reach_it(dtype, D):
    """NaN in the rows before and behind a sequence that ends inside a tile, and behind the last one."""
    T = 150
    x, la, form = make(3 * T + 9, D, dtype, "sigmoid", "normalized", True)
    cu = torch.tensor([0, T, 2 * T, 3 * T], dtype=torch.int32, device="cuda")
    dy = states(3 * T + 9, D).to(dtype)

    def run():
        y, h, saved = kda.kda_glr_scan(x, la, None, cu, checkpoints=True, **form)
        return y, h, kda.kda_glr_scan_backward(dy, None, x, la, saved, cu, **form)

    y0, h0, g0 = run()
    for t in (x, la, form["input_gate"], dy):
        t[:T] = float("nan")
        t[2 * T:] = float("nan")
    y, h, g = run()
    middle = slice(T, 2 * T)
    assert torch.equal(y[middle], y0[middle]) and torch.equal(h[1], h0[1])
    assert all(torch.equal(a[middle], b[middle]) for a, b in zip(g[:3], g0[:3])) and torch.equal(g[3][1], g0[3][1])


@gpu
def test_many_sequences_and_slots():
    """More sequences than a warp has lanes, of no, one and more tokens, states in a pool."""
    lens = [(7 * i) % 5 for i in range(100)] + [90, 0, 300]
    N, T, D = len(lens), sum(lens), 72
    x, la, form = make(T, D, BF16, "softplus", "none", True, seed=2)
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(N + 5, generator=g)[:N].to(torch.int32).cuda()
    pool = states(N + 5, D)
    was = pool.clone()
    first = was[slots.long()]
    y, _ = kda.kda_glr_scan(x, la, pool, offsets(lens), h_T=pool, slots=slots, max_seqlen=300, **form)
    ref = glr64.scan(glr64.Form(x, la, **form), first, lens)
    check(y, ref[0], ref[2])
    check(pool[slots.long()], ref[1], ref[3])
    rest = [i for i in range(N + 5) if i not in slots.tolist()]
    assert torch.equal(pool[rest], was[rest])


@gpu
@pytest.mark.parametrize("N, L", [(300, 5), (300, 70), (40, 200)])
def test_by_token_and_in_tiles_agree(N, L):
    """Many sequences are walked token by token; one of them alone is taken in tiles where it is long."""
    D = 4096
    x, la, form = make(N * L, D, BF16, "sigmoid", "normalized", False, seed=4)
    y, h, saved = kda.kda_glr_scan(x, la, None, None, N, checkpoints=True, **form)
    cols = slice(0, None, 61)
    for n in (0, N - 1):
        rows = slice(n * L, (n + 1) * L)
        part = {k: v[cols] if k.startswith("decay_") and torch.is_tensor(v) else v for k, v in form.items()}
        ref = glr64.scan(glr64.Form(x[rows, cols], la[rows, cols], **part), None, [L])
        check(y[rows, cols], ref[0], ref[2])
        check(h[n:n + 1, cols], ref[1], ref[3])
    dy = states(N * L, D).to(BF16)
    got = kda.kda_glr_scan_backward(dy, None, x, la, saved, None, N, **form)
    want = glr64.backward(glr64.Form(x[rows, cols], la[rows, cols], **part), None, [L], dy[rows, cols], None)
    check(got[0][rows, cols], *want["dx"])
    check(got[1][rows, cols], *want["dla"])


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_tokens(dtype):
    """Sequences without tokens hand their states, and the gradients of those, on."""
    D = 24
    x, la, form = make(0, D, dtype, "sigmoid", "none", True)
    h0 = states(3, D)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    for offs in (cu, None):
        y, h, saved = kda.kda_glr_scan(x, la, h0, offs, 3, checkpoints=True, **form)
        assert y.shape == (0, D) and torch.equal(h, h0)
        got = kda.kda_glr_scan_backward(None, h, x, la, saved, offs, 3, **form)
        assert torch.equal(got[3], h) and (got[4] == 0).all() and (got[5] == 0).all()
    pool = states(5, D, 3)
    was = pool.clone()
    kda.kda_glr_scan(x, la, pool, cu, h_T=pool, slots=torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda"), **form)
    assert torch.equal(pool, was) and kda.kda_get_last_error() == kda.KDA_OK


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [8, 1000, 1032, 4096])
@pytest.mark.parametrize("off", [0, 1, 2])
def test_states_at_any_place(dtype, D, off):
    """States, parameters and saved states at 16 bytes and not, in a step and in a few tokens each."""
    N, L = 40, 3
    x, la, form = make(N * L, D, dtype, "softplus", "normalized", True, seed=5)

    def at(t):
        flat = torch.zeros(t.numel() + off, device="cuda")
        flat[off:] = t.reshape(-1)
        return flat[off:].view(t.shape)

    form["decay_scale"], form["decay_bias"] = at(form["decay_scale"]), at(form["decay_bias"])
    h = at(states(N, D))
    ref = glr64.scan(glr64.Form(x, la, **form), h, [L] * N)
    saved = at(torch.zeros(N * L // 64 + N, D))
    y, end, _ = kda.kda_glr_scan(x, la, h, None, N, checkpoints=saved, **form)
    check(y, ref[0], ref[2])
    check(end, ref[1], ref[3])
    rows = [n * L // 64 + n for n in range(N)]
    assert torch.equal(saved[rows], h)
    form["input_gate"] = form["input_gate"].view(N, L, D)
    y = kda.kda_glr_step(x.view(N, L, D), la.view(N, L, D), h, **form)
    check(y.view(-1, D), ref[0], ref[2])
    check(h, ref[1], ref[3])


@no_gpu
@pytest.mark.parametrize("out", ["y", "h", "checkpoints"])
@pytest.mark.parametrize("at", ["x", "la", "cu", "input_gate", "decay_scale", "decay_bias", "slots"])
def test_an_output_at_an_input_is_refused(out, at):
    """Other CTAs still read the parameters, offsets and slots when one writes its outputs."""
    if at in ("x", "la", "cu"):
        kw, opt = {at: 8 * A}, {}
    else:
        kw, opt = {}, {at: 8 * A} | (dict(n_slots=4) if at == "slots" else {})
    opt["decay_from"] = 1
    where = opt if out == "checkpoints" else kw
    where[out] = 8 * A
    assert _scan(opt, **kw) == kda.KDA_ERR_ARG
    if at != "cu" and out != "checkpoints":
        assert _step(opt, **kw) == kda.KDA_ERR_ARG


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [15, 700, 3000])
def test_what_nan_spoils_of_the_gradient(dtype, T):
    """The table in the header, for a NaN in each input; everything else is the same to the bit."""
    D, at, ch = 72, T // 2, 5
    x, la, form = make(2 * T, D, dtype, "sigmoid", "normalized", True)
    dy, dh = states(2 * T, D).to(dtype), states(2, D, 3)

    def run(x, la, gate, dy, dh):
        f = form | dict(input_gate=gate)
        *_, saved = kda.kda_glr_scan(x, la, None, None, 2, checkpoints=True, **f)
        return kda.kda_glr_scan_backward(dy, dh, x, la, saved, None, 2, **f)

    inputs = dict(x=x, la=la, gate=form["input_gate"], dy=dy, dh=dh)
    clean = run(*inputs.values())
    upto, behind, here, every, none = slice(0, at + 1), slice(at, T), slice(at, at + 1), slice(0, T), slice(0, 0)
    #               dx     dla     dgate  dh0
    spoiled = dict(x=(none, behind, here, False), la=(upto, every, upto, True), gate=(here, behind, here, False),
                   dy=(upto, upto, upto, True), dh=(every, every, every, True))
    for name, (*rows, first) in spoiled.items():
        bad = {k: v.clone() for k, v in inputs.items()}
        bad[name][0 if name == "dh" else at, ch] = float("nan")
        got = run(*bad.values())
        for g, c, r in zip(got[:3], clean[:3], rows):
            nan = torch.zeros(2 * T, D, dtype=torch.bool, device="cuda")
            nan[r, ch] = True
            assert torch.equal(g.isnan(), nan) and torch.equal(g[~nan], c[~nan])
        nan = torch.zeros(2, D, dtype=torch.bool, device="cuda")
        nan[0, ch] = first
        assert torch.equal(got[3].isnan(), nan) and torch.equal(got[3][~nan], clean[3][~nan])
        for g, c in zip(got[4:], clean[4:]):
            nan = torch.arange(D, device="cuda") == ch
            assert torch.equal(g.isnan(), nan) and torch.equal(g[~nan], c[~nan])

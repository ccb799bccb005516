"""Sizes next to 2^31, where an index, or a size on its way to the library, no longer fits in 32
bits.  Arrays of such calls take some 10 to 45 GB; each test gives them back."""
import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda

gpu = pytest.mark.gpu
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="calls on stand-in tensors of the CPU")
BF16, F32 = torch.bfloat16, torch.float32
LARGEST = 2 ** 31 - 257  # the largest width that the library takes


@pytest.fixture(autouse=True)
def give_back():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def everywhere(t, value):
    """Whether all of t is `value`, without a copy of its size."""
    flat = t.view(-1)
    return all(bool((flat[i:i + 2 ** 28] == value).all()) for i in range(0, flat.numel(), 2 ** 28))


MANY = 2 ** 32 + 5  # of which 32 bits are 5


def _too_many(x):
    """Calls with MANY rows, on x [MANY, 1], or x [MANY, 0] for the products."""
    one, none = x[:1], x[:, :0]
    i8 = none.to(torch.int8)
    yield lambda: kda.kda_linear(none, none[:3])
    yield lambda: kda.kda_linear(one[:, :0], none)
    yield lambda: kda.kda_linear_i8(i8, None, i8[:3], None)
    yield lambda: kda.kda_linear_i8(i8[:3], None, i8, None)
    yield lambda: kda.kda_rmsnorm(x)
    yield lambda: kda.kda_rmsnorm(x.view(1, MANY))
    yield lambda: kda.kda_rmsnorm_i8(x)
    yield lambda: kda.kda_quantize_i8(x)
    yield lambda: kda.kda_glr_scan(x, x)
    yield lambda: kda.kda_glr_scan(one, one, N=MANY)
    yield lambda: kda.kda_glr_scan(one, one, max_seqlen=MANY)
    yield lambda: kda.kda_glr_step(x, x, x)
    yield lambda: kda.kda_glr_step(x.view(1, MANY, 1), x.view(1, MANY, 1), x)
    yield lambda: kda.kda_glr_scan_backward(x, None, x, x, x)
    yield lambda: kda.kda_glr_scan_backward(None, None, one, one, one, N=MANY)


def test_sizes_beyond_32_bits_do_not_fit():
    kda._sizes("call", 2 ** 31 - 1, 0)
    with pytest.raises(kda.KdaError) as e:
        kda._sizes("call", 1, 2 ** 31)
    assert e.value.status == kda.KDA_ERR_SHAPE


@no_gpu
def test_sizes_beyond_32_bits_are_refused_on_the_host(monkeypatch):
    """Before anything of their size is allocated: stand-ins without memory, the device not asked for."""
    monkeypatch.setattr(kda, "_one_device", lambda *a: 0)
    for call in _too_many(torch.empty(MANY, 1, dtype=BF16, device="meta")):
        with pytest.raises(kda.KdaError) as e:
            call()
        assert e.value.status == kda.KDA_ERR_SHAPE


@gpu
def test_sizes_beyond_32_bits_are_refused():
    for call in _too_many(torch.empty(MANY, 1, dtype=BF16, device="cuda")):
        with pytest.raises(kda.KdaError) as e:
            call()
        assert e.value.status == kda.KDA_ERR_SHAPE


@gpu
def test_a_pool_of_more_rows_than_32_bits():
    pool = torch.zeros(MANY, 1, device="cuda")
    slots = torch.tensor([7], dtype=torch.int32, device="cuda")
    x = torch.full((1, 1), 3.0, device="cuda")
    y, _ = kda.kda_glr_scan(x, x, pool, h_T=pool, slots=slots)
    assert y[0, 0] == 3 and pool[7, 0] == 3
    y = kda.kda_glr_step(x, x, pool, slots=slots)
    assert y[0, 0] == 6 and pool[7, 0] == 6 and kda.kda_get_last_error() == kda.KDA_OK


@gpu
def test_recurrence_of_the_widest_channels():
    """Two sequences of one token, as many channels as 16-byte rows can have: h = 1 + x, with a decay
    of 1 (each CTA has up to 1024 channels, which passes 2^31 when D is rounded up)."""
    D = LARGEST // 8 * 8
    assert D + 1023 >= 2 ** 31
    x = torch.full((2, D), 2.0, dtype=BF16, device="cuda")
    la = torch.zeros((2, D), dtype=BF16, device="cuda")
    x[1] = 4
    h = torch.ones((2, D), device="cuda")
    y, end = kda.kda_glr_scan(x, la, h, N=2)
    for t in (y, end):
        assert everywhere(t[0], 3) and everywhere(t[1], 5)
    del end, y
    y = kda.kda_glr_step(x, la, h)
    for t in (y, h):
        assert everywhere(t[0], 3) and everywhere(t[1], 5)
    assert kda.kda_get_last_error() == kda.KDA_OK


@gpu
def test_norm_of_the_widest_row():
    """One row of the largest width, with 4096 elements on either side of it that stay: a thread's next
    element, 1024 on, lies past 2^31 behind the last."""
    D, side = LARGEST, 4096
    assert D - 1 + 1024 >= 2 ** 31

    def row(dtype, value):
        whole = torch.full((D + 2 * side,), 7, dtype=dtype, device="cuda")
        whole[side:side + D] = value
        return whole, whole[side:side + D].view(1, D)

    _, x = row(BF16, 1)
    x[0, 0], x[0, -1] = 4, -2  # integers 32 (31.75), 127 and -64 (-63.5, the even one)
    (wy, y), (wq, q) = row(BF16, 0), row(torch.int8, 0)
    kda.kda_rmsnorm(x, y=y)
    inner = everywhere(y[0, 1:-1], 1)  # the mean is 1 + 18 / D
    assert inner and y[0, 0] == 4 and y[0, -1] == -2
    y.zero_()
    _, scale = kda.kda_rmsnorm_i8(x, q=q, y=y)
    assert everywhere(y[0, 1:-1], 1) and y[0, 0] == 4 and y[0, -1] == -2
    assert everywhere(q[0, 1:-1], 32) and q[0, 0] == 127 and q[0, -1] == -64
    assert abs(float(scale) * 127 - 4) < 1e-4
    for whole in (wy, wq):
        assert (whole[:side] == 7).all() and (whole[-side:] == 7).all()

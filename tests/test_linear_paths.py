"""kda_linear's kernels one by one: every variant that a size, a type or an alignment chooses, with
its epilogue (bias, activation, residual, y in place of the residual or in wider rows) and tiles that
the sizes do not fill, against the 64-bit product."""
import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import plain64
from tests.test_linear import BF16, F32, check, make

gpu = pytest.mark.gpu


def wider(t, more=5):
    """t's values as columns of a wider array, the rest of it -1."""
    big = torch.full((t.shape[0], t.shape[1] + more), -1.0, dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def run_all(M, K, N, dtype, act, seed):
    """The epilogue's forms on one shape; the call reports no error."""
    x, w, b, r = make(M, K, N, dtype, seed=seed)
    for bias, res in ((b, r), (None, None)):
        check(kda.kda_linear(x, w, bias, res, act=act), *plain64.linear(x, w, bias, res, act))
    y_ref = plain64.linear(x, w, b, r, act)
    y = r.clone()
    assert kda.kda_linear(x, w, b, y, y, act=act) is y
    check(y, *y_ref)
    y = wider(r)
    kda.kda_linear(x, w, b, y, y, act=act)
    check(y, *y_ref)
    behind = torch.as_strided(y, (M, 5), (N + 5, 1), N)
    assert (behind == -1).all()
    torch.cuda.synchronize()
    assert kda.kda_get_last_error() == kda.KDA_OK


# ------------------------------------------------------------------ K split over a cluster
@gpu
@pytest.mark.parametrize("M, K, N, dtype", [
    (16, 2048, 130, BF16), (37, 2048, 130, BF16), (64, 1024, 257, BF16), (100, 640, 385, BF16),
    (37, 2041, 130, BF16),                       # rows that are shifted into place
    (70, 1024, 70, F32), (65, 515, 129, F32)])
def test_split_with_lanes_outside(M, K, N, dtype):
    """The last tile's lanes fall outside y one by one: they meet the cluster's barrier in step."""
    run_all(M, K, N, dtype, "silu", seed=M + N)


# ------------------------------------------------------------------ pairs of CTAs
def pair_width(M, N):
    """The width of tile that pairs of CTAs take for aligned bf16 rows: the one whose waves cost
    least; None where too few tiles send the product to the split form."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    rows = -(-N // 256)
    if rows * -(-M // 128) < pairs // 2:
        return None
    return min((256, 224, 192, 160, 128),  # the first of equal ones
               key=lambda bn: -(-rows * -(-M // bn) // pairs) * (448 + bn))


PAIRS = [(1300, 1000, 128), (2900, 1000, 160), (3500, 1000, 192), (4100, 1000, 224), (4700, 1000, 256)]


@gpu
@pytest.mark.parametrize("M, N, width", PAIRS)
@pytest.mark.parametrize("K, act", [(136, "gelu_tanh"), (520, "silu"), (1000, "none")])
def test_pairs(M, N, width, K, act):
    """Every width, tiles that M, N and K leave part-filled, every form of the epilogue."""
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert pair_width(M, N) == width
    run_all(M, K, N, BF16, act, seed=M + K)


@gpu
@pytest.mark.parametrize("act", sorted(kda.ACTS))
def test_pairs_activations(act):
    """Odd rows of y: no two channels share an aligned word."""
    assert pair_width(1301, 1001) is not None
    run_all(1301, 264, 1001, BF16, act, seed=7)


@gpu
def test_pairs_several_tiles_each():
    """More tiles than pairs, so that accumulators and stages come round; wide rows of x and w."""
    M, K, N = 2700, 72, 5000
    assert pair_width(M, N) is not None
    x, w, b, r = make(M, K, N, BF16, seed=8)
    x, w = wider(x, 8), wider(w, 16)
    for _ in range(3):
        check(kda.kda_linear(x, w, b, r, act="gelu"), *plain64.linear(x, w, b, r, "gelu"))


@gpu
def test_pairs_what_is_not_finite():
    """NaN and infinities stay in their rows of x and w (and with them in y's)."""
    M, K, N = 1300, 136, 1000
    x, w, b, r = make(M, K, N, BF16, seed=9)
    x[17, 3], x[1299, 135], w[999, 0], w[4, 77] = float("nan"), float("inf"), float("-inf"), float("nan")
    y = kda.kda_linear(x, w, b, r, act="relu")
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[[17, 1299]] = False
    cols[[999, 4]] = False
    y_ref, off = plain64.linear(x[rows.cuda()], w[cols.cuda()], b[cols.cuda()], r[rows.cuda()][:, cols.cuda()], "relu")
    check(y[rows.cuda()][:, cols.cuda()], y_ref, off)
    assert y[17].isnan().all() and y[:, 4].isnan().all()


@gpu
def test_pairs_columns_behind_k_are_not_read():
    """Rows of x and w in wider arrays that hold NaN behind them."""
    M, K, N = 1300, 136, 1000
    x, w, b, r = make(M, K, N, BF16, seed=10)
    xs, ws = (torch.full((t.shape[0], K + 24), float("nan"), dtype=BF16, device="cuda") for t in (x, w))
    xs[:, :K], ws[:, :K] = x, w
    check(kda.kda_linear(xs[:, :K], ws[:, :K], b, r), *plain64.linear(x, w, b, r))


# ------------------------------------------------------------------ very long rows
@gpu
def test_a_product_of_seconds():
    """One row whose shifted parts of K take seconds: no wait of the call covers all of them."""
    K = 1_200_000_001
    x, w = (torch.zeros(K + 1, dtype=BF16, device="cuda")[1:].unsqueeze(0) for _ in range(2))
    at = torch.arange(0, K, 9_999_991, device="cuda")  # 121 places, the sum exact in fp32 and bf16
    x[0, at], w[0, at] = 1.0, 1.0
    w[0, K - 1], x[0, K - 1] = 2.0, 3.0
    y = kda.kda_linear(x, w)
    assert kda.kda_get_last_error() == kda.KDA_OK
    assert float(y) == len(at) + 6

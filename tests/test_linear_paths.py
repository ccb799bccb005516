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

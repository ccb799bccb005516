"""Calls of kda_gdr_prefill and kda_gdr_decode_step that their documentation allows, beyond those of
test_gdr.py: which kernel takes them, many sequences, states far into a pool."""
import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import kda
from tests import plain64
from tests.test_gdr import BF16, TOL, check, cu_of, draw, expect_prefill, pool

gpu = pytest.mark.gpu


@gpu
def test_short_equal_sequences_take_no_workspace():
    """Without cu_seqlens every length is T / N: a token each needs no solve of 64."""
    N, H, d = 256, 32, 64
    args = draw((N,), H, H, d, d, BF16, seed=31)
    S0 = pool(N, H, d, d)
    S_T, o = torch.empty_like(S0), torch.empty_like(args[2])
    kda.kda_gdr_prefill(*args, S0, N=N, o=o, S_T=S_T)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    kda.kda_gdr_prefill(*args, S0, N=N, o=o, S_T=S_T)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
    few = slice(0, 3)
    o_ref, S_ref = expect_prefill([x[few] for x in args], [1] * 3, S0[few])
    check(o[few], o_ref, TOL["simt"], "o")
    check(S_T[few], S_ref, TOL["simt"], "S_T")

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


@gpu
@pytest.mark.parametrize("impl, d, n", [("simt", 128, 2800), ("tc", 128, 2800), ("tc", 64, 11200)])
def test_prefill_far_into_a_pool(impl, d, n):
    """Slots whose offsets pass 2^31 elements, and 2^32; the walks on tcgen05 and on mma.sync."""
    Hv, lens = 96, [70, 5]
    P = torch.empty(n, Hv, d, d, device="cuda")  # 4.4e9 elements, 17.6 GB
    args = draw((sum(lens),), 48, Hv, d, d, BF16, seed=32)
    at = [n // 2, n - 1]
    before = torch.cat([pool(1, Hv, d, d, seed=i) for i in at])
    P[at] = before
    # where offsets cut to 32 bits would land, and next door
    others = [i % (2 ** 32 // (Hv * d * d)) for i in at] + [i - 1 for i in at]
    others = [i for i in others if i not in at]
    P[others] = 7.0
    o, S_T = kda.kda_gdr_prefill(*args, P, cu_of(lens), S_T=P, impl=impl,
                                 slots=torch.tensor(at, dtype=torch.int32, device="cuda"))
    assert S_T is P and kda.kda_get_last_error() == kda.KDA_OK
    o_ref, S_ref = expect_prefill(args, lens, before)
    check(o, o_ref, TOL[impl], "o")
    check(P[at], S_ref, TOL[impl], "states")
    assert (P[others] == 7.0).all()


@gpu
@pytest.mark.parametrize("impl, dk, dv", [("simt", 128, 128), ("tc", 128, 128), ("tc", 64, 64)])
def test_prefill_far_into_a_projection(impl, dk, dv):
    """Rows of q, k and v whose offsets pass 2^31 elements."""
    Hk, Hv, T, lens, wide = 2, 4, 3000, [2900, 70, 30], 1 << 20
    q, k, v, la, beta = draw((T,), Hk, Hv, dk, dv, BF16, seed=33)
    rows = torch.empty(T, wide, dtype=BF16, device="cuda")  # 3.1e9 elements, 6.3 GB
    parts = []
    for x, at in ((q, 0), (k, 4096), (v, wide - Hv * dv)):
        to = rows[:, at:at + x[0].numel()].unflatten(1, x.shape[1:])
        to.copy_(x)
        parts.append(to)
    cu = cu_of(lens)
    # the first sequence is left out
    slots = torch.tensor([-1, 1, 0], dtype=torch.int32, device="cuda")
    S0, S_T = pool(2, Hv, dk, dv), torch.empty(2, Hv, dk, dv, device="cuda")
    o, _ = kda.kda_gdr_prefill(*parts, la, beta, S0, cu, S_T=S_T, slots=slots, impl=impl)
    assert kda.kda_get_last_error() == kda.KDA_OK
    o_ref, S_ref = expect_prefill([x[2900:] for x in (q, k, v, la, beta)], lens[1:], S0[[1, 0]])
    check(o[2900:], o_ref, TOL[impl], "o")
    check(S_T[[1, 0]], S_ref, TOL[impl], "states")


@gpu
@pytest.mark.parametrize("dk, dv", [(128, 128), (64, 256)])
def test_more_sequences_than_a_warp(dk, dv):
    """The walk on tcgen05 with more than 32 sequences, some of them empty, one left out."""
    lens = [(i * 37) % 90 if i % 7 else 0 for i in range(41)]
    N, H = len(lens), 2
    args = draw((sum(lens),), 1, H, dk, dv, BF16, seed=34)
    S0 = pool(N + 3, H, dk, dv)
    slots = torch.arange(N + 2, 2, -1, dtype=torch.int32)
    slots[20] = -1
    P = S0.clone()
    o = torch.full_like(args[2], 5.0)
    kda.kda_gdr_prefill(*args, P, cu_of(lens), o=o, S_T=P, slots=slots.cuda(), impl="tc")
    assert kda.kda_get_last_error() == kda.KDA_OK
    used = slots.tolist()
    o_ref, S_ref = expect_prefill(args, lens, S0[[max(s, 0) for s in used]])
    at = 0
    for n, L in enumerate(lens):
        if used[n] < 0:
            assert L > 0 and (o[at:at + L] == 5.0).all()
        else:
            check(o[at:at + L], o_ref[at:at + L], TOL["tc"], f"o of sequence {n}")
            check(P[used[n]], S_ref[n], TOL["tc"], f"state of sequence {n}")
        at += L
    untouched = [i for i in range(N + 3) if i not in used]
    assert torch.equal(P[untouched], S0[untouched])


@gpu
@pytest.mark.parametrize("Hk, Hv, dk, dv", [(1, 2, 32, 256), (2, 2, 32, 128), (1, 3, 64, 32), (2, 4, 128, 32)])
def test_chunks_of_narrow_heads(Hk, Hv, dk, dv):
    """The walk on mma.sync: two slices of a head, slices of eight, four and two warps."""
    lens = [130, 1, 64, 0, 77]
    args = draw((sum(lens),), Hk, Hv, dk, dv, BF16, seed=35)
    S0 = pool(len(lens), Hv, dk, dv)
    o, S = kda.kda_gdr_prefill(*args, S0, cu_of(lens), impl="tc")
    o_ref, S_ref = expect_prefill(args, lens, S0)
    check(o, o_ref, TOL["tc"], "o")
    check(S, S_ref, TOL["tc"], "S_T")


@gpu
@pytest.mark.parametrize("impl", ["simt", "tc"])
def test_one_token_whatever_its_stride(impl):
    Hk, Hv, d = 1, 2, 128
    q, k, v, la, beta = draw((1,), Hk, Hv, d, d, BF16, seed=36)
    o, S = torch.empty_like(v), torch.empty(1, Hv, d, d, device="cuda")
    opt = kda.kda_gdr_options_init(impl=impl, ldq=1 << 40, ldk=1 << 41, ldv=1 << 42)
    ws = torch.empty(kda.kda_gdr_prefill_workspace_size(1, 1, Hk, Hv, d, d, kda.KDA_BF16, opt) or 16,
                     dtype=torch.uint8, device="cuda")
    opt.workspace, opt.workspace_bytes = ws.data_ptr(), ws.numel()
    rc = kda.load().kda_gdr_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), la.data_ptr(), beta.data_ptr(),
                                    None, None, 1, o.data_ptr(), S.data_ptr(), 1, Hk, Hv, d, d,
                                    kda.KDA_BF16, opt, torch.cuda.current_stream().cuda_stream)
    assert rc == kda.KDA_OK and kda.kda_get_last_error() == kda.KDA_OK
    o_ref, S_ref = expect_prefill((q, k, v, la, beta), [1], None)
    check(o, o_ref, TOL[impl], "o")
    check(S, S_ref, TOL[impl], "S_T")

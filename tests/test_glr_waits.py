"""What the gated linear recurrence does behind a wait that gives up: the kernels, built once more
with waits that give up at once where the test says so, on the GPU.  The status word is set, no state is
written, nothing is on its way any more, and the next call is right."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

from linear_attention_recurrence_prefill_gb300 import build as libbuild
from linear_attention_recurrence_prefill_gb300 import kda

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "csrc", "glr_waits.cu")
OUT = os.path.join(HERE, "_build", "libglr_waits.so")
BF16 = torch.bfloat16
WAIT, GIVE_UP = 0, 1


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    deps = [SRC, *libbuild._deps()]
    if not os.path.exists(OUT) or any(os.path.getmtime(d) > os.path.getmtime(OUT) for d in deps):
        cmd = [libbuild.nvcc(), *libbuild.flags(), "-shared", "-cudart", "shared", SRC, "-o", OUT]
        subprocess.run(cmd, check=True)
    l = ctypes.CDLL(OUT)
    vp, ci = ctypes.c_void_p, ctypes.c_int
    l.glr_waits_scan.argtypes = [vp] * 6 + [ci] * 4
    l.glr_waits_backward.argtypes = [vp] * 8 + [ci] * 4
    return l


def made(T, D):
    g = torch.Generator().manual_seed(3)
    x, dy = (torch.randn(T, D, generator=g).to(BF16).cuda() for _ in range(2))
    return x, (-torch.rand(T, D, generator=g)).to(BF16).cuda(), dy


def fives(*shape, dtype=torch.float32):
    return torch.full(shape, 5.0, dtype=dtype, device="cuda")


def call(lib, f, tensors, *numbers, waits):
    torch.cuda.synchronize()
    assert lib.glr_waits_set(*waits) == 0
    start = time.monotonic()
    assert f(*(t.data_ptr() for t in tensors), *numbers) == 0
    assert time.monotonic() - start < 1.5  # (a wait for something that never comes takes 2 s)


CASES = [(16, 1, GIVE_UP, WAIT), (16, 4, GIVE_UP, WAIT), (16, 4, WAIT, GIVE_UP), (16, 8, GIVE_UP, GIVE_UP),
         (4, 2, WAIT, GIVE_UP), (16, 2, WAIT, GIVE_UP)]


@pytest.mark.parametrize("T", [60, 700, 1500])
@pytest.mark.parametrize("bytes, ranks, tile, totals", CASES)
def test_scan(lib, T, bytes, ranks, tile, totals):
    D = 136
    x, la, _ = made(T, D)
    want, end, saved = kda.kda_glr_scan(x, la, checkpoints=True)
    sizes = (T, D, bytes, ranks)
    for give_up in (False, True, False):
        y, h, cp = fives(T, D, dtype=BF16), fives(1, D), fives(T // 64 + 1, D)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        waits = (tile, totals) if give_up else (WAIT, WAIT)
        call(lib, lib.glr_waits_scan, (x, la, y, h, cp, status), *sizes, waits=waits)
        if give_up:
            assert status.item() == kda.KDA_ERR_TIMEOUT
            assert (h == 5).all()
            done = 0 if tile == GIVE_UP else 64 * ranks  # tokens of the rounds before
            assert (y[done:] == 5).all() and (cp[done // 64:] == 5).all()
        else:
            assert status.item() == 0
            # the same sums in an order of their own for each number of CTAs: within their roundings
            assert ((y.double() - want.double()).abs() <= 2 ** -7 * want.double().abs() + 2 ** -12).all()
            assert ((h - end).abs() <= 2 ** -12).all()


@pytest.mark.parametrize("T", [60, 700, 1500])
@pytest.mark.parametrize("bytes, ranks, tile, totals", CASES)
def test_backward(lib, T, bytes, ranks, tile, totals):
    D = 136
    x, la, dy = made(T, D)
    _, _, saved = kda.kda_glr_scan(x, la, checkpoints=True)
    want = kda.kda_glr_scan_backward(dy, None, x, la, saved)
    sizes = (T, D, bytes, ranks)
    rounds = -(-(-(-T // 64)) // ranks)
    for give_up in (False, True, False):
        dx, dla, dh0 = fives(T, D, dtype=BF16), fives(T, D, dtype=BF16), fives(1, D)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        waits = (tile, totals) if give_up else (WAIT, WAIT)
        call(lib, lib.glr_waits_backward, (dy, x, la, saved, dx, dla, dh0, status), *sizes, waits=waits)
        if give_up:
            assert status.item() == kda.KDA_ERR_TIMEOUT
            assert (dh0 == 5).all()
            left = T if tile == GIVE_UP else 64 * ranks * (rounds - 1)  # tokens of the rounds not begun
            assert (dx[:left] == 5).all() and (dla[:left] == 5).all()
        else:
            assert status.item() == 0
            for got, ref in ((dx, want[0]), (dla, want[1]), (dh0, want[3])):
                assert ((got.double() - ref.double()).abs() <= 2 ** -7 * ref.double().abs() + 2 ** -12).all()

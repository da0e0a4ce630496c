"""Rows of the 16-bit gradients whose source is not there, on the GPU: they count as rows of zeros, whatever they hold."""
import ctypes

import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say
from test_gpu_layer import LAYOUTS, SIXTEEN
from test_gpu_moe import TYPES, rng_for, rows_tensor

pytestmark = pytest.mark.gpu

# S, tokens, slots, E, N, K: few tiles, short rows, sums in parts, tiles of 256 x 256, those in parts, one step a tile
CASES = [(90, 30, 3, 4, 40, 72), (70, 70, 1, 3, 5, 7), (9000, 4500, 2, 1, 136, 136), (6000, 6000, 1, 16, 1024, 1024),
         (20000, 10000, 2, 1, 264, 1848), (400, 50, 8, 40, 64, 64)]


def inputs(case, dtype, layout, gated):
    S, T, k, E, N, K = case
    rng = rng_for("absent", case, dtype, layout, gated)
    rows = 2 * N if gated else N
    A, dC = rows_tensor(rng, T, K, dtype, *layout), rows_tensor(rng, S, N, dtype, *layout)
    B = rows_tensor(rng, E * rows, K, dtype).reshape(E, rows, K)
    pre = rows_tensor(rng, S, 2 * N, dtype, *layout)
    src = rng.permutation(T * k)[:S] if S <= T * k else rng.integers(0, T * k, S)
    absent = np.unique(np.concatenate([[0, S - 1], rng.integers(0, S, max(S // 9, 3))]))
    src[absent] = rng.choice([-1, -2 ** 31, T * k, 2 ** 31 - 1], absent.size)
    bounds = np.concatenate([[0], np.sort(rng.integers(0, S, E - 1)), [S]])
    return A, B, dC, pre, *(torch.from_numpy(v.astype(np.int32)).cuda() for v in (bounds, src)), torch.from_numpy(absent).cuda()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", CASES)
def test_rows_without_a_source(case, dtype, layout, gated):
    say("absent", case, dtype, layout, gated)
    A, B, dC, pre, offsets, src, absent = inputs(case, dtype, layout, gated)
    args = dict(offsets=offsets, src=src, slots=case[2], dA=None)

    def gradient():
        return sp.moe_gated_backward(dC, pre, A, B, **args)[1] if gated else sp.moe_gemm_backward(dC, A, B, **args)[1]

    dC[absent], pre[absent] = 0, 0
    want = gradient()
    assert bool(torch.isfinite(want).all())
    for value in (3.0, float("nan"), float("inf")):
        dC[absent], pre[absent] = value, value
        assert torch.equal(gradient(), want), value


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("S,a_rows,N,K", [(90, 50, 40, 72), (9000, 100, 136, 136), (9000, 8200, 136, 136), (300, 0, 16, 24)])
def test_rows_behind_the_last_of_a(S, a_rows, N, K, layout):
    """Without sources, rows of dC from a_rows on."""
    say("behind", S, a_rows, N, K, layout)
    rng = rng_for("behind", S, a_rows, layout)
    A, dC, B = rows_tensor(rng, S, K, "bf16", *layout), rows_tensor(rng, S, N, "bf16", *layout), rows_tensor(rng, N, K, "bf16")
    need = ctypes.c_size_t()
    assert sp.lib().moe_gemm_backward_bufsize(S, 1, N, K, 1, ctypes.byref(need)) == 0
    work = torch.empty(max(need.value, 16), dtype=torch.uint8, device="cuda")

    def gradient():
        dB = torch.full((N, K), -7.0, dtype=torch.bfloat16, device="cuda")
        assert sp.lib().moe_gemm_backward(S, 1, N, K, 1, dC.data_ptr(), dC.stride(0), A.data_ptr(), a_rows, A.stride(0), None, 1,
                                          B.data_ptr(), B.stride(0), 0, None, None, 0, dB.data_ptr(), K, 0, work.data_ptr(),
                                          work.nbytes, torch.cuda.current_stream().cuda_stream) == 0
        return dB

    dC[a_rows:] = 0
    want = gradient()
    for value in (3.0, float("nan"), float("inf")):
        dC[a_rows:] = value
        assert torch.equal(gradient(), want), value
    assert bool(want.any()) == (a_rows > 0)

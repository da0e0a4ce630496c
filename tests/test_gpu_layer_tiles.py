"""Gradients of the 16-bit products in the tiles that many rows take, on the GPU against their definitions in 64 bits: 256 x 256
ones of every height, whole and in parts, with sources and without.  tests/test_layer_plan_host.py says which case is which."""
import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say
from test_gpu_layer import SIXTEEN, act_ref, backward_ref, check, gradient_buffers, products_inputs
from test_gpu_moe import HALF, LEAST, TYPES, U, dev, f64, rng_for, rows_tensor

pytestmark = pytest.mark.gpu

# T, slots, E (0: one matrix), N, K, dropped, kind
TILES = [(3000, 1, 0, 72, 2816, 0, "random"), (24, 1, 0, 136, 520, 0, "random"), (20000, 1, 0, 264, 1848, 0, "random"),
         (10000, 2, 1, 264, 1848, 0.1, "random"), (2000, 3, 16, 1288, 264, 0.1, "random")]
# rows of each expert, N, K: ends of one to four blocks of 64 rows, few rows, none
COUNTS = [((60, 100, 190, 256, 0, 1000, 700, 1790), 72, 2048), ((257, 320, 1, 3518), 72, 2568)]


def check_backward(rng, S, A, B, offsets, token, args, dtype, what):
    N = B.shape[-2]
    dC = rows_tensor(rng, S, N, dtype)
    dC[offsets[-1]:] = float("nan")
    buf, dA, bbuf, dB = gradient_buffers(S, A, B, dtype, (8, 0))
    sp.moe_gemm_backward(dC, A, B, dA=dA, dB=dB, **args)
    wa, ba, wb, bb = backward_ref(f64(dC), np.zeros(dC.shape), A, B, offsets, token, dtype)
    check(dA, wa, ba, what)
    check(dB, wb, bb, what)
    dA.fill_(-7.0), dB.fill_(-7.0)
    assert bool((buf == -7.0).all()) and bool((bbuf == -7.0).all())


@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", TILES)
def test_gradients_of_large_tiles(case, dtype):
    say("tiles", case, dtype)
    rng, S, A, B, offsets, token, args = products_inputs(case, dtype, (0, 0), False, bool(case[2]))
    check_backward(rng, S, A, B, offsets, token, args, dtype, case)


def counted(counts, rows, K, dtype):
    """Experts with these numbers of rows; tokens' rows in any order, one slot in five routed nowhere."""
    rng = rng_for("counted", counts, rows, K, dtype)
    E, n = len(counts), sum(counts)
    S = n + n // 4
    offsets = np.concatenate([[0], np.cumsum(counts)])
    src = np.concatenate([rng.permutation(S)[:n], np.full(S - n, -1)])
    A = rows_tensor(rng, (S + 1) // 2, K, dtype)
    B = rows_tensor(rng, E * rows, K, dtype, scale=K ** -0.5).reshape(E, rows, K)
    args = dict(offsets=dev(offsets.astype(np.int32)), src=dev(src.astype(np.int32)), slots=2)
    return rng, S, A, B, offsets, src // 2, args


@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("counts,N,K", COUNTS)
def test_gradients_of_experts_of_every_height(counts, N, K, dtype):
    say("heights", counts, N, K, dtype)
    rng, S, A, B, offsets, token, args = counted(counts, N, K, dtype)
    check_backward(rng, S, A, B, offsets, token, args, dtype, counts)


@pytest.mark.parametrize("dtype", SIXTEEN)
def test_gated_gradients_of_experts_of_every_height(dtype):
    counts, N, K = COUNTS[0]
    say("gated heights", counts, N, K, dtype)
    rng, S, A, B, offsets, token, args = counted(counts, 2 * N, K, dtype)
    pre, dH = rows_tensor(rng, S, 2 * N, dtype, scale=1.5), rows_tensor(rng, S, N, dtype)
    pre[offsets[-1]:], dH[offsets[-1]:] = float("nan"), float("nan")
    dA, dB = sp.moe_gated_backward(dH, pre, A, B, dA=torch.full((S, K), -7.0, dtype=TYPES[dtype], device="cuda"), **args)
    h, g, u = f64(dH), f64(pre)[:, :N], f64(pre)[:, N:]
    sig, p, dp = act_ref(g, "silu")
    d = np.concatenate([h * u * sig * (1 + g * dp * (1 - sig)), h * g * sig], 1)
    # in fp32: sig is off by u (4 + 4 |p|) of itself, 1 - sig by that of sig; then rounded
    rough = np.concatenate([np.abs(h * u) * sig * (1 + np.abs(g * dp)), np.abs(h * g * sig)], 1)
    off = rough * U * (16 + 8 * np.abs(np.concatenate([p, p], 1)))
    off = off + HALF[dtype] * (np.abs(d) + off) + LEAST[dtype]
    wa, ba, wb, bb = backward_ref(d, off, A, B, offsets, token, dtype)
    check(dA, wa, ba, counts)
    check(dB, wb, bb, counts)

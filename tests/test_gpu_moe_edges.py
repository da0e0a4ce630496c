"""Calls at the edges of the mixture-of-experts operators: operands on other streams, inside one buffer, scales and
sizes at the ends of their range, and launches with more work than workgroups."""
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say

pytestmark = pytest.mark.gpu


def codes(g, *shape, most=127):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ sums through a wave's own LDS
# each streaming tile (16 x 16, 16 x 32, 32 x 32, 32 x 64) with many steps a wave, aligned and not
@pytest.mark.parametrize("gap", [0, 1])
@pytest.mark.parametrize("M,N,K", [(3, 1500, 9216), (5, 5000, 8200), (5, 5000, 8192), (30, 6000, 8192),
                                   (60, 7000, 8208)])
def test_streaming_tiles_of_many_steps(M, N, K, gap):
    """Every 128 bytes of K take the place of the last ones in a wave's LDS: codes of different size in turn, whose
    exact sums (below 2^24) any word of another step would change."""
    say("streaming tiles", M, N, K, gap)
    g = gen(K)
    A, B = (torch.zeros(r, K + gap, dtype=torch.int8, device="cuda")[:, :K] for r in (M, N))
    size = 4 + torch.arange(K, device="cuda") // 128 % 7 * 4
    for t in (A, B):
        t.copy_((torch.randint(-128, 128, t.shape, generator=g, device="cuda") * size // 128).to(torch.int8))
    want = A.double() @ B.double().t()
    ones = torch.ones(max(M, N), device="cuda")
    for n in range(5):
        got = sp.gemm_i8(A, ones[:M], B, ones[:N], dtype=torch.float32)
        assert torch.equal(got.double(), want), n

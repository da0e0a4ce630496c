"""The cases of the 16-bit gradients' tests reach every kernel that the library has for them."""
import ctypes
import itertools

import spmm_csr_spmv_amd as sp
from layer_plan import kernels, work_bytes
from test_gpu_layer import LAYOUTS, PRODUCTS
from test_gpu_layer_edges import CUTS, LARGE, PLACES
from test_gpu_layer_tiles import COUNTS, TILES

SIZES = [1, 7, 16, 24, 33, 100, 128, 500, 777, 1024, 3000, 4096, 20000, 32768]


def test_rules_are_the_librarys():
    need = ctypes.c_size_t()
    for S, N, K, E in itertools.product(SIZES, (1, 72, 136, 513, 1024, 2048, 4096, 11400), (8, 136, 1111, 2048, 4096, 14336), (1, 3, 8, 64)):
        for gated, fn in ((False, sp.lib().moe_gemm_backward_bufsize), (True, sp.lib().moe_gated_backward_bufsize)):
            assert fn(S, E, N, K, 1, ctypes.byref(need)) == 0
            assert need.value == work_bytes(S, E, N, K, gated), (S, E, N, K, gated)


def test_every_kernel_is_reached():
    reached = set()
    for cases, layouts, gathers in ((PRODUCTS, LAYOUTS, (False, True)), (LARGE + CUTS, PLACES, (True,)), (TILES, [(0, 0)], (True,))):
        for (T, k, E, N, K, *_), (gap, shift), gather in itertools.product(cases, layouts, gathers):
            aligned = not (shift % 8 or (N + gap) % 8 or (K + gap) % 8)
            reached.update(kernels(T * k, max(E, 1), N, K, bool(E), gather and bool(E), aligned))
    for counts, N, K in COUNTS:
        S = sum(counts) + sum(counts) // 4
        assert kernels(S, len(counts), N, K, True, True, True)[0] == "dA 256"
        reached.update(kernels(S, len(counts), N, K, True, True, True))
    want = {"dA %s%s" % x for x in itertools.product(("thin 16", "thin 32", "staged", "128, four steps", "128, two steps"), ("", " in parts"))}
    want |= {"dA 256"}  # parts are of 128 x 128 tiles
    want |= {"dB %s%s%s" % x for x in itertools.product(("staged", "128", "256"), ("", " in parts"), ("", " of sources"))}
    assert not want - reached, sorted(want - reached)
    assert not reached - want, sorted(reached - want)

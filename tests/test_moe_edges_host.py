"""Calls at the edges of the mixture-of-experts entry points that are refused, or decided, on the host."""
import ctypes

import spmm_csr_spmv_amd as sp

WORKSPACE = 4


def test_sort_refuses_a_workspace_over_its_arrays():
    """The counts would overwrite ids that the second kernel reads again, and its places then leave src's range."""
    L = sp.lib()
    n, E = 1 << 20, 64
    size = ctypes.c_size_t()
    assert L.moe_sort_bufsize(n, E, ctypes.byref(size)) == 0 and size.value > 0
    base = 1 << 40  # addresses that are compared only
    at = {"ids": base, "offsets": base + (1 << 30), "src": base + (2 << 30), "pos": base + (3 << 30)}
    nbytes = {"ids": 4 * n, "offsets": 4 * (E + 1), "src": 4 * n, "pos": 4 * n}

    def call(work):
        return L.moe_sort(n, E, *(ctypes.c_void_p(at[k]) for k in ("ids", "offsets", "src", "pos")),
                          ctypes.c_void_p(work), size.value, None)

    for name, a in at.items():
        for work in (a, a + nbytes[name] - 4, a - size.value + 4):
            assert call(work) == WORKSPACE, (name, work - a)


def test_numbers_beyond_32_bits_keep_their_size():
    """What a C int cannot hold is refused as too large or too small, not taken for its low 32 bits."""
    from spmm_csr_spmv_amd._moe import _int32

    for v in (0, 1, -1, 1024, 2 ** 31 - 1, -2 ** 31):
        assert _int32(v) == v
    for v in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 63, 10 ** 30):
        assert _int32(v) == 2 ** 31 - 1 and _int32(-v) == -2 ** 31

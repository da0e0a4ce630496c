"""Calls at the edges of the mixture-of-experts entry points that are refused, or decided, on the host."""
import ctypes
import random

import pytest
import torch

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


def _bytes(t):
    """The addresses of all bytes of a tensor."""
    at = {0}
    for n, d in zip(t.shape, t.stride()):
        at = {x + i * d for x in at for i in range(n)}
    size = t.element_size()
    return {t.data_ptr() + x * size + i for x in at for i in range(size)}


def test_operands_share_bytes():
    """Whatever shares a byte is refused; apart are other ranges, and other columns of rows as far apart."""
    from spmm_csr_spmv_amd._moe import _apart, _rows

    rng = random.Random(1)
    store = torch.zeros(4096, dtype=torch.uint8)
    whole = {t: store.view(t) for t in (torch.int8, torch.float16, torch.float32)}
    seen = {True: 0, False: 0}
    for n in range(4000):
        pair = []
        pitch = 4 * rng.randint(2, 12)  # bytes
        for _ in range(2):
            t = rng.choice(list(whole))
            size = whole[t].element_size()
            ld = (pitch if rng.random() < 0.8 else 4 * rng.randint(2, 12)) // size
            shape, stride = [rng.randint(1, 6), rng.randint(1, ld)], [ld, 1]
            if rng.random() < 0.2:  # matrices, whole row distances apart
                shape, stride = [2] + shape, [ld * rng.randint(shape[0], shape[0] + 2)] + stride
            pair.append(whole[t].as_strided(shape, stride, rng.randint(0, 8 * ld)))
        a, b = pair
        share = bool(_bytes(a) & _bytes(b))
        if share:
            with pytest.raises(ValueError, match="overlaps"):
                _apart(a, "out", b)
        ranges = a.data_ptr() > max(_bytes(b)) or b.data_ptr() > max(_bytes(a))
        same = a.shape[0] > 1 and b.shape[0] > 1 and a.dim() == b.dim() == 2 and (
            a.stride(0) * a.element_size() == b.stride(0) * b.element_size())
        if not share and (ranges or same):
            off = (b.data_ptr() - a.data_ptr()) % (a.stride(0) * a.element_size())
            if ranges or off + b.shape[1] * b.element_size() <= a.stride(0) * a.element_size():
                _apart(a, "out", b)
        seen[share] += 1
    assert min(seen.values()) > 500
    assert _rows(store.view(64, 64)[:, :8], "x") == 64

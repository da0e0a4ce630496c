"""Refusals of the mixture-of-experts entry points, through the C ABI and the
binding; every call returns before it reaches a device."""
import ctypes

import pytest
import torch

import spmm_csr_spmv_amd as sp

SZ = ctypes.c_size_t
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1001)
NULL, SIZE, WORKSPACE, UNSUPPORTED = 1, 2, 4, 5


def test_sort_refusals():
    L = sp.lib()
    b = SZ()
    assert L.moe_sort_bufsize(100, 64, None) == NULL
    assert L.moe_sort_bufsize(-1, 64, ctypes.byref(b)) == SIZE
    assert L.moe_sort_bufsize(2 ** 31, 64, ctypes.byref(b)) == SIZE
    assert L.moe_sort_bufsize(100, 0, ctypes.byref(b)) == UNSUPPORTED
    assert L.moe_sort_bufsize(100, 1025, ctypes.byref(b)) == UNSUPPORTED
    assert L.moe_sort_bufsize(0, 1, ctypes.byref(b)) == 0 and b.value == 0
    assert L.moe_sort_bufsize(2 ** 31 - 1, 1024, ctypes.byref(b)) == 0 and 0 < b.value < 1 << 24
    assert L.moe_sort(100, 64, None, FAKE, FAKE, FAKE, None, 0, None) == NULL
    assert L.moe_sort(100, 64, FAKE, None, FAKE, FAKE, None, 0, None) == NULL
    assert L.moe_sort(100, 64, FAKE, FAKE, None, FAKE, None, 0, None) == NULL
    assert L.moe_sort(100, 64, FAKE, FAKE, FAKE, None, None, 0, None) == NULL
    assert L.moe_sort(100, 64, ODD, FAKE, FAKE, FAKE, None, 0, None) == UNSUPPORTED
    assert L.moe_sort(100, 64, FAKE, FAKE, FAKE, ODD, None, 0, None) == UNSUPPORTED
    big = 1 << 20
    assert L.moe_sort_bufsize(big, 64, ctypes.byref(b)) == 0 and b.value > 0
    assert L.moe_sort(big, 64, FAKE, FAKE, FAKE, FAKE, None, 0, None) == WORKSPACE
    assert L.moe_sort(big, 64, FAKE, FAKE, FAKE, FAKE, FAKE, b.value - 1, None) == WORKSPACE
    assert L.moe_sort(big, 64, FAKE, FAKE, FAKE, FAKE, ODD, b.value, None) == WORKSPACE


def _rows_calls(L):
    """The three row movements with their arguments by name (in order)."""
    return {
        "dispatch": (L.moe_dispatch, dict(T=8, k=2, H=16, S=16, dt=1, X=FAKE, ldx=16, pos=FAKE, Xs=FAKE, lds=16)),
        "combine": (L.moe_combine, dict(T=8, k=2, H=16, S=16, dt=1, Ys=FAKE, lds=16, pos=FAKE, w=FAKE, Y=FAKE,
                                        ldy=16)),
        "backward": (L.moe_combine_backward, dict(T=8, k=2, H=16, S=16, dt=1, dY=FAKE, ldy=16, Ys=FAKE, lds=16,
                                                  pos=FAKE, w=FAKE, dYs=FAKE, ldd=16, dw=FAKE)),
    }


@pytest.mark.parametrize("which", ["dispatch", "combine", "backward"])
def test_row_movement_refusals(which):
    fn, base = _rows_calls(sp.lib())[which]

    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*dict(base, **kw).values(), None)

    for bad in (dict(T=-1), dict(T=2 ** 31), dict(k=0), dict(k=-2), dict(H=-1), dict(S=-1), dict(S=2 ** 31),
                dict(T=2 ** 30, k=2), dict(H=2 ** 31)):
        assert call(**bad) == SIZE, bad
    for dt in (-1, 3):
        assert call(dt=dt) == UNSUPPORTED
    for ld in [n for n in base if n.startswith("ld")]:
        assert call(**{ld: 15}) == SIZE, ld
        assert call(**{ld: 2 ** 62}) == SIZE, ld
    pointers = [n for n, v in base.items() if v is FAKE]
    for p in pointers:
        if not (which == "combine" and p == "w"):  # without weights: all ones
            assert call(**{p: None}) == NULL, p
        assert call(**{p: ODD}) == UNSUPPORTED, p
    assert call(T=0) == 0
    if which != "backward":
        assert call(H=0) == 0
    if which == "dispatch":
        assert call(S=0) == 0


def test_quantize_refusals():
    L = sp.lib()
    base = dict(rows=4, K=32, dt=1, X=FAKE, ldx=32, q=FAKE, ldq=32, scale=FAKE)

    def call(**kw):
        return L.quantize_rows_i8(*dict(base, **kw).values(), None)

    for bad in (dict(rows=-1), dict(rows=2 ** 31), dict(K=-1), dict(K=2 ** 31), dict(ldx=31), dict(ldq=31),
                dict(ldx=2 ** 62)):
        assert call(**bad) == SIZE, bad
    assert call(dt=3) == UNSUPPORTED
    for p in ("X", "q", "scale"):
        assert call(**{p: None}) == NULL
    assert call(X=ODD) == UNSUPPORTED and call(scale=ODD) == UNSUPPORTED
    assert call(rows=0) == 0


def test_product_refusals():
    L = sp.lib()
    base = dict(M=4, N=8, K=32, A=FAKE, lda=32, sa=FAKE, B=FAKE, ldb=32, sb=FAKE, ct=1, C=FAKE, ldc=8)

    def call(**kw):
        return L.gemm_i8(*dict(base, **kw).values(), None)

    for bad in (dict(M=-1), dict(M=2 ** 31), dict(N=-1), dict(N=2 ** 31), dict(K=-1), dict(lda=31), dict(ldb=31),
                dict(ldc=7), dict(lda=2 ** 62)):
        assert call(**bad) == SIZE, bad
    assert call(K=131072, lda=131072, ldb=131072) == UNSUPPORTED  # an int32 sum could overflow
    assert call(ct=3) == UNSUPPORTED and call(ct=-1) == UNSUPPORTED
    for p in ("A", "B", "C", "sa", "sb"):
        assert call(**{p: None}) == NULL, p
    for p in ("C", "sa", "sb"):
        assert call(**{p: ODD}) == UNSUPPORTED, p
    assert call(M=0) == 0 and call(N=0) == 0

    base = dict(S=4, E=3, N=8, K=32, A=FAKE, rows=4, lda=32, sa=FAKE, src=FAKE, slots=2, B=FAKE, ldb=32, strideb=256,
                sb=FAKE, off=FAKE, ct=1, C=FAKE, ldc=8)

    def call(**kw):
        return L.moe_gemm_i8(*dict(base, **kw).values(), None)

    for bad in (dict(S=-1), dict(S=2 ** 31), dict(N=-1), dict(K=-1), dict(rows=-1), dict(slots=0), dict(lda=31),
                dict(ldb=31), dict(ldc=7), dict(strideb=255), dict(strideb=-256), dict(strideb=2 ** 62)):
        assert call(**bad) == SIZE, bad
    assert call(E=0) == UNSUPPORTED and call(E=1025) == UNSUPPORTED and call(ct=3) == UNSUPPORTED
    assert call(K=131072, lda=131072, ldb=131072, strideb=2 ** 20) == UNSUPPORTED
    for p in ("A", "B", "C", "sa", "sb", "off"):
        assert call(**{p: None}) == NULL, p
    for p in ("C", "sa", "sb", "off", "src"):
        assert call(**{p: ODD}) == UNSUPPORTED, p
    assert call(S=0) == 0 and call(N=0) == 0


def test_binding_takes_device_tensors_only():
    ids = torch.zeros(4, 2, dtype=torch.int32)
    x, w = torch.zeros(4, 8), torch.zeros(4, 2)
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sp.moe_sort(ids, 4), lambda: sp.moe_dispatch(x, ids), lambda: sp.moe_combine(x, ids, w),
                 lambda: sp.moe_combine_backward(x, x, ids, w), lambda: sp.quantize_rows_i8(x),
                 lambda: sp.gemm_i8(q, s, q, s), lambda: sp.moe_gemm_i8(q, s, q[None], s[None], off)):
        with pytest.raises(TypeError, match="device tensor"):
            call()


def test_binding_refuses_other_types():
    with pytest.raises(TypeError, match="int32"):
        sp.moe_sort(torch.zeros(4, 2, dtype=torch.int64), 4)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sp.moe_dispatch(torch.zeros(4, 8, dtype=torch.float64), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sp.quantize_rows_i8(torch.zeros(4, 8, dtype=torch.int32))
    with pytest.raises(TypeError, match="int8"):
        sp.gemm_i8(torch.zeros(4, 8), torch.zeros(4), torch.zeros(4, 8), torch.zeros(4))

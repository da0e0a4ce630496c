"""Refusals of the norm, the gated products and the experts' products in 16 bits, through
the C ABI and the binding; every call returns before it reaches a device."""
import ctypes

import pytest
import torch

import spmm_csr_spmv_amd as sp

SZ = ctypes.c_size_t
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1001)
NULL, SIZE, WORKSPACE, UNSUPPORTED = 1, 2, 4, 5
BIG = 1 << 40


def caller(fn, base):
    def call(**kw):
        assert set(kw) <= set(base)
        return fn(*dict(base, **kw).values(), None)
    return call


def norms():
    L = sp.lib()
    rows = dict(rows=4, H=32, dt=1, X=FAKE, ldx=32, R=FAKE, ldr=32, w=FAKE, wt=1, eps=1e-5, sum=FAKE, lds=32)
    return {
        "norm": caller(L.rms_norm, dict(rows, Y=FAKE, ldy=32)),
        "int8": caller(L.rms_norm_i8, dict(rows, Y=FAKE, ldy=32, scale=FAKE)),
        "backward": caller(L.rms_norm_backward, dict(rows=4, H=32, dt=1, dY=FAKE, lddy=32, X=FAKE, ldx=32, w=FAKE, wt=1,
                                                     eps=1e-5, R=FAKE, ldr=32, Y=FAKE, ldy=32, dw=FAKE, work=FAKE, bytes=BIG)),
    }


@pytest.mark.parametrize("which", ["norm", "int8", "backward"])
def test_norm_refusals(which):
    call = norms()[which]
    for bad in (dict(rows=-1), dict(rows=2 ** 31), dict(H=-1), dict(H=2 ** 31), dict(ldx=31), dict(ldr=31), dict(ldy=31),
                dict(ldx=2 ** 62), dict(ldr=2 ** 62), dict(ldy=2 ** 62)):
        assert call(**bad) == SIZE, bad
    for bad in (dict(dt=3), dict(dt=-1), dict(wt=2), dict(dt=0, wt=1), dict(eps=-1e-9), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert call(**bad) == UNSUPPORTED, bad
    for p in ("X", "R", "w"):
        assert call(**{p: ODD}) == UNSUPPORTED, p
    for p in ("X", "Y"):
        assert call(**{p: None}) == NULL, p
    if which == "backward":
        assert call(dY=None) == NULL and call(dY=ODD) == UNSUPPORTED and call(dw=ODD) == UNSUPPORTED
        assert call(lddy=31) == SIZE
        need = SZ()
        assert sp.lib().rms_norm_backward_bufsize(4, 32, 1, ctypes.byref(need)) == 0 and need.value > 0
        assert call(work=None) == WORKSPACE and call(work=ODD) == WORKSPACE and call(bytes=need.value - 1) == WORKSPACE
        assert call(rows=0, dw=None) == 0
    else:
        assert call(sum=None) == NULL and call(sum=ODD) == UNSUPPORTED and call(lds=31) == SIZE and call(lds=2 ** 62) == SIZE
        assert call(rows=0) == 0
    if which == "int8":
        assert call(scale=None) == NULL and call(scale=ODD) == UNSUPPORTED
    else:
        assert call(Y=ODD) == UNSUPPORTED
        assert call(H=0) == 0


def test_norm_workspace_sizes():
    L, b = sp.lib(), SZ()
    assert L.rms_norm_backward_bufsize(4, 32, 1, None) == NULL
    assert L.rms_norm_backward_bufsize(-1, 32, 1, ctypes.byref(b)) == SIZE
    assert L.rms_norm_backward_bufsize(4, 2 ** 31, 1, ctypes.byref(b)) == SIZE
    assert L.rms_norm_backward_bufsize(4, 32, 3, ctypes.byref(b)) == UNSUPPORTED
    for dt in (0, 1, 2):
        for rows, H in ((0, 100), (100, 0)):
            assert L.rms_norm_backward_bufsize(rows, H, dt, ctypes.byref(b)) == 0 and b.value == 0
        for rows, H in ((1, 1), (2 ** 31 - 1, 1), (100, 1 << 20), (2 ** 31 - 1, 2 ** 31 - 1)):
            assert L.rms_norm_backward_bufsize(rows, H, dt, ctypes.byref(b)) == 0 and b.value >= 4 * H


def int8(which):
    L = sp.lib()
    if which == "matrix":
        return caller(L.gated_i8, dict(M=4, N=8, K=32, A=FAKE, lda=32, sa=FAKE, B=FAKE, ldb=32, sb=FAKE, act=0, ct=1, C=FAKE,
                                       ldc=8))
    return caller(L.moe_gated_i8, dict(M=4, E=3, N=8, K=32, A=FAKE, rows=4, lda=32, sa=FAKE, src=FAKE, slots=2, B=FAKE, ldb=32,
                                       strideb=512, sb=FAKE, off=FAKE, act=0, ct=1, C=FAKE, ldc=8))


@pytest.mark.parametrize("which", ["matrix", "experts"])
def test_gated_int8_refusals(which):
    call = int8(which)
    for bad in (dict(M=-1), dict(M=2 ** 31), dict(N=-1), dict(N=2 ** 31), dict(K=-1), dict(lda=31), dict(ldb=31), dict(ldc=7),
                dict(lda=2 ** 62)):
        assert call(**bad) == SIZE, bad
    for bad in (dict(act=-1), dict(act=2), dict(ct=3), dict(K=131072, lda=131072, ldb=131072)):
        assert call(**bad) == UNSUPPORTED, bad
    for p in ("A", "B", "C", "sa", "sb"):
        assert call(**{p: None}) == NULL, p
    for p in ("C", "sa", "sb"):
        assert call(**{p: ODD}) == UNSUPPORTED, p
    assert call(M=0) == 0 and call(N=0) == 0
    if which == "experts":
        for bad in (dict(rows=-1), dict(slots=0), dict(strideb=511), dict(strideb=-512), dict(strideb=2 ** 62)):
            assert call(**bad) == SIZE, bad
        assert call(E=0) == UNSUPPORTED and call(E=1025) == UNSUPPORTED
        assert call(off=None) == NULL and call(off=ODD) == UNSUPPORTED and call(src=ODD) == UNSUPPORTED


def products():
    L = sp.lib()
    head = dict(S=4, E=3, N=8, K=32, dt=1)
    mid = dict(A=FAKE, rows=4, lda=32, src=FAKE, slots=2, B=FAKE, ldb=32, strideb=512, off=FAKE)
    tail = dict(dA=FAKE, ldda=32, dB=FAKE, lddb=32, stridedb=512, work=FAKE, bytes=BIG)
    return {
        "product": caller(L.moe_gemm, dict(head, **mid, C=FAKE, ldc=8)),
        "gated": caller(L.moe_gated, dict(head, **mid, act=0, pre=FAKE, ldp=16, C=FAKE, ldc=8)),
        "product backward": caller(L.moe_gemm_backward, dict(head, C=FAKE, ldc=8, **mid, **tail)),
        "gated backward": caller(L.moe_gated_backward, dict(head, act=0, C=FAKE, ldc=8, pre=FAKE, ldp=16, **mid, **tail)),
    }


@pytest.mark.parametrize("which", ["product", "gated", "product backward", "gated backward"])
def test_product_refusals(which):
    call = products()[which]
    back, gated = "backward" in which, "gated" in which
    for bad in (dict(S=-1), dict(S=2 ** 31 - 1023), dict(S=2 ** 31), dict(N=-1), dict(K=-1), dict(rows=-1), dict(rows=2 ** 31),
                dict(slots=0), dict(slots=-2), dict(lda=31), dict(ldb=31), dict(ldc=7), dict(strideb=(16 if gated else 8) * 32 - 1),
                dict(strideb=-512), dict(strideb=2 ** 62), dict(lda=2 ** 62), dict(ldb=2 ** 62), dict(ldc=2 ** 62)):
        assert call(**bad) == SIZE, bad
    wide = 2 ** 29 + 1
    for bad in (dict(dt=0), dict(dt=3), dict(dt=-1), dict(E=0), dict(E=1025), dict(off=None), dict(N=wide),
                dict(K=wide, lda=wide, ldb=wide)):
        assert call(**bad) == UNSUPPORTED, bad
    for p in ("A", "B", "C", "off", "src"):
        assert call(**{p: ODD}) == UNSUPPORTED, p
    for p in ("A", "B", "C"):
        assert call(**{p: None}) == NULL, p
    if gated:
        assert call(act=2) == UNSUPPORTED and call(act=-1) == UNSUPPORTED
        assert call(pre=ODD) == UNSUPPORTED and call(ldp=15) == SIZE and call(ldp=2 ** 62) == SIZE
    if back:
        for bad in (dict(ldda=31), dict(lddb=31), dict(stridedb=(16 if gated else 8) * 32 - 1), dict(stridedb=2 ** 62),
                    dict(ldda=2 ** 62)):
            assert call(**bad) == SIZE, bad
        assert call(dA=ODD) == UNSUPPORTED and call(dB=ODD) == UNSUPPORTED
        if gated:
            assert call(pre=None) == NULL and call(dA=None, dB=None) == 0
            need = SZ()
            assert sp.lib().moe_gated_backward_bufsize(4, 3, 8, 32, 1, ctypes.byref(need)) == 0 and need.value >= 4 * 16 * 2
            for bad in (dict(work=None), dict(work=ODD), dict(bytes=need.value - 1)):
                assert call(**bad) == WORKSPACE, bad
    else:
        assert call(S=0) == 0 and call(N=0) == 0


@pytest.mark.parametrize("name", ["moe_gemm_backward_bufsize", "moe_gated_backward_bufsize"])
def test_product_workspace_sizes(name):
    size, b = getattr(sp.lib(), name), SZ()
    assert size(4, 3, 8, 32, 1, None) == NULL
    for bad in ((-1, 3, 8, 32, 1), (2 ** 31, 3, 8, 32, 1), (4, 3, -1, 32, 1), (4, 3, 8, -1, 1)):
        assert size(*bad, ctypes.byref(b)) == SIZE, bad
    for bad in ((4, 0, 8, 32, 1), (4, 1025, 8, 32, 1), (4, 3, 8, 32, 0), (4, 3, 2 ** 29 + 1, 32, 1), (4, 3, 8, 2 ** 29 + 1, 1)):
        assert size(*bad, ctypes.byref(b)) == UNSUPPORTED, bad
    for ok in ((0, 1, 0, 0, 1), (4, 3, 8, 32, 2), (2 ** 31 - 1024, 1024, 2 ** 29, 1, 1)):
        assert size(*ok, ctypes.byref(b)) == 0, ok


def test_binding_takes_device_tensors_only():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8)
    q, s = torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sp.rms_norm(x, w), lambda: sp.rms_norm_i8(x, w, residual=x), lambda: sp.rms_norm_backward(x, x, w),
                 lambda: sp.gated_i8(q, s, q, s), lambda: sp.moe_gated_i8(q, s, q[None], s[None], off),
                 lambda: sp.moe_gemm(x, x), lambda: sp.moe_gated(x, x[None], off), lambda: sp.moe_gemm_backward(x, x, x),
                 lambda: sp.moe_gated_backward(x, x, x, x)):
        with pytest.raises(TypeError, match="device tensor"):
            call()


def test_binding_refuses_other_types():
    f = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        sp.moe_gemm(f, f)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        sp.moe_gated_backward(f, f, f, f)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        sp.rms_norm(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(TypeError, match="int8"):
        sp.gated_i8(f, torch.zeros(4), f, torch.zeros(4))

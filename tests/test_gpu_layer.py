"""The norm, the gated products and the experts' products in 16 bits on the GPU against their definitions in 64 bits.

Tolerances: u = 2^-24 is fp32's rounding, h = eps / 2 the output type's.  A sum of m
terms formed by m fp32 steps is off by at most m u sum |terms|; the matrix cores'
additions are counted with 2 u each.  Second-order terms are covered by counting a few steps more.
"""
import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say
from test_gpu_moe import HALF, LEAST, TYPES, U, dev, f64, filled, i64, rng_for, route, rows_tensor, sort_ref

pytestmark = pytest.mark.gpu

EPS = 1e-5
LAYOUTS = [(0, 0), (3, 1), (8, 0), (13, 5)]  # gap between rows, first element's offset
SIXTEEN = ["bf16", "f16"]


def check(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), "%s: %d of %d outside, first %s: got %r, want %r, bound %r" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], ref[bad][0], np.broadcast_to(bound, ref.shape)[bad][0])


# ------------------------------------------------------------------ norm
NORMS = [(0, 8), (1, 1), (3, 7), (5, 8), (2, 9), (17, 64), (33, 511), (16, 512), (9, 513), (7, 2045), (6, 2048), (5, 2049),
         (1, 4096), (3, 8192), (3, 8200), (2, 16387), (1030, 72), (2100, 40)]
WEIGHTS = ["same", "f32", None]


def steps_of(H):
    """fp32 steps of a sum over a row: a lane's own elements, then across 256 lanes."""
    return max(32, (H + 255) // 256 + 8) + 12


def norm_inputs(rng, rows, H, dtype, wtype, residual, layout, scale=1.0):
    x = rows_tensor(rng, rows, H, dtype, *layout, scale=scale)
    r = rows_tensor(rng, rows, H, dtype, *layout, scale=3 * scale) if residual else None
    w = None
    if wtype:
        w = torch.from_numpy(1 + 0.2 * rng.standard_normal(H)).to(torch.float32 if wtype == "f32" else TYPES[dtype]).cuda()
    s = (x.float() + r.float()).to(x.dtype) if residual else x
    return x, r, w, s


def norm_ref(s, w, eps=EPS):
    s, w = f64(s), 1.0 if w is None else f64(w)
    i = 1 / np.sqrt((s * s).mean(1, keepdims=True) + eps) if s.shape[1] else np.ones((s.shape[0], 1))
    return s, w, i


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("wtype", WEIGHTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm(dtype, layout, wtype, residual):
    for rows, H in NORMS:
        say("norm", rows, H, dtype, layout, wtype, residual)
        rng = rng_for(rows, H, dtype, layout, wtype)
        x, r, w, s = norm_inputs(rng, rows, H, dtype, wtype, residual, layout)
        buf, out = filled(rows, H, dtype, *layout)
        got = sp.rms_norm(x, w, residual=r, eps=EPS, out=out)
        if residual:
            assert got[0] is out and torch.equal(got[1], s)
        else:
            assert got is out
        s64, w64, i = norm_ref(s, w)
        y = s64 * i * w64
        check(out, y, np.abs(y) * (HALF[dtype] + (0.5 * steps_of(H) + 6) * U) + LEAST[dtype], (rows, H))
        out.fill_(-7.0)
        assert bool((buf == -7.0).all())  # what lies between the rows


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm_into_int8(dtype, layout, residual):
    for rows, H in NORMS + [(4, 0)]:
        for wtype in WEIGHTS:
            say("norm int8", rows, H, dtype, layout, wtype, residual)
            rng = rng_for(rows, H, dtype, layout, wtype, "i8")
            x, r, w, s = norm_inputs(rng, rows, H, dtype, wtype, residual, layout)
            if rows > 3:
                x[2] = 0
                if residual:
                    r[2] = 0
                    s[2] = 0
            got = sp.rms_norm_i8(x, w, residual=r, eps=EPS)
            if residual:
                assert torch.equal(got[2], s)
            q, scale = i64(got[0]), f64(got[1])
            s64, w64, i = norm_ref(s, w)
            t = s64 * w64
            a = np.abs(t).max(1) if H else np.zeros(rows)
            want = a * i[:, 0] / 127
            assert (np.abs(scale - want) <= want * (0.5 * steps_of(H) + 8) * U).all()
            # s w, its largest, their quotient times 127: five roundings of a value up to 127, then half a code
            assert (np.abs(q - 127 * t / np.where(a, a, 1)[:, None]) <= 0.5 + 127 * 5 * U).all()
            if rows > 3:
                assert scale[2] == 0 and (q[2] == 0).all()


def test_norm_into_int8_with_given_buffers():
    rng = rng_for("given")
    x, r, w, s = norm_inputs(rng, 5, 77, "bf16", "same", True, (0, 0))
    q = torch.full((5, 90), 99, dtype=torch.int8, device="cuda")[:, 3:80]
    scale = torch.empty(5, device="cuda")
    got = sp.rms_norm_i8(x, w, residual=r, q=q, scale=scale, sum_out=r)
    want = sp.rms_norm_i8(s, w)
    assert got[0] is q and got[1] is scale and got[2] is r and torch.equal(r, s)
    assert torch.equal(q, want[0]) and torch.equal(scale, want[1])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm_sum_in_place(dtype):
    for rows, H in [(3, 7), (40, 600), (5, 4096), (3, 9001), (2, 20000)]:
        for into in ("x", "r"):
            x, r, w, s = norm_inputs(rng_for(rows, H, dtype, into), rows, H, dtype, "same", True, (0, 0))
            want = sp.rms_norm(x.clone(), w, residual=r.clone())
            to = x if into == "x" else r
            y, total = sp.rms_norm(x, w, residual=r, sum_out=to)
            assert total is to and torch.equal(to, s) and torch.equal(y, want[0]) and torch.equal(want[1], s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [40, 600, 2500, 9001])
def test_norm_of_rows_whose_squares_leave_the_range(dtype, H):
    rng = rng_for(dtype, H, "range")
    base = rng.standard_normal((6, H))
    x = torch.from_numpy(base * np.array([1e25, 1e-25, 2e36, 1.0, 1e19, 1e-19])[:, None]).to(TYPES[dtype]).cuda()
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(H)).to(TYPES[dtype]).cuda()
    dy = torch.from_numpy(rng.standard_normal((6, H))).to(TYPES[dtype]).cuda()
    for eps in (0.0, 1e-35):
        s64, w64, i = norm_ref(x, w, eps)
        y = s64 * i * w64
        check(sp.rms_norm(x, w, eps=eps), y, np.abs(y) * (HALF[dtype] + (0.5 * steps_of(H) + 8) * U) + LEAST[dtype], eps)
        q, scale = sp.rms_norm_i8(x, w, eps=eps)
        a = np.abs(s64 * w64).max(1)
        assert (np.abs(f64(scale) * 127 / (a * i[:, 0]) - 1) <= (0.5 * steps_of(H) + 8) * U).all()
        assert (np.abs(i64(q) - 127 * s64 * w64 / a[:, None]) <= 0.5 + 127 * 5 * U).all()
        dx, dw = sp.rms_norm_backward(dy, x, w, eps=eps)
        d, bound, dwr, dwb = norm_backward_ref(x, w, dy, None, dtype, eps)
        keep = [1, 3, 4, 5]  # gradients of the largest rows are denormal
        check(dx[keep], d[keep], bound[keep], eps)
        check(dw, dwr, dwb, eps)


def test_norm_of_non_finite_rows():
    x = torch.ones(4, 300, device="cuda", dtype=torch.bfloat16)
    x[1, 5] = float("inf")
    x[2, 299] = float("nan")
    y = sp.rms_norm(x)
    assert torch.isnan(y[1, 5]) and bool((y[1, :5] == 0).all()) and bool(torch.isnan(y[2]).all())
    assert bool((y[0] == 1).all()) and bool((y[3] == 1).all())
    q, scale = sp.rms_norm_i8(x)
    assert torch.isnan(scale[1:3]).all() and not q[1:3].any() and bool((q[0] == 127).all())


def norm_backward_ref(s, w, dy, dsum, dtype, eps=EPS):
    s64, w64, i = norm_ref(s, w, eps)
    H, m = s64.shape[1], steps_of(s64.shape[1])
    dy64, d64 = f64(dy), 0.0 if dsum is None else f64(dsum)
    n, dn = s64 * i, dy64 * w64
    mean = (dn * n).mean(1, keepdims=True)
    dx = i * (dn - n * mean) + d64
    a, b = np.abs(i * dn), np.abs(i * n)
    size = np.abs(dn * n).mean(1, keepdims=True)
    bound = U * ((a + b * size) * (1.5 * m + 12) + b * size * (m + 4) + 2 * np.abs(d64)) + HALF[dtype] * np.abs(dx) + LEAST[dtype]
    dw, rows = (dy64 * n).sum(0), s64.shape[0]
    return dx, bound, dw, U * np.abs(dy64 * n).sum(0) * (rows + 0.5 * m + 40) + 1e-40 + 0 * H


@pytest.mark.parametrize("extra", [False, True])
@pytest.mark.parametrize("wtype", WEIGHTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm_backward(dtype, layout, wtype, extra):
    for rows, H in NORMS[1:]:
        say("norm backward", rows, H, dtype, layout, wtype, extra)
        rng = rng_for(rows, H, dtype, layout, wtype, "back")
        s, dsum, w, _ = norm_inputs(rng, rows, H, dtype, wtype, True, layout)
        dsum = dsum if extra else None
        dy = rows_tensor(rng, rows, H, dtype, *layout)
        buf, out = filled(rows, H, dtype, *layout)
        dx, dw = sp.rms_norm_backward(dy, s, w, eps=EPS, dsum=dsum, dx=out)
        assert dx is out
        want, bound, dwr, dwb = norm_backward_ref(s, w, dy, dsum, dtype)
        check(dx, want, bound, (rows, H))
        if w is None:
            assert dw is None
        else:
            assert dw.dtype == torch.float32
            check(dw, dwr, dwb, (rows, H, "weight"))
        out.fill_(-7.0)
        assert bool((buf == -7.0).all())


def test_norm_backward_of_no_rows_and_a_workspace():
    w = torch.ones(33, device="cuda")
    dx, dw = sp.rms_norm_backward(torch.empty(0, 33, device="cuda"), torch.empty(0, 33, device="cuda"), w)
    assert dx.shape == (0, 33) and not dw.any()
    rng = rng_for("work")
    s, dy, _, _ = norm_inputs(rng, 50, 33, "f32", None, True, (0, 0))
    want = sp.rms_norm_backward(dy, s, w)
    work = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for g, r in zip(sp.rms_norm_backward(dy, s, w, work=work), want):
            assert torch.equal(g, r)
    with pytest.raises(sp.SparseError) as e:
        sp.rms_norm_backward(dy, s, w, work=work[:100])
    assert e.value.code == 4


def test_norm_backward_against_differences():
    rng = rng_for("differences")
    s = rng.standard_normal((4, 70))
    w, dy, v, vw = rng.standard_normal(70), rng.standard_normal((4, 70)), rng.standard_normal((4, 70)), rng.standard_normal(70)

    def f(s, w):
        return (dy * s * w / np.sqrt((s * s).mean(1, keepdims=True) + EPS)).sum()

    t = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    dx, dw = sp.rms_norm_backward(t(dy), t(s), t(w), eps=EPS)
    step = 1e-5  # differences of 64-bit values: the step's square and 2^-53 / step are below 1e-9
    along = (f(s + step * v, w + step * vw) - f(s - step * v, w - step * vw)) / (2 * step)
    terms = np.abs(f64(dx) * v).sum() + np.abs(f64(dw) * vw).sum()
    # inputs and gradients are rounded to fp32: some 60 roundings of each term
    assert abs((f64(dx) * v).sum() + (f64(dw) * vw).sum() - along) <= 100 * U * terms + 1e-8 * terms


# ------------------------------------------------------------------ activations
def act_ref(g, act):
    """sig(p), p, p' in 64 bits."""
    c = 2 * np.sqrt(2 / np.pi)
    p, dp = (g, np.ones_like(g)) if act == "silu" else (c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g))
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-p)), p, dp


def gated_ref(g, u, eg, eu, act, half, least):
    """a(g) u and its bound, for g and u off by eg and eu: |a'| is below 1.13, exp(-p) is off by u (2 + 4 |p|)."""
    sig, p, _ = act_ref(g, act)
    h = g * sig * u
    bound = 1.13 * eg * (np.abs(u) + eu) + np.abs(g * sig) * eu + np.abs(h) * (half + U * (12 + 4 * np.abs(p))) + least
    return h, bound


# ------------------------------------------------------------------ gated products in int8
# T, slots, E (0: one matrix), N, K, dropped, kind
GATED = [(1, 1, 0, 1, 1, 0, "random"), (1, 1, 0, 33, 64, 0, "random"), (5, 1, 0, 7, 100, 0, "random"),
         (16, 1, 0, 100, 513, 0, "random"), (33, 1, 0, 257, 128, 0, "random"), (130, 1, 0, 300, 272, 0, "random"),
         (300, 1, 0, 129, 400, 0, "random"), (600, 1, 0, 520, 160, 0, "random"),
         (1, 8, 16, 40, 64, 0, "random"), (3, 2, 4, 5, 9, 0, "random"), (40, 4, 8, 65, 200, 0.2, "skew"),
         (100, 3, 5, 31, 96, 0.1, "random"), (70, 2, 3, 64, 15, 0, "one"), (9, 2, 3, 64, 48, 0, "none"),
         (500, 2, 3, 144, 128, 0.05, "skew"), (64, 1, 2, 48, 4100, 0, "random")]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("case", GATED)
def test_gated_int8(case, pad, out, act):
    say("gated int8", case, pad, out, act)
    T, k, E, N, K, dropped, kind = case
    rng = rng_for(case, pad, out)
    codes = lambda *shape: dev(rng.integers(-127, 128, shape).astype(np.int8))  # noqa: E731
    A = codes(T, K + pad)[:, :K]
    sa = dev((rng.random(T) * 0.02 + 0.01).astype(np.float32))
    B = codes(max(E, 1), 2 * N, K + pad)[:, :, :K]
    sb = dev((rng.random((max(E, 1), 2 * N)) * 0.03 / np.sqrt(K)).astype(np.float32))
    S = T * k
    buf, C = filled(S, N, out, 3, 1)
    if E:
        offsets, src, _ = sort_ref(route(rng, T, k, E, dropped, kind), E)
        got = sp.moe_gated_i8(A, sa, B, sb, dev(offsets.astype(np.int32)), src=dev(src.astype(np.int32)), slots=k, act=act, out=C)
    else:
        offsets, src = np.array([0, T]), np.arange(T)
        got = sp.gated_i8(A, sa, B[0], sb[0], act=act, out=C)
    assert got is C
    want, bound = np.full((S, N), -7.0), np.zeros((S, N))
    for e in range(max(E, 1)):
        mine = np.arange(offsets[e], offsets[e + 1])
        row = src[mine] // k
        y = (i64(A)[row] @ i64(B[e]).T) * f64(sa)[row][:, None] * f64(sb[e])
        # the float of the sum, then two products
        want[mine], bound[mine] = gated_ref(y[:, :N], y[:, N:], 3.1 * U * np.abs(y[:, :N]), 3.1 * U * np.abs(y[:, N:]), act,
                                            HALF[out], LEAST[out])
    check(C, want, bound, case)
    C.fill_(-7.0)
    assert bool((buf == -7.0).all())


def test_gated_int8_with_far_scales():
    """Scales whose products with a sum pass fp32's range on the way only."""
    M, N, K = 70, 40, 96
    rng = rng_for("far")
    A, B = (dev(rng.integers(-127, 128, s).astype(np.int8)) for s in ((M, K), (2 * N, K)))
    sa = torch.full((M,), 2.0 ** 100, device="cuda")
    sa[::3] = 1.0
    sb = torch.full((2 * N,), 2.0 ** -110, device="cuda")
    got = sp.gated_i8(A, sa, B, sb, dtype=torch.float32)
    y = (i64(A) @ i64(B).T) * f64(sa)[:, None] * f64(sb)
    h, bound = gated_ref(y[:, :N], y[:, N:], 3.1 * U * np.abs(y[:, :N]), 3.1 * U * np.abs(y[:, N:]), "silu", HALF["f32"], LEAST["f32"])
    check(got, h, bound, "far")


# ------------------------------------------------------------------ products in 16 bits
# T, slots, E (0: one matrix), N, K, dropped, kind
PRODUCTS = [(1, 1, 0, 1, 1, 0, "random"), (1, 1, 0, 9, 8, 0, "random"), (2, 1, 0, 16, 7, 0, "random"),
            (1, 1, 0, 128, 256, 0, "random"), (16, 1, 0, 72, 520, 0, "random"), (37, 1, 0, 131, 65, 0, "random"),
            (100, 1, 0, 264, 192, 0, "random"), (257, 1, 0, 300, 128, 0, "random"), (520, 1, 0, 280, 328, 0, "random"),
            (1, 8, 16, 40, 64, 0, "random"), (3, 2, 4, 5, 9, 0, "random"), (24, 2, 6, 96, 136, 0.2, "random"),
            (40, 4, 8, 33, 200, 0.2, "skew"), (90, 2, 3, 64, 15, 0, "one"), (9, 2, 3, 24, 48, 0, "none"),
            (300, 3, 4, 144, 72, 0.1, "skew"), (500, 2, 3, 264, 136, 0.05, "random"), (64, 1, 2, 8, 2064, 0, "random")]


def products_inputs(case, dtype, layout, gate, gather):
    T, k, E, N, K, dropped, kind = case
    rng = rng_for(case, dtype, layout, gate, gather)
    S, rows, n = T * k, (2 * N if gate else N), max(E, 1)
    A = rows_tensor(rng, T if gather else S, K, dtype, *layout)
    B = rows_tensor(rng, n * rows + (n - 1) * 3, K, dtype, *layout, scale=1 / np.sqrt(K))
    ld = B.stride(0)
    B = torch.as_strided(B, (n, rows, K), ((rows + 3) * ld, ld, 1), B.storage_offset())
    if E:
        offsets, src, _ = sort_ref(route(rng, T, k, E, dropped, kind), E)
        args = dict(offsets=dev(offsets.astype(np.int32)))
        if gather:
            args.update(src=dev(src.astype(np.int32)), slots=k)
    else:
        offsets, src, args, B = np.array([0, S]), np.arange(S), {}, B[0]
    token = src // k if gather else np.arange(S)
    return rng, S, A, B, offsets, token, args


def experts(offsets, B):
    for e in range(len(offsets) - 1):
        yield np.arange(offsets[e], offsets[e + 1]), B[e] if B.dim() == 3 else B


def sums_ref(a, b):
    """a b and the bound of fp32 sums of it."""
    return a @ b, 2 * U * (a.shape[1] + 16) * (np.abs(a) @ np.abs(b))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", PRODUCTS)
def test_product(case, dtype, layout, gather):
    say("product", case, dtype, layout, gather)
    if gather and not case[2]:
        gather = False
    _, S, A, B, offsets, token, args = products_inputs(case, dtype, layout, False, gather)
    N = case[3]
    buf, C = filled(S, N, dtype, *layout)
    assert sp.moe_gemm(A, B, out=C, **args) is C
    want, bound = np.full((S, N), -7.0), np.zeros((S, N))
    for mine, b in experts(offsets, B):
        y, e = sums_ref(f64(A)[token[mine]], f64(b).T)
        want[mine], bound[mine] = y, e + HALF[dtype] * (np.abs(y) + e) + LEAST[dtype]
    check(C, want, bound, case)
    C.fill_(-7.0)
    assert bool((buf == -7.0).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", PRODUCTS)
def test_gated(case, dtype, layout, act):
    say("gated", case, dtype, layout, act)
    _, S, A, B, offsets, token, args = products_inputs(case, dtype, layout, True, bool(case[2]))
    N = case[3]
    buf, C = filled(S, N, dtype, *layout)
    pre_buf, pre = filled(S, 2 * N, dtype, *layout)
    assert sp.moe_gated(A, B, act=act, pre=pre, out=C, **args) is C
    h, hb = np.full((S, N), -7.0), np.zeros((S, N))
    y, yb = np.full((S, 2 * N), -7.0), np.zeros((S, 2 * N))
    for mine, b in experts(offsets, B):
        p, e = sums_ref(f64(A)[token[mine]], f64(b).T)
        y[mine], yb[mine] = p, e + HALF[dtype] * (np.abs(p) + e) + LEAST[dtype]
        h[mine], hb[mine] = gated_ref(p[:, :N], p[:, N:], e[:, :N], e[:, N:], act, HALF[dtype], LEAST[dtype])
    check(C, h, hb, case)
    check(pre, y, yb, case)
    again = sp.moe_gated(A, B, act=act, **args)  # without the pre-activations
    for mine, _ in experts(offsets, B):
        assert torch.equal(again[torch.from_numpy(mine)], C[torch.from_numpy(mine)])
    C.fill_(-7.0), pre.fill_(-7.0)
    assert bool((buf == -7.0).all()) and bool((pre_buf == -7.0).all())


def backward_ref(dC, eC, A, B, offsets, token, dtype):
    """dA, dB and their bounds for a dC (64 bits) that is off by eC; rows of dA behind the last are -7."""
    a64 = f64(A)
    dA, bA = np.full((dC.shape[0], a64.shape[1]), -7.0), np.zeros((dC.shape[0], a64.shape[1]))
    dB, bB = [], []
    for mine, b in experts(offsets, B):
        b, d, ed, a = f64(b), dC[mine], eC[mine], a64[token[mine]]
        y, e = sums_ref(d, b)
        e = e * 1.01 + 1.01 * (ed @ np.abs(b))
        dA[mine], bA[mine] = y, e + HALF[dtype] * (np.abs(y) + e) + LEAST[dtype]
        y, e = sums_ref(d.T, a)
        e = e * 1.01 + 1.01 * (ed.T @ np.abs(a))
        dB.append(y), bB.append(e + HALF[dtype] * (np.abs(y) + e) + LEAST[dtype])
    if B.dim() == 2:
        return dA, bA, dB[0], bB[0]
    return dA, bA, np.stack(dB), np.stack(bB)


def gradient_buffers(S, A, B, dtype, layout):
    K = A.shape[1]
    buf, dA = filled(S, K, dtype, *layout)
    rows = B.shape[-2]
    n = B.shape[0] if B.dim() == 3 else 1
    bbuf, flat = filled(n * (rows + 2), K, dtype, *layout)
    dB = torch.as_strided(flat, (n, rows, K), ((rows + 2) * flat.stride(0), flat.stride(0), 1), flat.storage_offset())
    return buf, dA, bbuf, dB if B.dim() == 3 else dB[0]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", PRODUCTS)
def test_product_backward(case, dtype, layout, gather):
    say("product backward", case, dtype, layout, gather)
    if gather and not case[2]:
        gather = False
    rng, S, A, B, offsets, token, args = products_inputs(case, dtype, layout, False, gather)
    dC = rows_tensor(rng, S, case[3], dtype, *layout)
    dC[offsets[-1]:] = float("nan")  # rows that no expert has
    buf, dA, bbuf, dB = gradient_buffers(S, A, B, dtype, layout)
    got = sp.moe_gemm_backward(dC, A, B, dA=dA, dB=dB, **args)
    assert got[0] is dA and got[1] is dB
    wa, ba, wb, bb = backward_ref(f64(dC), np.zeros(dC.shape), A, B, offsets, token, dtype)
    check(dA, wa, ba, case)
    check(dB, wb, bb, case)
    one = sp.moe_gemm_backward(dC, A, B, dA=None, **args)  # either alone
    assert one[0] is None and torch.equal(one[1], dB)
    one = sp.moe_gemm_backward(dC, A, B, dB=None, **args)
    assert one[1] is None and torch.equal(one[0][:offsets[-1]], dA[:offsets[-1]])
    dA.fill_(-7.0), dB.fill_(-7.0)
    assert bool((buf == -7.0).all()) and bool((bbuf == -7.0).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", PRODUCTS)
def test_gated_backward(case, dtype, layout, act):
    say("gated backward", case, dtype, layout, act)
    rng, S, A, B, offsets, token, args = products_inputs(case, dtype, layout, True, bool(case[2]))
    N = case[3]
    dH, pre = rows_tensor(rng, S, N, dtype, *layout), rows_tensor(rng, S, 2 * N, dtype, *layout, scale=1.5)
    dH[offsets[-1]:] = float("nan")
    pre[offsets[-1]:] = float("nan")
    buf, dA, bbuf, dB = gradient_buffers(S, A, B, dtype, layout)
    got = sp.moe_gated_backward(dH, pre, A, B, act=act, dA=dA, dB=dB, **args)
    assert got[0] is dA and got[1] is dB
    h, g, u = f64(dH), f64(pre)[:, :N], f64(pre)[:, N:]
    sig, p, dp = act_ref(g, act)
    d = np.concatenate([h * u * sig * (1 + g * dp * (1 - sig)), h * g * sig], 1)
    # in fp32: sig is off by u (4 + 4 |p|) of itself, 1 - sig by that of sig; then rounded
    rough = np.concatenate([np.abs(h * u) * sig * (1 + np.abs(g * dp)), np.abs(h * g * sig)], 1)
    off = rough * U * (16 + 8 * np.abs(np.concatenate([p, p], 1)))
    off = off + HALF[dtype] * (np.abs(d) + off) + LEAST[dtype]
    wa, ba, wb, bb = backward_ref(d, off, A, B, offsets, token, dtype)
    check(dA, wa, ba, case)
    check(dB, wb, bb, case)
    dA.fill_(-7.0), dB.fill_(-7.0)
    assert bool((buf == -7.0).all()) and bool((bbuf == -7.0).all())


def test_gated_backward_against_differences():
    """A directional derivative of sum(dH * gated(A, B)) from the kernels' gradients and from 64-bit differences."""
    rng = rng_for("gated differences")
    T, E, k, N, K = 20, 3, 2, 24, 40
    offsets, src, _ = sort_ref(route(rng, T, k, E), E)
    token = src // k
    # values that 16 bits hold
    h16 = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
    A, B, dH = h16(T, K), (h16(E, 2 * N, K) / 8).astype(np.float16), h16(T * k, N)
    vA, vB = rng.standard_normal(A.shape), rng.standard_normal(B.shape)

    def f(a, b, act):
        total = 0.0
        for e in range(E):
            mine = np.arange(offsets[e], offsets[e + 1])
            y = a[token[mine]] @ b[e].T
            total += (dH[mine] * y[:, :N] * act_ref(y[:, :N], act)[0] * y[:, N:]).sum()
        return total

    o, s, r = dev(offsets.astype(np.int32)), dev(src.astype(np.int32)), dev(dH)
    for act in ("silu", "gelu_tanh"):
        pre = torch.empty(T * k, 2 * N, dtype=torch.float16, device="cuda")
        sp.moe_gated(dev(A), dev(B), o, src=s, slots=k, act=act, pre=pre)
        dA, dB = sp.moe_gated_backward(r, pre, dev(A), dev(B), o, src=s, slots=k, act=act)
        a64, b64, step = A.astype(np.float64), B.astype(np.float64), 1e-5
        along = (f(a64 + step * vA, b64 + step * vB, act) - f(a64 - step * vA, b64 - step * vB, act)) / (2 * step)
        got = (f64(dA) * vA[token]).sum() + (f64(dB) * vB).sum()
        # pre, dpre and the gradients are each rounded by 2^-11 of values whose absolute sum this is (a'' is below 1.2)
        y = np.concatenate([a64[token[offsets[e]:offsets[e + 1]]] @ b64[e].T for e in range(E)])
        d = np.abs(np.concatenate([dH * y[:, N:], dH * y[:, :N]], 1)) * 1.2 + np.abs(np.concatenate([dH * y[:, N:] * y[:, :N], dH * y[:, :N] * y[:, N:]], 1)) * 1.2
        terms = sum((d[offsets[e]:offsets[e + 1]] * (np.abs(vA[token[offsets[e]:offsets[e + 1]]]) @ np.abs(b64[e]).T
                                                     + np.abs(a64[token[offsets[e]:offsets[e + 1]]]) @ np.abs(vB[e]).T)).sum()
                    for e in range(E))
        assert abs(got - along) <= 3.5 * HALF["f16"] * terms


# ------------------------------------------------------------------ what a caller may get wrong, or rely on
def test_rows_hold_non_finite_values_apart():
    """An Inf or a NaN in one row, in a column behind a row's end or in the padding reaches its own results only."""
    for dtype in SIXTEEN:
        for K, N, S in ((72, 40, 70), (65, 33, 50), (200, 264, 300), (1, 3, 5)):
            say("apart", dtype, K, N, S)
            rng = rng_for("apart", K)
            buf = torch.full((S, K + 8), float("nan"), dtype=TYPES[dtype], device="cuda")
            A = buf[:, :K]
            A.copy_(torch.from_numpy(rng.standard_normal((S, K))))
            bbuf = torch.full((N, K + 8), float("inf"), dtype=TYPES[dtype], device="cuda")
            B = bbuf[:, :K]
            B.copy_(torch.from_numpy(rng.standard_normal((N, K))))
            clean = sp.moe_gemm(A, B)
            assert bool(torch.isfinite(clean).all())
            dC = torch.full((S, N + 8), float("nan"), dtype=TYPES[dtype], device="cuda")[:, :N]
            dC.copy_(torch.from_numpy(rng.standard_normal((S, N))))
            dA, dB = sp.moe_gemm_backward(dC, A, B)
            assert bool(torch.isfinite(dA).all()) and bool(torch.isfinite(dB).all())
            A[S // 2, 0], B[N // 2, K - 1] = float("nan"), float("inf")
            got = sp.moe_gemm(A, B)
            hit = torch.zeros(S, N, dtype=torch.bool, device="cuda")
            hit[S // 2] = True
            hit[:, N // 2] = True
            assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], clean[~hit])


def test_offsets_of_any_kind():
    """Offsets outside the rows, descending ones and sources outside A: nothing outside is touched."""
    rng = rng_for("offsets")
    S, N, K, E = 60, 24, 40, 4
    A, B = rows_tensor(rng, S, K, "bf16"), rows_tensor(rng, E * N, K, "bf16").reshape(E, N, K)
    dC = rows_tensor(rng, S, N, "bf16")
    for offsets in ([-5, 10, 30, 90, 2 ** 31 - 1], [0, 30, 20, 40, 60], [10, 20, 20, 20, 50], [0, 0, 0, 0, 0]):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        clip = np.clip(offsets, 0, S)
        _, out = filled(S, N, "bf16")
        sp.moe_gemm(A, B, o, out=out)
        _, dA = filled(S, K, "bf16")
        _, dB = sp.moe_gemm_backward(dC, A, B, o, dA=dA)
        rows = np.zeros(S, int)
        for e in range(E):
            mine = np.arange(clip[e], max(clip[e], clip[e + 1]))
            rows[mine] += 1
            y, b = sums_ref(f64(dC)[mine].T, f64(A)[mine])
            check(dB[e], y, b + HALF["bf16"] * (np.abs(y) + b) + LEAST["bf16"], offsets)
        assert bool((out[torch.from_numpy(rows == 0)] == -7.0).all()) and bool((dA[torch.from_numpy(rows == 0)] == -7.0).all())
        if rows.max() < 2:
            for e in range(E):
                mine = np.arange(clip[e], max(clip[e], clip[e + 1]))
                y, b = sums_ref(f64(A)[mine], f64(B[e]).T)
                check(out[torch.from_numpy(mine)], y, b + HALF["bf16"] * (np.abs(y) + b) + LEAST["bf16"], offsets)
    src = torch.from_numpy(rng.permutation(S).astype(np.int32)).cuda()
    src[3], src[40], src[59] = -1, S, 2 ** 31 - 1
    o = torch.tensor([0, 25, 25, 50, 60], dtype=torch.int32, device="cuda")
    _, out = filled(S, N, "bf16")
    sp.moe_gemm(A, B, o, src=src, out=out)
    assert bool((out[[3, 40, 59]] == -7.0).all())
    _, dB = sp.moe_gemm_backward(dC, A, B, o, src=src)
    for e, (lo, hi) in enumerate(((0, 25), (25, 25), (25, 50), (50, 60))):
        mine = [p for p in range(lo, hi) if p not in (3, 40, 59)]
        y, b = sums_ref(f64(dC)[mine].T, f64(A)[i64(src)[mine]])
        check(dB[e], y, b + HALF["bf16"] * (np.abs(y) + b) + LEAST["bf16"], "sources")


def test_empty_operands():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert sp.moe_gemm(z(0, 8), z(3, 5, 8), o).shape == (0, 5)
    dA, dB = sp.moe_gemm_backward(z(0, 5), z(0, 8), z(3, 5, 8), o)
    assert dA.shape == (0, 8) and dB.shape == (3, 5, 8) and not dB.any()
    dA, dB = sp.moe_gated_backward(z(0, 5), z(0, 10), z(0, 8), z(3, 10, 8), o)
    assert dA.shape == (0, 8) and dB.shape == (3, 10, 8) and not dB.any()
    assert not sp.moe_gemm(z(4, 0), z(5, 0)).any() and not sp.moe_gated(z(4, 0), z(6, 0)).any()
    assert sp.moe_gemm(z(4, 8), z(0, 8)).shape == (4, 0)
    dA, dB = sp.moe_gemm_backward(z(4, 0), z(4, 8) + 1, z(0, 8))
    assert not dA.any() and dB.shape == (0, 8)
    dA, dB = sp.moe_gemm_backward(z(4, 5), z(4, 0), z(5, 0))
    assert dA.shape == (4, 0) and dB.shape == (5, 0)
    assert sp.rms_norm(z(0, 8)).shape == (0, 8) and sp.rms_norm(z(4, 0)).shape == (4, 0)
    assert sp.gated_i8(torch.zeros(0, 8, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda"),
                       torch.zeros(6, 8, dtype=torch.int8, device="cuda"), torch.zeros(6, device="cuda")).shape == (0, 3)


def test_results_are_reproducible():
    rng = rng_for("again")
    A, B, dH = (rows_tensor(rng, r, c, "bf16") for r, c in ((900, 136), (528, 136), (900, 264)))
    pre = rows_tensor(rng, 900, 528, "bf16")
    s, dy, w = (rows_tensor(rng, r, 520, "bf16") for r in (3000, 3000, 1))
    first = None
    for _ in range(5):
        got = (sp.moe_gated(A, B), *sp.moe_gated_backward(dH, pre, A, B), *sp.rms_norm_backward(dy, s, w[0]))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_on_a_stream_of_its_own():
    rng = rng_for("stream")
    A, B, dC = (rows_tensor(rng, r, c, "f16") for r, c in ((300, 72), (40, 72), (300, 40)))
    want = (sp.moe_gemm(A, B), *sp.moe_gemm_backward(dC, A, B), *sp.rms_norm(A, residual=A))
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    got = (sp.moe_gemm(A, B, stream=stream), *sp.moe_gemm_backward(dC, A, B, stream=stream),
           *sp.rms_norm(A, residual=A, stream=stream))
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_captured_into_a_graph():
    """A layer's step, forward and backward, replayed on other inputs; eager calls between the replays."""
    rng = rng_for("graph")
    T, k, E, N, K = 50, 2, 4, 40, 72
    offsets, src, pos = sort_ref(route(rng, T, k, E), E)
    o, s, p = (dev(a.astype(np.int32)) for a in (offsets, src, pos))
    x, r = rows_tensor(rng, T, K, "bf16"), rows_tensor(rng, T, K, "bf16")
    w, B1, B2 = rows_tensor(rng, 1, K, "bf16")[0], rows_tensor(rng, E * 2 * N, K, "bf16").reshape(E, 2 * N, K), \
        rows_tensor(rng, E * K, N, "bf16").reshape(E, K, N)
    pre = torch.empty(T * k, 2 * N, dtype=torch.bfloat16, device="cuda")

    def step():
        y, total = sp.rms_norm(x, w, residual=r)
        h = sp.moe_gated(y, B1, o, src=s, slots=k, pre=pre)
        out = sp.moe_combine(sp.moe_gemm(h, B2, o), p)
        d = sp.moe_dispatch(out, p)
        dh, dB2 = sp.moe_gemm_backward(d, h, B2, o)
        dx, dB1 = sp.moe_gated_backward(dh, pre, y, B1, o, src=s, slots=k)
        return (out, dB2, dB1, *sp.rms_norm_backward(sp.moe_combine(dx, p), total, w, dsum=out))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = step()
    for seed in range(4):
        x.copy_(rows_tensor(rng_for("graph", seed), T, K, "bf16"))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(static, want))


# ------------------------------------------------------------------ together
def test_a_served_layer():
    """norm -> int8 -> gated experts -> int8 -> experts -> back to the tokens, against 64 bits with the codes that the
    calls gave."""
    rng = rng_for("served")
    for T in (1, 7, 200):
        k, E, H, N = 3, 6, 136, 88
        x, r, w, s = norm_inputs(rng, T, H, "bf16", "f32", True, (0, 0))
        codes = lambda *shape: dev(rng.integers(-127, 128, shape).astype(np.int8))  # noqa: E731
        B1, B2 = codes(E, 2 * N, H), codes(E, H, N)
        s1, s2 = (dev((rng.random(t) * 0.01 / np.sqrt(c)).astype(np.float32)) for t, c in (((E, 2 * N), H), ((E, H), N)))
        ids = dev(route(rng, T, k, E, 0.1))
        weights = dev(rng.random((T, k)).astype(np.float32))
        offsets, src, pos = sp.moe_sort(ids, E)
        q, sq, total = sp.rms_norm_i8(x, w, residual=r)
        h = sp.moe_gated_i8(q, sq, B1, s1, offsets, src=src, slots=k)
        qh, sh = sp.quantize_rows_i8(h)
        y = sp.moe_combine(sp.moe_gemm_i8(qh, sh, B2, s2, offsets), pos, weights)
        assert torch.equal(total, s)
        out, size = np.zeros((T, H)), np.zeros((T, H))
        for t in range(T):
            for j in range(k):
                e, p = int(ids[t, j]), int(pos[t, j])
                if p < 0:
                    continue
                g = (i64(q)[t] @ i64(B1[e]).T) * f64(sq)[t] * f64(s1[e])
                hr, hb = gated_ref(g[:N], g[N:], 3.1 * U * np.abs(g[:N]), 3.1 * U * np.abs(g[N:]), "silu", HALF["bf16"], LEAST["bf16"])
                assert (np.abs(f64(h)[p] - hr) <= hb).all()
                v = f64(weights)[t, j] * (i64(qh)[p] @ i64(B2[e]).T) * f64(sh)[p] * f64(s2[e])
                out[t] += v
                size[t] += np.abs(v)
        # each expert's row is rounded to bf16, then the sum of k of them
        check(y, out, size * (1.01 * HALF["bf16"] + 8 * U) + HALF["bf16"] * np.abs(out) * 1.01 + LEAST["bf16"] * (k + 1), T)


class _Layer(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, w, B1, B2, weights, offsets, src, pos):
        k = pos.shape[1]
        y, s = sp.rms_norm(x, w, residual=r)
        pre = torch.empty(src.shape[0], B1.shape[1], dtype=x.dtype, device=x.device)
        h = sp.moe_gated(y, B1, offsets, src=src, slots=k, pre=pre)
        z = sp.moe_gemm(h, B2, offsets)
        ctx.save_for_backward(y, s, w, B1, B2, weights, offsets, src, pos, pre, h, z)
        return sp.moe_combine(z, pos, weights), s

    @staticmethod
    def backward(ctx, dout, ds):
        y, s, w, B1, B2, weights, offsets, src, pos, pre, h, z = ctx.saved_tensors
        dz, dweights = sp.moe_combine_backward(dout.contiguous(), z, pos, weights)
        dh, dB2 = sp.moe_gemm_backward(dz, h, B2, offsets)
        dys, dB1 = sp.moe_gated_backward(dh, pre, y, B1, offsets, src=src, slots=pos.shape[1])
        dx, dw = sp.rms_norm_backward(sp.moe_combine(dys, pos), s, w, dsum=ds.contiguous())
        return dx, dx, dw.to(w.dtype), dB1, dB2, dweights, None, None, None


@pytest.mark.parametrize("dtype", SIXTEEN)
def test_a_trained_layer(dtype):
    """The gradients of a layer in the framework's calls against autograd's of the same formulas in 64 bits."""
    rng = rng_for("trained", dtype)
    T, k, E, H, N = 60, 2, 4, 72, 48
    t = lambda *shape, scale=1.0: torch.from_numpy(rng.standard_normal(shape) * scale).to(TYPES[dtype]).cuda()  # noqa: E731
    leaves = [t(T, H), t(T, H), 1 + t(H, scale=0.1), t(E, 2 * N, H, scale=H ** -0.5), t(E, H, N, scale=N ** -0.5),
              torch.rand(T, k, device="cuda") * 0.5 + 0.25]
    ids = route(rng, T, k, E, 0.1)
    offsets, src, pos = sp.moe_sort(dev(ids), E)
    d1, d2 = t(T, H), t(T, H)
    own = [v.clone().requires_grad_() for v in leaves]
    out, s = _Layer.apply(*own, offsets, src, pos)
    torch.autograd.backward((out, s), (d1, d2))

    ref = [v.detach().cpu().double().requires_grad_() for v in leaves]
    x, r, w, B1, B2, weights = ref
    s64 = x + r
    y = s64 * torch.rsqrt((s64 * s64).mean(1, keepdim=True) + 1e-6) * w
    outs = []
    for a in range(T):
        row = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = int(ids[a, j])
            if 0 <= e < E:
                g = B1[e] @ y[a]
                row = row + weights[a, j] * (B2[e] @ (torch.nn.functional.silu(g[:N]) * g[N:]))
        outs.append(row)
    torch.autograd.backward((torch.stack(outs), s64), (d1.cpu().double(), d2.cpu().double()))
    # a chain of at most ten roundings to 16 bits (s, y, pre, h, z, dz, dh, dpre, dys, dx), each of at most h relative to
    # values whose norm the products keep about; independent, so that norms add as squares: 2 sqrt(10) h with a factor
    # of two for the chain's amplification
    for name, a, b in zip(("x", "r", "w", "B1", "B2", "weights"), own, ref):
        got, want = f64(a.grad), b.grad.numpy()
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert off <= 2 * np.sqrt(10) * HALF[dtype], (name, off)

"""The mixture-of-experts operators on the GPU against their definitions in 64 bits.

Tolerances: u = 2^-24 is fp32's rounding, h = eps / 2 the output type's.  A sum of
m fp32 products formed by m fused steps is off by at most m u sum |terms| (first
order; the bounds below add one more u for the second), then rounded once by h.
"""
import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # below the normal range: half a step, at most


def rng_for(*key):
    return np.random.default_rng(list(str(key).encode()))


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def i64(t):
    return t.detach().cpu().numpy().astype(np.int64)


def rows_tensor(rng, rows, H, dtype, gap=0, shift=0, scale=1.0):
    """rows x H values of `dtype`, rows H + gap elements apart, `shift` elements off the buffer's start."""
    buf = torch.from_numpy(rng.standard_normal(rows * (H + gap) + shift + 1) * scale).to(TYPES[dtype]).cuda()
    return torch.as_strided(buf, (rows, H), (H + gap, 1), shift)


def filled(rows, H, dtype, gap=0, shift=0, value=-7.0):
    buf = torch.full((rows * (H + gap) + shift + 1,), value, dtype=TYPES[dtype], device="cuda")
    return buf, torch.as_strided(buf, (rows, H), (H + gap, 1), shift)


def route(rng, T, k, E, dropped=0.0, kind="random"):
    if kind == "one":      # every slot to the last expert
        ids = np.full((T, k), E - 1)
    elif kind == "none":   # nothing is routed
        ids = np.where(rng.random((T, k)) < 0.5, -1, E + rng.integers(0, 9, (T, k)))
    elif kind == "skew":   # a few experts take nearly all
        ids = np.minimum(rng.geometric(0.5, (T, k)) - 1, E - 1)
    else:
        ids = rng.integers(0, E, (T, k))
    if dropped:
        ids = np.where(rng.random((T, k)) < dropped, rng.choice([-1, -2 ** 31, E, 2 ** 31 - 1], (T, k)), ids)
    return ids.astype(np.int32)


def sort_ref(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    kept = np.flatnonzero((flat >= 0) & (flat < E))
    order = kept[np.argsort(flat[kept], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))])
    src = np.full(flat.size, -1)
    src[:order.size] = order
    pos = np.full(flat.size, -1)
    pos[order] = np.arange(order.size)
    return offsets, src, pos.reshape(ids.shape)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ sort
SORTS = [(0, 1, 1, 0, "random"), (1, 1, 1, 0, "random"), (1, 8, 64, 0, "random"), (1, 1, 1024, 0, "random"),
         (7, 3, 5, 0.3, "random"), (63, 1, 2, 0, "random"), (64, 1, 64, 0, "random"), (65, 1, 65, 0.1, "random"),
         (100, 8, 257, 0, "skew"), (33, 8, 512, 0.2, "random"), (50, 2, 1, 0, "one"), (50, 2, 7, 0, "none"),
         (2048, 4, 128, 0, "random"), (8192, 1, 1024, 0.1, "random"), (8193, 1, 128, 0, "random"),
         (4097, 2, 513, 0, "random"), (20000, 3, 9, 0.5, "skew"), (20000, 8, 256, 0.1, "random"),
         (70001, 1, 1000, 0.05, "random"), (30000, 4, 33, 0, "one"), (30000, 4, 33, 0, "none"),
         (300007, 8, 60, 0.02, "skew")]


@pytest.mark.parametrize("T,k,E,dropped,kind", SORTS)
def test_sort(T, k, E, dropped, kind):
    say("sort", T, k, E, dropped, kind)
    ids = route(rng_for(T, k, E), T, k, E, dropped, kind)
    got = sp.moe_sort(dev(ids), E)
    for name, g, r in zip(("offsets", "src", "pos"), got, sort_ref(ids, E)):
        assert g.dtype == torch.int32 and tuple(g.shape) == r.shape
        np.testing.assert_array_equal(i64(g), r, err_msg=name)


def test_sort_of_sorted_and_reversed_ids():
    E = 40
    for ids in (np.sort(np.arange(9000) % E), np.sort(np.arange(9000) % E)[::-1]):
        ids = ids.astype(np.int32).reshape(-1, 1).copy()
        for g, r in zip(sp.moe_sort(dev(ids), E), sort_ref(ids, E)):
            np.testing.assert_array_equal(i64(g), r)


def test_sort_with_a_workspace_and_other_shapes():
    rng = rng_for("workspace")
    for shape in ((9000,), (3000, 3), (30, 20, 15), ()):
        ids = rng.integers(-1, 20, shape).astype(np.int32)
        work = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        got = sp.moe_sort(dev(ids).reshape(shape), 20, work=work)
        for g, r in zip(got, sort_ref(ids, 20)):
            np.testing.assert_array_equal(i64(g), r)
    with pytest.raises(sp.SparseError) as e:
        sp.moe_sort(dev(rng.integers(0, 20, 9000).astype(np.int32)), 20, work=work[:100])
    assert e.value.code == 4


# ------------------------------------------------------------------ rows
# T, slots, E, H, share routed nowhere, kind
MOVES = [(1, 1, 1, 1, 0, "random"), (1, 8, 64, 4096, 0, "random"), (3, 2, 4, 7, 0, "random"),
         (5, 3, 2, 8, 0.4, "random"), (9, 4, 16, 9, 0, "random"), (17, 8, 8, 64, 0.2, "random"),
         (33, 5, 11, 257, 0.2, "random"), (40, 9, 12, 130, 0.1, "random"), (64, 17, 3, 100, 0.1, "skew"),
         (21, 6, 7, 2045, 0.3, "random"), (300, 2, 8, 1001, 0.1, "skew"), (30, 2, 8, 8200, 0, "random"),
         (6, 2, 5, 33, 0, "none"), (1030, 1, 5, 72, 0.5, "random"), (4, 2, 3, 0, 0, "random"),
         # whole lines by 64 lanes a token, and whole rows a workgroup (2048 tokens and more)
         (40, 3, 5, 320, 0.1, "random"), (33, 2, 5, 512, 0, "random"), (2050, 2, 4, 2176, 0.1, "random")]
LAYOUTS = [(0, 0), (3, 1), (8, 0), (13, 5)]  # gap between rows, first element's offset


def _moves(case, dtype, layout):
    T, k, E, H, dropped, kind = case
    rng = rng_for(case, dtype, layout)
    ids = route(rng, T, k, E, dropped, kind)
    _, src, pos = sort_ref(ids, E)
    return rng, T, k, H, src, pos, dev(pos.astype(np.int32))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", MOVES)
def test_dispatch(case, dtype, layout):
    say("dispatch", case, dtype, layout)
    rng, T, k, H, src, pos, dpos = _moves(case, dtype, layout)
    X = rows_tensor(rng, T, H, dtype, *layout)
    buf, out = filled(T * k, H, dtype, *layout)
    want_buf, want = filled(T * k, H, dtype, *layout)
    got = sp.moe_dispatch(X, dpos, out=out)
    assert got is out
    live = torch.from_numpy(np.flatnonzero(src >= 0)).cuda()
    want[live] = X[torch.from_numpy(src[src >= 0] // k).cuda()]
    assert torch.equal(buf, want_buf)  # rows behind the last routed one and the gaps too


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", MOVES)
def test_combine(case, dtype, layout, weighted):
    say("combine", case, dtype, layout, weighted)
    rng, T, k, H, src, pos, dpos = _moves(case, dtype, layout)
    Ys = rows_tensor(rng, T * k, H, dtype, *layout)
    Ys[torch.from_numpy(np.flatnonzero(src < 0)).cuda()] = float("nan")  # rows that no slot names
    w = rng.random((T, k)).astype(np.float32)
    w = np.where(pos < 0, np.float32("inf"), w)                          # weights of slots routed nowhere
    buf, out = filled(T, H, dtype, *layout)
    sp.moe_combine(Ys, dpos, dev(w) if weighted else None, out=out)
    y = f64(Ys)
    ref, mag = np.zeros((T, H)), np.zeros((T, H))
    for j in range(k):
        t = np.flatnonzero(pos[:, j] >= 0)
        term = (w[t, j, None].astype(np.float64) if weighted else 1.0) * y[pos[t, j]]
        ref[t] += term
        mag[t] += np.abs(term)
    tol = (k + 1) * U * mag
    tol += HALF[dtype] * (np.abs(ref) + tol) + LEAST[dtype]
    err = np.abs(f64(out) - ref)
    assert (err <= tol).all(), (err - tol).max()
    if layout[0] and T and H:  # the gaps are not written
        gaps = torch.as_strided(buf, (T, layout[0]), (H + layout[0], 1), layout[1] + H)
        assert (gaps[:-1] == -7).all() and (buf[:layout[1]] == -7).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("case", MOVES)
def test_combine_backward(case, dtype, layout):
    say("combine backward", case, dtype, layout)
    rng, T, k, H, src, pos, dpos = _moves(case, dtype, layout)
    dY = rows_tensor(rng, T, H, dtype, *layout)
    Ys = rows_tensor(rng, T * k, H, dtype, *layout)
    Ys[torch.from_numpy(np.flatnonzero(src < 0)).cuda()] = float("nan")
    w = np.where(pos < 0, np.float32("nan"), rng.standard_normal((T, k)).astype(np.float32))
    buf, dYs = filled(T * k, H, dtype, *layout)
    got, dw = sp.moe_combine_backward(dY, Ys, dpos, dev(w), dYs=dYs)
    assert got is dYs
    g, y, o = f64(dY), f64(Ys), f64(dYs)
    live = np.flatnonzero(src >= 0)
    ref = w.reshape(-1)[src[live], None].astype(np.float64) * g[src[live] // k]
    tol = U * np.abs(ref)
    tol += HALF[dtype] * (np.abs(ref) + tol) + LEAST[dtype]
    assert (np.abs(o[live] - ref) <= tol).all()
    assert (o[src < 0] == -7).all()
    p = np.maximum(pos, 0)
    terms = np.where(pos[..., None] >= 0, g[:, None, :] * np.nan_to_num(y)[p], 0.0)
    err = np.abs(f64(dw) - terms.sum(-1))
    assert (err <= (H + 1) * U * np.abs(terms).sum(-1)).all()
    assert (i64(dw == 0)[pos < 0] == 1).all()


def test_gradients_against_differences():
    """<loss weights, dispatch and combine> in 64-bit differences: both operators are linear in each argument, so a
    central difference of the fp32 result is exact up to its own rounding."""
    rng = rng_for("differences")
    T, k, E, H = 12, 3, 5, 20
    ids = route(rng, T, k, E, 0.2)
    _, src, pos = sort_ref(ids, E)
    dpos = dev(pos.astype(np.int32))
    X, Ys = (rows_tensor(rng, n, H, "f32") for n in (T, T * k))
    w, up_y, up_s = dev(rng.standard_normal((T, k)).astype(np.float32)), rows_tensor(rng, T, H, "f32"), rows_tensor(
        rng, T * k, H, "f32")
    live = torch.from_numpy(src >= 0).cuda()
    up_s[~live] = 0

    def f_dispatch(x):
        return float((sp.moe_dispatch(x, dpos, out=torch.zeros(T * k, H, device="cuda")).double() * up_s.double()).sum())

    def f_combine(ys, ww):
        return float((sp.moe_combine(ys, dpos, ww).double() * up_y.double()).sum())

    dX = sp.moe_combine(up_s, dpos)
    dYs, dw = sp.moe_combine_backward(up_y, Ys, dpos, w, dYs=torch.zeros(T * k, H, device="cuda"))
    step = 0.5
    # each output is off by at most (k + 1) u of the terms it sums; two evaluations, divided by 2 step
    noise = 2 * (k + 2) * U * float((up_y.abs().sum() + up_s.abs().sum()) * 8 * k) / (2 * step)
    for _ in range(25):
        for t, grad, f in ((X, dX, f_dispatch), (Ys, dYs, lambda v: f_combine(v, w)), (w, dw, lambda v: f_combine(Ys, v))):
            i, j = rng.integers(t.shape[0]), rng.integers(t.shape[1])
            a, b = t.clone(), t.clone()
            a[i, j] += step
            b[i, j] -= step
            slope = (f(a) - f(b)) / float(a[i, j].double() - b[i, j].double())
            assert abs(slope - float(grad[i, j])) <= noise, (slope, float(grad[i, j]))


def test_fewer_places_than_slots():
    """S below T * slots: what was sorted behind it is dropped, as a capacity over all experts would."""
    rng = rng_for("capacity")
    T, k, E, H, S = 50, 4, 6, 40, 120
    _, src, pos = sort_ref(route(rng, T, k, E), E)
    dpos = dev(pos.astype(np.int32))
    X = rows_tensor(rng, T, H, "f32")
    Xs = sp.moe_dispatch(X, dpos, S=S)
    np.testing.assert_array_equal(f64(Xs), f64(X)[src[:S] // k])
    dweights = torch.full((T, k), 9.0, device="cuda")
    dYs, dw = sp.moe_combine_backward(X, Xs, dpos, torch.ones(T, k, device="cuda"), dweights=dweights)
    assert dw is dweights
    np.testing.assert_array_equal(f64(dYs), f64(X)[src[:S] // k])
    norm = (f64(X) ** 2).sum(-1, keepdims=True)
    assert (np.abs(f64(dw) - np.where(pos < S, norm, 0)) <= (H + 1) * U * norm).all()


def test_places_out_of_range_are_skipped():
    rng = rng_for("range")
    T, k, H, S = 6, 3, 24, 10
    pos = rng.permutation(T * k).reshape(T, k).astype(np.int64)
    pos[0, 0], pos[1, 1], pos[2, 2] = -5, 2 ** 31 - 1, -2 ** 31
    ok = (pos >= 0) & (pos < S)
    X = rows_tensor(rng, T, H, "bf16")
    buf, out = filled(S, H, "bf16")
    sp.moe_dispatch(X, dev(pos.astype(np.int32)), out=out)
    want = np.full((S, H), -7.0)
    want[pos[ok]] = f64(X)[np.nonzero(ok)[0]]
    np.testing.assert_array_equal(f64(out), want)
    Y = sp.moe_combine(out, dev(pos.astype(np.int32)))
    ref = np.stack([f64(out)[pos[t][ok[t]]].sum(0) for t in range(T)])
    assert (np.abs(f64(Y) - ref) <= (HALF["bf16"] + 8 * U) * np.abs(ref) + 8 * U * 60).all()


@pytest.mark.parametrize("H", [3, 200])
def test_no_sorted_rows(H):
    """S = 0: every slot is routed nowhere, whatever its place says."""
    pos = dev(np.array([[0, -1], [5, 1], [2, 2]], np.int32))
    Ys = torch.empty(0, H, device="cuda")
    assert (sp.moe_combine(Ys, pos, torch.ones(3, 2, device="cuda")) == 0).all()
    dYs, dw = sp.moe_combine_backward(torch.ones(3, H, device="cuda"), Ys, pos, torch.ones(3, 2, device="cuda"))
    assert dYs.shape == (0, H) and (dw == 0).all()
    assert sp.moe_dispatch(torch.ones(3, H, device="cuda"), pos, S=0).shape == (0, H)


def test_infinities_travel():
    pos = dev(np.array([[0, 1], [2, -1]], np.int32))
    Ys = torch.tensor([[float("inf"), 1.0], [float("-inf"), 2.0], [float("inf"), float("nan")]], device="cuda")
    w = torch.tensor([[1.0, 1.0], [0.0, 5.0]], device="cuda")
    Y = sp.moe_combine(Ys, pos, w).cpu()
    assert Y[0, 0].isnan() and Y[0, 1] == 3.0 and Y[1].isnan().all()  # inf - inf, 0 inf, 0 nan
    Y = sp.moe_combine(Ys, pos).cpu()
    assert Y[0, 0].isnan() and Y[1, 0] == float("inf") and Y[1, 1].isnan()


# ------------------------------------------------------------------ quantised rows
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 16), (3, 7), (5, 64), (2, 255), (9, 1111), (4, 4096), (3, 8200), (2, 40000),
                                    (513, 40), (2, 0)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_quantize(rows, K, dtype, layout):
    say("quantize", rows, K, dtype, layout)
    rng = rng_for(rows, K, dtype, layout)
    X = rows_tensor(rng, rows, K, dtype, *layout)
    if rows > 2 and K > 3:
        X[0] = 0
        X[1, 2] = X[1].abs().max() * 2      # halves of the largest value: 63.5 rounds to 64
        X[1, 1] = X[1, 2] / 2
        X[1, 0] = -X[1, 2] / 2
    qb = torch.full((rows * (K + layout[0]) + layout[1] + 1,), 99, dtype=torch.int8, device="cuda")
    q = torch.as_strided(qb, (rows, K), (K + layout[0], 1), layout[1])
    _, s = sp.quantize_rows_i8(X, q=q)
    x = f64(X)
    a = np.abs(x).max(1, initial=0.0)
    live = a >= 2.0 ** -119
    ref = 127 * x / np.where(live, a, 1.0)[:, None]
    np.testing.assert_array_equal(s.cpu().numpy(), np.where(live, a.astype(np.float32) / np.float32(127), 0))
    got = i64(q)
    if dtype == "f32":  # 127 x and the quotient are rounded to 24 bits before rint
        assert (np.abs(got - ref) <= 0.5 + 127 * 2 * U).all()
    else:               # exact: halves to even
        np.testing.assert_array_equal(got, np.rint(ref))
    if layout[0] and K:
        gaps = torch.as_strided(qb, (rows, layout[0]), (K + layout[0], 1), layout[1] + K)
        assert (gaps[:-1] == 99).all() and (qb[:layout[1]] == 99).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_quantize_special_rows(dtype):
    """Infinities, NaN, and magnitudes at both ends of the range."""
    t = TYPES[dtype]
    top = torch.finfo(t).max
    least = torch.finfo(t).smallest_normal
    rows = torch.zeros(9, 70)
    rows[:, 0], rows[:, 1], rows[:, 2] = 1.0, -0.5, 0.25
    rows[0, 69], rows[1, 68], rows[2, 3] = float("inf"), float("nan"), float("-inf")
    rows[3, 5], rows[3, 6] = top, -top
    rows[4, :3] = torch.tensor([least, -least, least / 2])
    rows[5, :3] = torch.tensor([2.0 ** -119, -2.0 ** -119, 2.0 ** -120])
    rows[6, :3] = torch.tensor([2.0 ** -120, -2.0 ** -121, 0])
    rows[7, :3] = 0
    X = rows.to(t).cuda()
    q, s = sp.quantize_rows_i8(X)
    x = f64(X)
    a = np.abs(x).max(1)
    got, scale = i64(q), f64(s)
    assert np.isnan(scale[:3]).all() and (got[:3] == 0).all()
    for r in range(3, 9):
        if a[r] < 2.0 ** -119:
            assert scale[r] == 0 and (got[r] == 0).all()
        else:
            assert scale[r] == np.float64(np.float32(a[r]) / np.float32(127))
            np.testing.assert_array_equal(got[r], np.rint(127 * x[r] / a[r]))


# ------------------------------------------------------------------ products
def codes(rng, *shape):
    v = np.clip(np.rint(rng.standard_normal(shape) * 40), -128, 127)
    return v.astype(np.int8)


def strided(a, gap=0, shift=0):
    """An int8 matrix on the device, rows gap bytes further apart than its columns, shift bytes off."""
    rows, K = a.shape
    buf = torch.full((rows * (K + gap) + shift + 16,), 77, dtype=torch.int8, device="cuda")
    v = torch.as_strided(buf, (rows, K), (K + gap, 1), shift)
    v.copy_(torch.from_numpy(a))
    return v


def product_close(got, sums, sa, sb, dtype):
    ref = sums * sa[:, None].astype(np.float64) * sb.astype(np.float64)
    tol = 3.001 * U * np.abs(ref)
    tol += HALF[dtype] * (np.abs(ref) + tol) + LEAST[dtype]
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), (np.argwhere(~(err <= tol))[:5], (err - tol).max())


# M, N, K
PRODUCTS = [(1, 1, 1), (1, 64, 64), (1, 130, 1111), (2, 17, 16), (3, 33, 100), (5, 200, 4096), (15, 31, 127),
            (16, 16, 64), (17, 257, 129), (31, 64, 640), (33, 96, 255), (64, 128, 256), (65, 129, 1024), (100, 300, 513),
            (127, 255, 128), (130, 258, 192), (256, 256, 512), (257, 513, 1000), (300, 40, 2000), (40, 300, 8192),
            (513, 1025, 384), (7, 5, 0), (2, 3, 131071), (520, 264, 65),
            # one or more of each tile size: 16x32, 32x32, 32x64, 128x128 with four and two steps in LDS, 256x256
            (3, 8200, 80), (16, 4200, 300), (130, 1000, 200), (300, 1000, 129), (600, 1100, 700), (2100, 2100, 136),
            (2049, 2200, 400), (3000, 3100, 300), (2817, 4097, 128)]
STRIDES = [(0, 0), (16, 16), (5, 3)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K, stride, dtype):
    say("product", M, N, K, stride, dtype)
    rng = rng_for(M, N, K, stride)
    gap = stride[0] if stride[0] != 16 else (-K) % 16 + 16  # rows a multiple of 16 bytes apart
    A, B = codes(rng, M, K), codes(rng, N, K)
    sa = (rng.random(M) * 1e-2).astype(np.float32)
    sb = ((rng.random(N) + 0.5) / (40 * np.sqrt(K + 1))).astype(np.float32)
    buf, out = filled(M, N, dtype, *((7, 3) if stride[0] else (0, 0)))
    sp.gemm_i8(strided(A, gap, stride[1]), dev(sa), strided(B, gap, stride[1]), dev(sb), out=out)
    product_close(out, A.astype(np.float64) @ B.astype(np.float64).T, sa, sb, dtype)
    if stride[0]:
        gaps = torch.as_strided(buf, (M, 7), (N + 7, 1), 3 + N)
        assert (gaps[:-1] == -7).all() and (buf[:3] == -7).all()


def test_product_of_extreme_codes():
    """The largest sums that int32 has to hold: K = 131071 products of -128 and -128."""
    K = 131071
    A = np.full((20, K), -128, np.int8)
    B = np.full((33, K), -128, np.int8)
    B[1::2] = 127
    one = np.ones(64, np.float32)
    for gap in (0, 1):  # rows 16-byte aligned and not
        got = sp.gemm_i8(strided(A, gap), dev(one[:20]), strided(B, gap), dev(one[:33]), dtype=torch.float32)
        product_close(got, A.astype(np.float64) @ B.astype(np.float64).T, one[:20], one[:33], "f32")


@pytest.mark.parametrize("M,N,K", [(3, 70, 64), (40, 70, 160), (300, 400, 128), (600, 1100, 48)])
def test_product_of_unaligned_buffers(M, N, K):
    """Row distances of whole 16 bytes, first elements off by one: each operand alone, then both."""
    rng = rng_for("unaligned", M)
    A, B = codes(rng, M, K), codes(rng, N, K)
    sa, sb = np.ones(M, np.float32), np.ones(N, np.float32)
    want = A.astype(np.float64) @ B.astype(np.float64).T
    for a, b in ((0, 1), (1, 0), (1, 1)):
        got = sp.gemm_i8(strided(A, 0, a), dev(sa), strided(B, 0, b), dev(sb), dtype=torch.float32)
        np.testing.assert_array_equal(f64(got), want)  # sums below 2^24


def test_scales_travel():
    """A NaN scale makes its row NaN, an infinite one infinite (NaN where the sum is 0), a zero one zero, and no other."""
    rng = rng_for("scales")
    for M in (5, 150):
        A, B = codes(rng, M, 64), codes(rng, 70, 64)
        B[3] = 0
        sa = np.ones(M, np.float32)
        sa[1], sa[2], sa[3] = np.nan, np.inf, 0
        sums = A.astype(np.float64) @ B.astype(np.float64).T
        got = f64(sp.gemm_i8(dev(A), dev(sa), dev(B), dev(np.ones(70, np.float32)), dtype=torch.float32))
        assert np.isnan(got[1]).all() and (got[3] == 0).all() and np.isnan(got[2, 3])
        np.testing.assert_array_equal(got[2][sums[2] != 0], np.sign(sums[2][sums[2] != 0]) * np.inf)
        rest = [0] + list(range(4, M))
        np.testing.assert_array_equal(got[rest], sums[rest])


def test_empty_products():
    z8, z = torch.zeros(0, 32, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda")
    a8, a = torch.ones(4, 32, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    assert sp.gemm_i8(z8, z, a8, a).shape == (0, 4) and sp.gemm_i8(a8, a, z8, z).shape == (4, 0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    b8, b = torch.ones(2, 4, 32, dtype=torch.int8, device="cuda"), torch.ones(2, 4, device="cuda")
    assert sp.moe_gemm_i8(z8, z, b8, b, off).shape == (0, 4)
    src = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    out = torch.full((6, 4), 5.0, device="cuda")
    sp.moe_gemm_i8(z8, z, b8, b, off + 6, src=src, slots=2, out=out)  # rows to fill, but A has none
    assert (out == 5).all()
    q, s = sp.quantize_rows_i8(torch.zeros(0, 7, device="cuda"))
    assert q.shape == (0, 7) and s.shape == (0,)


def test_beyond_32_bits():
    """Outputs and operands of more than 2^31 elements, and of more than 4 GB."""
    say("beyond 32 bits")
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 70000, 40000, 32  # 5.6 GB of bf16
    A = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    one = torch.ones(M, device="cuda")
    C = sp.gemm_i8(A, one, B, one[:N])
    rows = torch.tensor([0, 1, 53686, 53688, 69998, 69999], device="cuda")
    want = (A[rows].double() @ B.double().t()).to(torch.bfloat16)  # exact sums, one rounding
    assert torch.equal(C[rows], want)
    # the same values as rows to quantise, and as sorted rows of 80000 elements
    q, s = sp.quantize_rows_i8(C)
    x = C[rows].double()
    top = x.abs().amax(1)
    assert torch.equal(q[rows], torch.round(127 * x / top[:, None]).to(torch.int8))
    assert torch.equal(s[rows], (top.float() / 127))
    Ys = C.view(M // 2, 2 * N)
    pos = torch.randperm(M // 2, generator=g, device="cuda").to(torch.int32).view(-1, 2)
    w = torch.rand(pos.shape, generator=g, device="cuda")
    Y = sp.moe_combine(Ys, pos, w)
    t = torch.tensor([0, 9000, M // 4 - 1], device="cuda")
    terms = w[t].double().unsqueeze(-1) * Ys[pos[t].long()].double()
    ref, mag = terms.sum(1), terms.abs().sum(1)
    assert ((Y[t].double() - ref).abs() <= (2.0 ** -8) * (ref.abs() + 3 * U * mag) + 3 * U * mag).all()
    back = sp.moe_dispatch(Y, pos, out=Ys)  # over the rows they came from
    assert torch.equal(back[pos[t].long()], Y[t].unsqueeze(1).expand(-1, 2, -1))
    del C, q, Ys, Y, back, terms
    # 4.8 GB of expert weights
    E, F, H = 24, 8192, 24576
    W = torch.randint(-127, 128, (E, F, H), generator=g, device="cuda", dtype=torch.int8)
    X = torch.randint(-127, 128, (48, H), generator=g, device="cuda", dtype=torch.int8)
    off = torch.arange(0, 49, 2, device="cuda", dtype=torch.int32)
    out = sp.moe_gemm_i8(X, one[:48], W, torch.ones(E, F, device="cuda"), off, dtype=torch.float32)
    for e in (0, 10, 11, E - 1):
        want = X[2 * e:2 * e + 2].double() @ W[e].double().t()
        assert ((out[2 * e:2 * e + 2].double() - want).abs() <= 3.001 * U * want.abs()).all()


# T, slots, E, N, K, share routed nowhere, kind, gathered
EXPERTS = [(1, 1, 1, 16, 16, 0, "random", True), (1, 8, 64, 130, 256, 0, "random", True),
           (4, 2, 3, 33, 100, 0.3, "random", True), (32, 8, 64, 96, 512, 0, "random", True),
           (50, 2, 7, 64, 128, 0, "none", True), (300, 3, 4, 257, 192, 0.1, "skew", True),
           (700, 2, 5, 300, 320, 0, "one", True), (130, 4, 9, 128, 1111, 0.2, "random", True),
           (600, 1, 130, 70, 64, 0.1, "random", False), (2000, 2, 8, 272, 512, 0.1, "skew", False),
           (90, 3, 1024, 24, 48, 0, "random", True), (5, 2, 3, 8, 0, 0, "random", True),
           # the same for the experts: few rows each, 8 to 12, up to 48, up to 96, many
           (60, 4, 32, 700, 272, 0.1, "random", True), (50, 7, 32, 600, 272, 0, "skew", True),
           (100, 8, 32, 600, 144, 0.05, "random", True), (300, 8, 30, 1100, 300, 0.1, "skew", True),
           (2600, 2, 4, 1700, 130, 0.05, "random", True), (5300, 1, 3, 1800, 272, 0, "skew", False),
           # long sums with few rows each
           (60, 4, 32, 300, 2064, 0.1, "random", True), (100, 3, 30, 310, 2200, 0.1, "skew", True),
           (9, 2, 4, 1000, 4097, 0, "random", True)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("case", EXPERTS)
def test_expert_products(case, pad, dtype):
    say("expert products", case, pad, dtype)
    T, k, E, N, K, dropped, kind, gathered = case
    rng = rng_for(case)
    ids = route(rng, T, k, E, dropped, kind)
    offsets, src, _ = sort_ref(ids, E)
    S, R = T * k, T if gathered else T * k
    A, B = codes(rng, R, K), codes(rng, E * N, K)
    gap = 3 if pad == 1 else (-K) % 16
    sa = (rng.random(R) * 1e-2).astype(np.float32)
    sb = ((rng.random((E, N)) + 0.5) / (40 * np.sqrt(K + 1))).astype(np.float32)
    Bd = strided(B, gap)
    Bd = torch.as_strided(Bd, (E, N, K), (N * (K + gap), K + gap, 1), 0)
    buf, out = filled(S, N, dtype)
    sp.moe_gemm_i8(strided(A, gap), dev(sa), Bd, dev(sb), dev(offsets.astype(np.int32)),
                   src=dev(src.astype(np.int32)) if gathered else None, slots=k, out=out)
    live = int(offsets[-1])
    row = src[:live] // k if gathered else np.arange(live)
    e = np.repeat(np.arange(E), np.diff(offsets))
    sums = np.empty((live, N))
    for x in np.unique(e):
        at = e == x
        sums[at] = A[row[at]].astype(np.float64) @ B[x * N:(x + 1) * N].astype(np.float64).T
    product_close(out[:live], sums, sa[row], sb[e], dtype)
    assert (out[live:] == -7).all()


# M, N, K: few rows of many columns; 512 tiles of 32 x 64
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("M,N,K", [(13, 8300, 2100), (20, 8700, 2100), (32, 17000, 2064), (32, 17001, 130), (33, 9000, 2064),
                                   (250, 4100, 300), (513, 2040, 80)])
def test_product_of_few_rows(M, N, K, stride, dtype):
    test_product(M, N, K, stride, dtype)


# 8 to 16 rows an expert with long and short sums; many rows, several rounds of tiles on every XCD and a rest; one
# expert with nearly all; a few rows each of experts with many and with none
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("case", [(200, 2, 32, 330, 2100, 0, "random", True), (150, 2, 33, 333, 2065, 0.1, "random", True),
                                  (200, 2, 32, 330, 2000, 0, "random", True), (110, 2, 32, 500, 1000, 0.1, "random", True),
                                  (3000, 3, 6, 1300, 144, 0.02, "random", True), (9001, 1, 7, 1290, 129, 0, "skew", False),
                                  (700, 8, 90, 520, 100, 0, "skew", True), (1500, 4, 64, 600, 2050, 0, "skew", True),
                                  (12000, 1, 5, 300, 64, 0.1, "random", False)])
def test_expert_products_of_more_shapes(case, pad, dtype):
    test_expert_products(case, pad, dtype)


def test_strided_and_repeated_sources():
    """The same token for all rows of an expert, in both orders, and weights whose experts lie apart."""
    rng = rng_for("repeated")
    E, N, K, R, S = 5, 300, 2100, 3, 320
    A, B = codes(rng, R, K), codes(rng, E * N, K)
    whole = torch.zeros(E, N + 7, 2112, dtype=torch.int8, device="cuda")
    Bd = whole[:, 3:3 + N, :K]
    Bd.copy_(dev(B).view(E, N, K))
    sa, sb = (rng.random(R) + 0.5).astype(np.float32), (rng.random((E, N)) + 0.5).astype(np.float32)
    offsets = np.array([0, 0, 64, 65, 320, 320], np.int32)
    src = np.concatenate([np.full(64, 2), [0], np.sort(rng.integers(0, R, S - 65))[::-1]]).astype(np.int32)
    out = sp.moe_gemm_i8(strided(A, 12), dev(sa), Bd, dev(sb), dev(offsets), src=dev(src), dtype=torch.float32)
    e = np.repeat(np.arange(E), np.diff(offsets))
    sums = np.einsum("pk,pnk->pn", A[src].astype(np.float64), B.reshape(E, N, K)[e].astype(np.float64))
    product_close(out, sums, sa[src], sb[e], "f32")


def test_expert_products_with_bad_offsets_and_sources():
    """Nothing is validated on the device: out-of-range offsets are clamped, sources outside A are skipped."""
    rng = rng_for("bad")
    S, E, N, K, R = 40, 4, 48, 96, 10
    A, B = codes(rng, R, K), codes(rng, E * N, K)
    sa, sb = np.ones(R, np.float32), np.ones((E, N), np.float32)
    src = rng.integers(0, 2 * R, S)
    src[3], src[20], src[21] = -9, 2 * R, 2 ** 31 - 1
    offsets = np.array([-100, 12, 5, 25, 2 ** 31 - 1])  # expert 1's pair descends: empty
    buf, out = filled(S, N, "f32")
    sp.moe_gemm_i8(strided(A), dev(sa), dev(B).view(E, N, K), dev(sb),
                   dev(offsets.astype(np.int32)), src=dev(src.astype(np.int32)), slots=2, out=out)
    got = f64(out)
    # experts 0 and 2 both claim rows 5 .. 12; the others are one expert's
    for p in list(range(0, 5)) + list(range(12, S)):
        if src[p] < 0 or src[p] // 2 >= R:
            assert (got[p] == -7).all()
        else:
            x = 0 if p < 12 else 2 if p < 25 else 3
            np.testing.assert_array_equal(got[p], A[src[p] // 2].astype(np.float64) @ B[x * N:(x + 1) * N].T)


# ------------------------------------------------------------------ together
def _layer(x, ids, w, B1, s1, B2, s2, E, stream=None):
    """A mixture-of-experts layer served in int8: sort, quantise, first product on gathered rows, activation,
    quantise, second product, back."""
    k = ids.shape[1]
    offsets, src, pos = sp.moe_sort(ids, E, stream=stream)
    q, s = sp.quantize_rows_i8(x, stream=stream)
    h = sp.moe_gemm_i8(q, s, B1, s1, offsets, src=src, slots=k, stream=stream)
    h = torch.nn.functional.silu(h)
    q, s = sp.quantize_rows_i8(h, stream=stream)
    y = sp.moe_gemm_i8(q, s, B2, s2, offsets, stream=stream)
    return sp.moe_combine(y, pos, w, stream=stream)


def _layer_inputs(T, k, E, H, F, seed, dropped=0.1):
    rng = rng_for("layer", T, seed)
    ids = route(rng, T, k, E, dropped)
    w = rng.random((T, k)).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16).cuda()
    W1, W2 = (torch.from_numpy(rng.standard_normal((E, a, b)) / np.sqrt(b)).float().cuda() for a, b in ((F, H), (H, F)))
    q1, s1 = sp.quantize_rows_i8(W1.view(E * F, H))
    q2, s2 = sp.quantize_rows_i8(W2.view(E * H, F))
    return (x, dev(ids), dev(w), torch.as_strided(q1, (E, F, H), (F * q1.stride(0), q1.stride(0), 1)), s1.view(E, F),
            torch.as_strided(q2, (E, H, F), (H * q2.stride(0), q2.stride(0), 1)), s2.view(E, H), E), (ids, w, W1, W2)


@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 8, 256, 320), (37, 3, 6, 200, 130), (500, 2, 4, 512, 384)])
def test_layer(T, k, E, H, F):
    """The whole run against the same steps in 64 bits with real-valued weights and activations: what is left is the
    quantisation, half a step of 1 / 127 of the largest value at each of four operands."""
    say("layer", T, k, E, H, F)
    args, (ids, w, W1, W2) = _layer_inputs(T, k, E, H, F, 1)
    got = f64(_layer(*args))
    x, W1, W2 = f64(args[0]), f64(W1), f64(W2)
    ref = np.zeros((T, H))
    bound = np.zeros((T, H))
    step = lambda a: np.abs(a).max(-1, keepdims=True) / 254 * 1.001  # noqa: E731
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            h = W1[e] @ x[t]
            # |dh| from x's and W1's half steps, and bf16's rounding of h and of the activation (slope at most 1.1)
            dh = np.abs(W1[e]) @ np.full(H, step(x[t])[0]) + (np.abs(x[t]) + step(x[t])) @ (step(W1[e]) * np.ones(H)).T
            act = h / (1 + np.exp(-h))
            da = 1.1 * (dh + 2.0 ** -8 * (np.abs(h) + dh)) + 2.0 ** -8 * (np.abs(act) + 1.1 * dh)
            qa = da + (np.abs(act) + da).max() / 254 * 1.001
            y = W2[e] @ act
            dy = np.abs(W2[e]) @ qa + (step(W2[e]) * np.ones(F)) @ (np.abs(act) + qa)
            dy += 2.0 ** -8 * (np.abs(y) + dy)
            ref[t] += w[t, j] * y
            bound[t] += w[t, j] * dy
    bound += 2.0 ** -8 * (np.abs(ref) + bound) + 1e-6
    assert (np.abs(got - ref) <= bound).all()
    # and the errors are far below that bound on the whole: they add as random numbers do
    assert np.linalg.norm(got - ref) <= 0.1 * np.linalg.norm(bound) + 1e-6


def test_layer_in_a_graph():
    """Captured once, replayed with new contents of the inputs, eager work in between."""
    say("layer graph")
    args, _ = _layer_inputs(60, 4, 8, 256, 192, 2)
    x, ids, w = args[:3]
    _layer(*args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _layer(*args)
    rng = rng_for("graph")
    for n in range(4):
        ids.copy_(dev(route(rng, 60, 4, 8, 0.2 * n, "skew" if n % 2 else "random")))
        x.copy_(torch.from_numpy(rng.standard_normal((60, 256))).to(torch.bfloat16))
        want = _layer(*args)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), n


def test_long_sort_in_two_graphs():
    """Two captured sorts of the two-kernel size, each with scratch of its own, replayed in turn and at once."""
    say("sort graphs")
    E = 48
    rng = rng_for("two graphs")
    ids = [dev(route(rng, 9000 + 4000 * i, 2, E)) for i in range(2)]
    for i in ids:
        sp.moe_sort(i, E)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in ids:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sp.moe_sort(i, E))
        graphs.append(g)
    side = torch.cuda.Stream()
    for n in range(3):
        for i in ids:
            i.copy_(dev(route(rng, *i.shape, E, 0.1)))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for i, o in zip(ids, outs):
            for g, r in zip(o, sort_ref(i.cpu().numpy(), E)):
                np.testing.assert_array_equal(i64(g), r)


def test_backward_in_a_graph():
    say("backward graph")
    rng = rng_for("bwd graph")
    T, k, E, H = 50, 3, 6, 136
    _, src, pos = sort_ref(route(rng, T, k, E, 0.1), E)
    dpos, w = dev(pos.astype(np.int32)), dev(rng.random((T, k)).astype(np.float32))
    dY, Ys = rows_tensor(rng, T, H, "bf16"), rows_tensor(rng, T * k, H, "bf16")
    dYs, dXs = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(Ys)

    def step():
        sp.moe_dispatch(dY, dpos, out=dXs)
        a, b = sp.moe_combine_backward(dY, Ys, dpos, w, dYs=dYs)
        return a, b, sp.moe_combine(a, dpos), dXs

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for n in range(3):
        dY.copy_(rows_tensor(rng, T, H, "bf16"))
        want = [o.clone() for o in step()]
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert torch.equal(o, v)


def test_side_stream_and_two_streams_at_once():
    say("streams")
    a1, _ = _layer_inputs(40, 2, 4, 256, 128, 3)
    a2, _ = _layer_inputs(90, 2, 4, 256, 128, 4)
    want1, want2 = _layer(*a1).clone(), _layer(*a2).clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for n in range(5):
        with torch.cuda.stream(s1):
            o1 = _layer(*a1, stream=s1)
        with torch.cuda.stream(s2):
            o2 = _layer(*a2, stream=s2)
        outs.append((o1, o2))
    torch.cuda.synchronize()
    for o1, o2 in outs:
        assert torch.equal(o1, want1) and torch.equal(o2, want2)


def test_binding_refusals():
    say("refusals")
    pos = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    q = torch.zeros(4, 16, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    off = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [lambda: sp.moe_sort(pos.t(), 4),                                    # not contiguous
           lambda: sp.moe_dispatch(x.t(), pos),                                # last dimension strided
           lambda: sp.moe_dispatch(x[:1].expand(4, 16), pos),                  # rows that overlap
           lambda: sp.moe_dispatch(x, pos[:3]),
           lambda: sp.moe_dispatch(x, pos, out=x),                             # overlap
           lambda: sp.moe_dispatch(x, pos, out=torch.zeros(8, 17, device="cuda")),
           lambda: sp.moe_dispatch(x, pos[:, :0]),                             # no slots
           lambda: sp.moe_combine(x, pos, w[:3]),
           lambda: sp.moe_combine(x, pos, w, out=torch.zeros(3, 16, device="cuda")),
           lambda: sp.moe_combine_backward(x, x, pos, w, dYs=x),
           lambda: sp.moe_combine_backward(x[:3], x, pos, w),
           lambda: sp.quantize_rows_i8(x, q=q[:, :8]),
           lambda: sp.quantize_rows_i8(x, scale=s[:3]),
           lambda: sp.gemm_i8(q, s[:3], q, s),
           lambda: sp.gemm_i8(q, s, q[:, :8], s),
           lambda: sp.gemm_i8(q, s, q, s, out=torch.zeros(4, 5, device="cuda")),
           lambda: sp.moe_gemm_i8(q, s, q[None], s[None], off[:1]),
           lambda: sp.moe_gemm_i8(q, s, q[None].expand(2, 4, 16), s[None].expand(2, 4).contiguous(),
                                  torch.zeros(3, dtype=torch.int32, device="cuda"), slots=0)]
    for n, call in enumerate(bad):
        with pytest.raises((ValueError, sp.SparseError)):
            call()
            pytest.fail("call %d was taken" % n)
    with pytest.raises(TypeError):
        sp.moe_combine(x, pos, w.half())
    with pytest.raises(TypeError):
        sp.gemm_i8(q, s, q, s, dtype=torch.int32)
    with pytest.raises(sp.SparseError) as e:
        sp.moe_sort(pos, 2000)
    assert e.value.code == 5

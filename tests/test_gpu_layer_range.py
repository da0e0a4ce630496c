"""The norm and the gated gradient at the ends of their types' ranges on the GPU, against their definitions in 64 bits.

Tolerances as in test_gpu_layer.py: u = 2^-24 is fp32's rounding, half a step of the output's type, and steps_of(H) of a sum.
"""
import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say
from test_gpu_layer import SIXTEEN, check, norm_backward_ref, norm_ref, steps_of
from test_gpu_moe import HALF, LEAST, TYPES, U, f64, i64, rng_for

pytestmark = pytest.mark.gpu

LENGTHS = [40, 600, 2500, 9001]


def tensor(a, dtype):
    return torch.from_numpy(np.asarray(a)).to(TYPES[dtype]).cuda()


# ------------------------------------------------------------------ gated gradient
def saturated(g, act):
    """a(g) and a'(g) of |g| up to the type's largest: their limits where exp(-|p|) is below 2^-1000."""
    c = 2 * np.sqrt(2 / np.pi)
    m = np.clip(g, -800, 800) if act == "silu" else np.clip(g, -100, 100)
    p, dp = (m, np.ones_like(m)) if act == "silu" else (c * (m + 0.044715 * m ** 3), c * (1 + 3 * 0.044715 * m * m))
    with np.errstate(over="ignore"):
        sig = 1 / (1 + np.exp(-p))
    far = np.abs(p) > 700
    a = np.where(far, np.where(g > 0, g, 0), m * sig)
    da = np.where(far, g > 0, sig * (1 + m * dp * (1 - sig)))
    rough = np.where(far, da, sig * (1 + np.abs(m * dp)))  # without the cancellation in a'
    return a, da, rough, np.where(far, 0, np.abs(p))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", SIXTEEN)
def test_gated_backward_of_far_pre_activations(dtype, act):
    """Up to the type's largest, where the derivative's factors leave fp32's range though the derivative does not."""
    say("far pre-activations", dtype, act)
    far = [2e4, 6e4] if dtype == "f16" else [1e13, 2e13, 1e14, 1.8e19, 1e20, 1e30, 3e38]
    values = np.array([0, 0.5, 3, 9, 15, 40, 88, 90, 120, 1e3] + far)
    values = np.concatenate([values, -values])
    N = values.size
    rng = rng_for("far pre", dtype, act)
    S = 9
    pre = tensor(np.concatenate([np.tile(values, (S, 1)), rng.standard_normal((S, N))], 1), dtype)
    dH = tensor(rng.uniform(0.25, 0.5, (S, N)) * rng.choice([-1, 1], (S, N)), dtype)
    one = torch.eye(2 * N, dtype=TYPES[dtype], device="cuda")
    dA, dB = sp.moe_gated_backward(dH, pre, one[:S], one, act=act)
    g, u, d = f64(pre)[:, :N], f64(pre)[:, N:], f64(dH)
    a, da, rough, p = saturated(g, act)
    want = np.concatenate([d * u * da, d * a], 1)
    rough = np.concatenate([np.abs(d * u) * rough, np.abs(d * a)], 1)
    # sig is off by u (4 + 4 |p|) of itself, as is 1 - sig; products with the unit matrix are exact.  Below fp32's normal
    # range exp may be 0: at most 2^-126 times the other factors, which are below 2^8 there
    off = rough * U * (16 + 8 * np.concatenate([p, p], 1)) + 2.0 ** -110
    check(dA, want, off + HALF[dtype] * (np.abs(want) + off) + LEAST[dtype], (dtype, act))
    assert torch.equal(dB.t()[:S], dA)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward_of_pre_activations_beyond_fp16(act):
    """A gate's sum that fp16 cannot hold is kept as an Inf; below, the product and its gradient are 0."""
    S, N, K = 5, 8, 64
    A = torch.full((S, K), 64.0, dtype=torch.float16, device="cuda")
    B = torch.full((2 * N, K), 1 / 64, dtype=torch.float16, device="cuda")
    B[:3] = -64.0  # sums of -2^18
    B[5] = 64.0  # and 2^18
    B[N + 5] = 2.0 ** -14
    pre = torch.empty(S, 2 * N, dtype=torch.float16, device="cuda")
    out = sp.moe_gated(A, B, act=act, pre=pre)
    assert bool((pre[:, :3] == -float("inf")).all()) and bool((pre[:, 5] == float("inf")).all())
    assert bool((out[:, :3] == 0).all())
    dH = torch.full((S, N), 0.5, dtype=torch.float16, device="cuda")
    for columns in (slice(0, 5), slice(6, 8)):
        rows = list(range(N))[columns] + list(range(N, 2 * N))[columns]
        dA, dB = sp.moe_gated_backward(dH[:, columns].contiguous(), pre[:, rows].contiguous(), A, B[rows].contiguous(), act=act)
        assert bool(torch.isfinite(dA).all()) and bool(torch.isfinite(dB).all())
        if columns.start == 0:
            assert not dB[:3].any() and not dB[5:8].any()
    # a'(Inf) = 1: the gate's own gradient is dH u
    dP = sp.moe_gated_backward(dH[:, 5:6].contiguous(), pre[:, [5, 13]].contiguous(), torch.ones(S, 1, dtype=torch.float16, device="cuda"),
                               torch.ones(2, 1, dtype=torch.float16, device="cuda"), act=act, dA=None)[1]
    assert float(dP[0, 0]) == S * 0.5 * float(pre[0, 13]) and float(dP[1, 0]) == float("inf")


# ------------------------------------------------------------------ norm
def weights_of(rng, H, scale):
    return tensor((1 + 0.2 * rng.standard_normal(H)) * scale, "f32")


def check_norm(x, w, eps, dtype, what):
    s64, w64, i = norm_ref(x, w, eps)
    y = s64 * i * w64
    check(sp.rms_norm(x, w, eps=eps), y, np.abs(y) * (HALF[dtype] + (0.5 * steps_of(x.shape[1]) + 8) * U) + LEAST[dtype], what)


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_large_rows_under_large_weights(dtype, H):
    """s weight leaves the range, the norm does not."""
    say("norm, large rows and weights", dtype, H)
    rng = rng_for("large", dtype, H)
    x = tensor(rng.standard_normal((5, H)) * np.array([2.0 ** 55, 1, 2.0 ** 100, 2.0 ** -40, 2.0 ** 57])[:, None], dtype)
    for scale in (2.0 ** 75, 2.0 ** 110, 2.0 ** -100):
        check_norm(x, weights_of(rng, H, scale), 1e-6, dtype, (dtype, H, scale))


def check_codes(x, w, eps, what):
    """The codes are those of y = s i weight: four roundings and a sum's, a quotient and a product, then half a code; a row
    below 2^-119 is zeros."""
    say("norm int8", what)
    q, scale = sp.rms_norm_i8(x, w, eps=eps)
    s64, w64, i = norm_ref(x, w, eps)
    y = s64 * i * w64
    a = np.abs(y).max(1)
    off = (0.5 * steps_of(x.shape[1]) + 10) * U
    live = a >= 2.0 ** -119
    assert (np.abs(f64(scale) - np.where(live, a / 127, 0)) <= off * a / 127).all(), (what, f64(scale), a / 127)
    # a row's i is in all its values alike
    assert (np.abs(i64(q) - 127 * y / np.where(live, a, np.inf)[:, None]) <= np.where(live, 0.5 + 127 * 8 * U, 0)[:, None]).all(), what


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_into_int8_under_large_weights(dtype, H):
    """s weight is beyond 2^120 where the sum of squares is an ordinary one, and the other way round."""
    rng = rng_for("codes, large", dtype, H)
    x = tensor(rng.standard_normal((5, H)) * np.array([1, 2.0 ** 55, 2.0 ** -20, 2.0 ** 100, 30])[:, None], dtype)
    for scale in (2.0 ** 119, 2.0 ** 121, 2.0 ** 123, 2.0 ** 75, 2.0 ** -60):
        check_codes(x, weights_of(rng, H, scale), 1e-6 if scale > 1e36 else 0.0, (dtype, H, scale))
    y, scale = sp.rms_norm_i8(torch.ones(3, H, device="cuda"), torch.full((H,), 2.0 ** 121, device="cuda"), eps=0.0)
    assert bool((y == 127).all()) and torch.allclose(scale, torch.full_like(scale, 2.0 ** 121 / 127), rtol=4 * U)


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_into_int8_of_tiny_rows(dtype, H):
    """s weight is below fp32's normal range, or its reciprocal above it; the norm is ordinary."""
    rng = rng_for("codes, tiny", dtype, H)
    base = rng.uniform(1, 2, (4, H)) * rng.choice([-1, 1], (4, H))
    for eps, size, scale in ((1e-6, 9e-40, 1), (1e-12, 9e-40, 1), (1e-12, 2.0 ** -135, 1), (1e-9, 4e-39, 1), (1e-6, 1e-10, 2.0 ** -95),
                             (1e-6, 2.0 ** -60, 2.0 ** -66)):
        check_codes(tensor(base * size, dtype), tensor(rng.uniform(0.9, 1.1, H) * scale, "f32"), eps, (dtype, H, eps, size, scale))
    x = tensor(base, dtype)
    x[1] = 0
    x[2] = tensor(base[2] * 1e-38, dtype)
    q, scale = sp.rms_norm_i8(x, eps=1.0)  # a row whose scale would be denormal is zeros
    assert not scale[1:3].any() and not q[1:3].any() and bool((scale[[0, 3]] > 0).all())


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_small_rows_without_eps(dtype, H):
    """Sums of squares on both sides of where a row is summed again from scaled values."""
    rng = rng_for("small", dtype, H)
    logs = np.array([-50, -59.5, -60.5, -61, -62, -63, -63.9, -64.5, -66, -80, -120, -200])  # of the sum of squares
    x = rng.standard_normal((logs.size, H))
    x = tensor(x * np.sqrt(2.0 ** logs / (x * x).sum(1))[:, None], dtype)
    w, dy = weights_of(rng, H, 1), tensor(rng.standard_normal(x.shape), dtype)
    for eps in (0.0, 1e-35):
        check_norm(x, w, eps, dtype, (dtype, H, eps))
        check_codes(x, w, eps, (dtype, H, eps))
        dx, dw = sp.rms_norm_backward(dy, x, w, eps=eps)
        d, bound, dwr, dwb = norm_backward_ref(x, w, dy, None, dtype, eps)
        check(dx, d, bound, (dtype, H, eps))
        check(dw, dwr, dwb, (dtype, H, eps))


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_backward_of_large_rows(dtype, H):
    """dy weight s leaves the range, and so does its sum; the gradient does not."""
    rng = rng_for("large gradient", dtype, H)
    s = tensor(rng.standard_normal((5, H)) * np.array([2.0 ** 55, 1, 2.0 ** 57, 2.0 ** 30, 2.0 ** 100])[:, None], dtype)
    dy = tensor(rng.standard_normal((5, H)) * np.array([2.0 ** 75, 2.0 ** 100, 2.0 ** 80, 2.0 ** 112, 2.0 ** 60])[:, None], dtype)
    w = weights_of(rng, H, 1)
    dx, dw = sp.rms_norm_backward(dy, s, w, eps=1e-6)
    want, bound, dwr, dwb = norm_backward_ref(s, w, dy, None, dtype, 1e-6)
    check(dx, want, bound, (dtype, H))
    check(dw, dwr, dwb, (dtype, H))


@pytest.mark.parametrize("H", [8, 40, 128, 600, 2500, 9001])
def test_equal_values_of_a_row_have_equal_norms(H):
    """Wherever in a row a value stands, and wherever the row: one rounding to fp32, then one to fp16."""
    say("equal values", H)
    rows = 40000 if H < 1000 else 8000
    v = tensor(rng_for("equal", H).standard_normal(rows), "f16")
    x = v[:, None].expand(rows, H).contiguous()
    beside = torch.empty(rows, H + 1, dtype=torch.float16, device="cuda")[:, :H]  # rows that do not lie on lines
    beside.copy_(x)
    for w in (None, torch.full((H,), 1.2345, device="cuda"), torch.full((H,), 1.2345, dtype=torch.float16, device="cuda")):
        for call in (lambda x: sp.rms_norm(x, w, eps=1.0), lambda x: sp.rms_norm(x, w, residual=x, eps=1.0)[0],
                     lambda x: sp.rms_norm_backward(x, x, w, eps=1.0)[0], lambda x: sp.rms_norm_backward(x, x, w, dsum=x, eps=1.0)[0]):
            y = call(x)
            assert torch.equal(y, y[:, :1].expand(rows, H)) and torch.equal(call(beside), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_into_int8_of_the_largest_rows_under_large_weights(dtype):
    """1 / rms is near fp32's smallest normal numbers, and the norm near the largest."""
    for H in LENGTHS:
        rng = rng_for("codes, largest", dtype, H)
        x = tensor(rng.uniform(0.25, 1, (6, H)) * rng.choice([-1, 1], (6, H)) * 2.0 ** np.array([127, 126, 125, 120, 118, 110])[:, None], dtype)
        for scale in (2.0 ** 118, 2.0 ** 121, 2.0 ** 125):
            check_codes(x, tensor(rng.uniform(0.9, 1.1, H) * scale, "f32"), 0.0, (dtype, H, scale))

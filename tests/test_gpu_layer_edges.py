"""The norm, the gated products and the experts' products in 16 bits beyond small operands: every kind of tile and cut,
rows beyond 32 bits, workspaces and graphs, operands of other streams, and what the binding refuses on device tensors."""
import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say
from test_gpu_layer import (SIXTEEN, act_ref, backward_ref, check, experts, gated_ref, gradient_buffers, norm_backward_ref,
                            norm_inputs, products_inputs, sums_ref)
from test_gpu_moe import HALF, LEAST, TYPES, U, dev, f64, filled, rng_for, route, rows_tensor, sort_ref
from test_gpu_moe_edges import busy

pytestmark = pytest.mark.gpu

# T, slots, E (0: one matrix), N, K, dropped, kind: few and many tiles of every height, short and long sums, experts of
# few, uneven and many rows, one slot a token
LARGE = [(16, 1, 0, 4400, 136, 0, "random"), (16, 1, 0, 11400, 72, 0, "random"), (100, 1, 0, 11400, 40, 0, "random"),
         (100, 1, 0, 1200, 136, 0, "random"), (300, 1, 0, 1600, 136, 0, "random"),
         (300, 1, 0, 2900, 136, 0, "random"), (2200, 1, 0, 2200, 72, 0, "random"), (3000, 1, 0, 3000, 72, 0, "random"),
         (4000, 1, 0, 40, 72, 0, "random"), (20, 1, 0, 1400, 304, 0, "random"), (28, 1, 0, 2100, 1104, 0, "random"),
         (2600, 1, 0, 136, 2600, 0, "random"), (700, 2, 5, 520, 264, 0.1, "skew"), (1500, 4, 6, 1100, 200, 0.05, "random"),
         (64, 8, 32, 704, 160, 0, "random"), (1500, 1, 3, 264, 1032, 0.1, "random"), (3000, 1, 2, 72, 136, 0, "skew")]
# long sums of dA in parts: of experts, and of so many tiles that there are two parts' a CU
CUTS = [(100, 2, 3, 2400, 136, 0, "random"), (1152, 1, 0, 7040, 1920, 0, "random")]
PLACES = [(0, 0), (8, 0), (13, 5)]  # gap between rows, first element's offset


@pytest.mark.parametrize("layout", PLACES)
@pytest.mark.parametrize("dtype", SIXTEEN)
@pytest.mark.parametrize("case", LARGE + CUTS)
def test_products_of_every_tile(case, dtype, layout):
    say("large", case, dtype, layout)
    rng, S, A, B, offsets, token, args = products_inputs(case, dtype, layout, False, bool(case[2]))
    N = case[3]
    buf, C = filled(S, N, dtype, *layout)
    sp.moe_gemm(A, B, out=C, **args)
    want, bound = np.full((S, N), -7.0), np.zeros((S, N))
    for mine, b in experts(offsets, B):
        y, e = sums_ref(f64(A)[token[mine]], f64(b).T)
        want[mine], bound[mine] = y, e + HALF[dtype] * (np.abs(y) + e) + LEAST[dtype]
    check(C, want, bound, case)
    C.fill_(-7.0)
    assert bool((buf == -7.0).all())
    dC = rows_tensor(rng, S, N, dtype, *layout)
    dC[offsets[-1]:] = float("nan")
    buf, dA, bbuf, dB = gradient_buffers(S, A, B, dtype, layout)
    sp.moe_gemm_backward(dC, A, B, dA=dA, dB=dB, **args)
    wa, ba, wb, bb = backward_ref(f64(dC), np.zeros(dC.shape), A, B, offsets, token, dtype)
    check(dA, wa, ba, case)
    check(dB, wb, bb, case)
    dA.fill_(-7.0), dB.fill_(-7.0)
    assert bool((buf == -7.0).all()) and bool((bbuf == -7.0).all())


@pytest.mark.parametrize("layout", PLACES)
@pytest.mark.parametrize("case", LARGE)
def test_gated_products_of_every_tile(case, layout):
    dtype = SIXTEEN[case[3] // 8 % 2]
    say("large gated", case, dtype, layout)
    _, S, A, B, offsets, token, args = products_inputs(case, dtype, layout, True, bool(case[2]))
    N = case[3]
    _, C = filled(S, N, dtype, *layout)
    _, pre = filled(S, 2 * N, dtype, *layout)
    sp.moe_gated(A, B, act="gelu_tanh", pre=pre, out=C, **args)
    h, hb = np.full((S, N), -7.0), np.zeros((S, N))
    y, yb = np.full((S, 2 * N), -7.0), np.zeros((S, 2 * N))
    for mine, b in experts(offsets, B):
        p, e = sums_ref(f64(A)[token[mine]], f64(b).T)
        y[mine], yb[mine] = p, e + HALF[dtype] * (np.abs(p) + e) + LEAST[dtype]
        h[mine], hb[mine] = gated_ref(p[:, :N], p[:, N:], e[:, :N], e[:, N:], "gelu_tanh", HALF[dtype], LEAST[dtype])
    check(C, h, hb, case)
    check(pre, y, yb, case)
    dH = rows_tensor(rng_for("dH", case), S, N, dtype, *layout)
    dA, dB = sp.moe_gated_backward(dH, pre, A, B, act="gelu_tanh", **args)
    g, u, d = f64(pre)[:, :N], f64(pre)[:, N:], f64(dH)
    sig, p, dp = act_ref(g, "gelu_tanh")
    dpre = np.concatenate([d * u * sig * (1 + g * dp * (1 - sig)), d * g * sig], 1)
    rough = np.concatenate([np.abs(d * u) * sig * (1 + np.abs(g * dp)), np.abs(d * g * sig)], 1)
    off = rough * U * (16 + 8 * np.abs(np.concatenate([p, p], 1)))
    off = off + HALF[dtype] * (np.abs(dpre) + off) + LEAST[dtype]
    wa, ba, wb, bb = backward_ref(dpre, off, A, B, offsets, token, dtype)
    check(dA[:offsets[-1]], wa[:offsets[-1]], ba[:offsets[-1]], case)
    check(dB, wb, bb, case)


# M, N, K of gated int8 products that take every kind of tile
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("M,N,K", [(40, 3000, 256), (120, 700, 128), (300, 900, 128), (300, 1500, 256), (1200, 2100, 128),
                                   (2500, 1500, 128), (90, 400, 3000)])
def test_gated_int8_of_every_tile(M, N, K, aligned):
    say("large gated int8", M, N, K, aligned)
    rng = rng_for(M, N, K)
    pad = 0 if aligned else 7
    codes = lambda *s: dev(rng.integers(-127, 128, s).astype(np.int8))[:, :K]  # noqa: E731
    A, B = codes(M, K + pad), codes(2 * N, K + pad)
    sa, sb = dev((rng.random(M) * 0.02 + 0.01).astype(np.float32)), dev((rng.random(2 * N) * 0.03 / np.sqrt(K)).astype(np.float32))
    y = (f64(A) @ f64(B).T) * f64(sa)[:, None] * f64(sb)  # whole numbers below 2^53: exact
    h, bound = gated_ref(y[:, :N], y[:, N:], 3.1 * U * np.abs(y[:, :N]), 3.1 * U * np.abs(y[:, N:]), "silu", HALF["bf16"], LEAST["bf16"])
    check(sp.gated_i8(A, sa, B, sb), h, bound, (M, N, K))


def test_gated_gradient_of_offsets_that_descend():
    """An expert's rows may lie behind the last offset."""
    rng = rng_for("descend")
    S, N, K = 60, 24, 40
    A, B, dH = rows_tensor(rng, S, K, "bf16"), rows_tensor(rng, 3 * 2 * N, K, "bf16").reshape(3, 2 * N, K), rows_tensor(rng, S, N, "bf16")
    pre = rows_tensor(rng, S, 2 * N, "bf16")
    o = torch.tensor([0, 50, 20, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # 0 .. 50, none, 20 .. 60
    _, dB = sp.moe_gated_backward(dH, pre, A, B, o, dA=None)
    for e, rows in enumerate((slice(0, 50), slice(0, 0), slice(20, 60))):
        _, want = sp.moe_gated_backward(dH[rows].contiguous(), pre[rows].contiguous(), A[rows].contiguous(), B[e], dA=None)
        assert torch.allclose(dB[e].float(), want.float(), rtol=4 * HALF["bf16"], atol=1e-5)  # two roundings, sums in other orders
    o = torch.tensor([0, 50, 20, 20], dtype=torch.int32, device="cuda")
    dA, _ = sp.moe_gated_backward(dH, pre, A, B, o, dB=None)
    want, _ = sp.moe_gated_backward(dH[:50].contiguous(), pre[:50].contiguous(), A[:50].contiguous(), B[0], dB=None)
    assert torch.allclose(dA[:50].float(), want.float(), rtol=4 * HALF["bf16"], atol=1e-5)


def test_the_same_source_again():
    """Many rows that read one token's."""
    rng = rng_for("again")
    S, N, K = 300, 40, 72
    A, B, dC = rows_tensor(rng, 5, K, "bf16"), rows_tensor(rng, N, K, "bf16"), rows_tensor(rng, S, N, "bf16")
    o, src = torch.tensor([0, S], dtype=torch.int32, device="cuda"), torch.full((S,), 7, dtype=torch.int32, device="cuda")
    copies = A[3:4].expand(S, K).contiguous()
    assert torch.equal(sp.moe_gemm(A, B[None], o, src=src, slots=2), sp.moe_gemm(copies, B[None], o))
    for got, want in zip(sp.moe_gemm_backward(dC, A, B[None], o, src=src, slots=2), sp.moe_gemm_backward(dC, copies, B[None], o)):
        assert torch.equal(got, want)


# ------------------------------------------------------------------ beyond 32 bits
def test_rows_far_apart():
    """Rows whose distances pass 2^31 elements and 2^32 bytes from the first to the last."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    S, K, N, far = 40, 72, 24, (1 << 26) + 8
    rng = rng_for("far")
    buf = torch.zeros(S * far, dtype=torch.bfloat16, device="cuda")

    def spread(rows, cols, at):
        t = torch.as_strided(buf, (rows, cols), (far, 1), at)
        t.copy_(torch.from_numpy(rng.standard_normal((rows, cols))))
        return t

    A, B, dC = spread(S, K, 0), spread(N, K, 80), spread(S, N, 160)
    near = [t.contiguous() for t in (A, B, dC)]
    say("far rows")
    assert torch.equal(sp.moe_gemm(A, B), sp.moe_gemm(near[0], near[1]))
    for got, want in zip(sp.moe_gemm_backward(dC, A, B, dA=torch.as_strided(buf, (S, K), (far, 1), 240),
                                              dB=torch.as_strided(buf, (N, K), (far, 1), 320)),
                         sp.moe_gemm_backward(near[2], near[0], near[1])):
        assert torch.equal(got, want)
    out = torch.as_strided(buf, (S, K), (far, 1), 400)
    y, s = sp.rms_norm(A, residual=A, out=out)
    want = sp.rms_norm(near[0], residual=near[0])
    assert torch.equal(y, want[0]) and torch.equal(s, want[1])
    w = torch.ones(K, device="cuda")
    for got, want in zip(sp.rms_norm_backward(A, A, w, dsum=A, dx=out), sp.rms_norm_backward(near[0], near[0], w, dsum=near[0])):
        assert torch.equal(got, want)


def test_many_short_rows():
    """More rows than a launch has workgroups, and a norm of more than 2^31 values."""
    rows, H = (1 << 25) + 3, 72
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    say("many rows")
    x = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    x[-5:] = torch.arange(H, device="cuda") - 30
    y = sp.rms_norm(x, eps=1.0)
    assert not y[:-5].any() and torch.equal(y[-1], sp.rms_norm(x[-1:], eps=1.0)[0])
    dx, dw = sp.rms_norm_backward(x, x, torch.ones(H, device="cuda"), eps=1.0)
    want = sp.rms_norm_backward(x[-5:], x[-5:], torch.ones(H, device="cuda"), eps=1.0)
    assert torch.equal(dx[-5:], want[0]) and torch.allclose(dw, want[1], rtol=8 * U)  # five rows, added in another order


# ------------------------------------------------------------------ long rows of the norm
@pytest.mark.parametrize("rows,H", [(3, 4104), (2, 8193), (700, 4100), (37, 16384), (5, 40000)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_norm_backward_of_long_rows(rows, H, dtype):
    say("long rows", rows, H, dtype)
    rng = rng_for(rows, H, dtype)
    s, dsum, w, _ = norm_inputs(rng, rows, H, dtype, "f32", True, (0, 0))
    dy = rows_tensor(rng, rows, H, dtype)
    dx, dw = sp.rms_norm_backward(dy, s, w, eps=1e-5, dsum=dsum)
    want, bound, dwr, dwb = norm_backward_ref(s, w, dy, dsum, dtype)
    check(dx, want, bound, (rows, H))
    check(dw, dwr, dwb, (rows, H))


# ------------------------------------------------------------------ workspaces, graphs, streams
def layer_inputs(seed):
    rng = rng_for("layer", seed)
    T, k, E, N, K = 90, 2, 4, 104, 136
    offsets, src, pos = sort_ref(route(rng, T, k, E), E)
    o, s = dev(offsets.astype(np.int32)), dev(src.astype(np.int32))
    return (rows_tensor(rng, T * k, N, "bf16"), rows_tensor(rng, T * k, 2 * N, "bf16"), rows_tensor(rng, T, K, "bf16"),
            rows_tensor(rng, E * 2 * N, K, "bf16").reshape(E, 2 * N, K), o, s, k)


def test_two_graphs_that_share_a_workspace():
    """Replayed in turn, with eager calls between: what one leaves in the workspace does not reach the other."""
    dH, pre, A, B, o, s, k = layer_inputs(1)
    x, w = rows_tensor(rng_for("shared"), 300, 264, "f32"), torch.ones(264, device="cuda")
    work = torch.full((8 << 20,), 255, dtype=torch.uint8, device="cuda")
    one = lambda: sp.moe_gated_backward(dH, pre, A, B, o, src=s, slots=k, work=work)  # noqa: E731
    two = lambda: sp.rms_norm_backward(x, x, w, work=work)  # noqa: E731
    want = [[t.clone() for t in f()] for f in (one, two)]
    torch.cuda.synchronize()
    graphs, static = [], []
    for f in (one, two):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            static.append(f())
    for _ in range(3):
        for g, got, ref in zip(graphs, static, want):
            for t in got:
                t.fill_(-7.0)
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
        two(), one()


def test_operands_of_a_side_stream_call_are_kept():
    """Memory of an operand that is dropped right after a call on a side stream is not handed out before the call has
    read it."""
    say("kept operands")
    dH, pre, A, B, o, s, k = layer_inputs(2)
    want = sp.moe_gated_backward(dH, pre, A, B, o, src=s, slots=k)
    x = rows_tensor(rng_for("kept"), 500, 520, "bf16")
    norm = sp.rms_norm(x, x[0].clone(), residual=x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy(side)
    args = [t.clone() for t in (dH, pre, A, B, o, s)]
    rows = [x.clone(), x[0].clone(), x.clone()]
    torch.cuda.current_stream().synchronize()
    got = sp.moe_gated_backward(*args[:5], src=args[5], slots=k, stream=side)
    got += sp.rms_norm(rows[0], rows[1], residual=rows[2], stream=side)
    sizes = [t.numel() * t.element_size() for t in args + rows]
    del args, rows
    for n in sizes:  # would take their memory
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want + norm))


def test_two_streams_at_once():
    """The same operands on two streams, each call with a workspace of its own."""
    dH, pre, A, B, o, s, k = layer_inputs(3)
    want = sp.moe_gated_backward(dH, pre, A, B, o, src=s, slots=k)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [sp.moe_gated_backward(dH, pre, A, B, o, src=s, slots=k, stream=t) for t in streams]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


# ------------------------------------------------------------------ what the binding refuses
def test_refused_operands():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    x, w, A, B = z(6, 16), z(16), z(6, 16), z(10, 16)
    o = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    pre, dH = z(6, 10), z(6, 5)
    q, s = z(6, 16, dtype=torch.int8), z(6, dtype=torch.float32)
    half = z(6, 32)
    for error, call in [
            (ValueError, lambda: sp.rms_norm(x, z(15))), (TypeError, lambda: sp.rms_norm(x, z(16, dtype=torch.float16))),
            (ValueError, lambda: sp.rms_norm(x, residual=z(5, 16))), (TypeError, lambda: sp.rms_norm(x, residual=z(6, 16, dtype=torch.float16))),
            (ValueError, lambda: sp.rms_norm(x, w, out=x)), (ValueError, lambda: sp.rms_norm(x, w, sum_out=z(6, 16))),
            (ValueError, lambda: sp.rms_norm(x, w, residual=z(6, 16), out=x)),
            (ValueError, lambda: sp.rms_norm(half[:, :16], w, residual=z(6, 16), sum_out=half[:, 1:17])),
            (ValueError, lambda: sp.rms_norm(x.t())), (ValueError, lambda: sp.rms_norm_i8(x, q=z(6, 15, dtype=torch.int8))),
            (ValueError, lambda: sp.rms_norm_i8(x, scale=z(5, dtype=torch.float32))),
            (ValueError, lambda: sp.rms_norm_backward(x, x, w, dx=x)), (ValueError, lambda: sp.rms_norm_backward(x, x, dweight=z(16, dtype=torch.float32))),
            (ValueError, lambda: sp.rms_norm_backward(z(6, 15), x, w)), (ValueError, lambda: sp.rms_norm_backward(x, z(6, 16), w, work=x.view(torch.uint8))),
            (ValueError, lambda: sp.gated_i8(q, s, z(11, 16, dtype=torch.int8), z(11, dtype=torch.float32))),
            (ValueError, lambda: sp.gated_i8(q, s, z(10, 16, dtype=torch.int8), z(10, dtype=torch.float32), act="relu")),
            (ValueError, lambda: sp.moe_gated_i8(q, s, z(1, 10, 16, dtype=torch.int8), z(1, 9, dtype=torch.float32), o)),
            (ValueError, lambda: sp.moe_gemm(A, z(10, 15))), (ValueError, lambda: sp.moe_gemm(A, z(10, 16)[None])),
            (TypeError, lambda: sp.moe_gemm(A, z(10, 16, dtype=torch.float16))), (ValueError, lambda: sp.moe_gemm(A, z(2, 10, 16), o)),
            (TypeError, lambda: sp.moe_gemm(A, B[None], o.long())), (ValueError, lambda: sp.moe_gemm(A, B, out=z(6, 9))),
            (ValueError, lambda: sp.moe_gemm(A, A, out=A[:, :6])), (ValueError, lambda: sp.moe_gated(A, z(11, 16))),
            (ValueError, lambda: sp.moe_gated(A, B, act="relu")), (ValueError, lambda: sp.moe_gated(A, B, pre=z(6, 5))),
            (ValueError, lambda: sp.moe_gated(A, B, pre=half[:, :10], out=half[:, 5:10])),
            (ValueError, lambda: sp.moe_gemm_backward(z(6, 9), A, B)), (ValueError, lambda: sp.moe_gemm_backward(pre, A, B, dA=A)),
            (ValueError, lambda: sp.moe_gemm_backward(pre, A, B, dB=z(10, 15))), (ValueError, lambda: sp.moe_gemm_backward(pre, A, B, dB=B)),
            (ValueError, lambda: sp.moe_gated_backward(dH, z(6, 9), A, B)), (ValueError, lambda: sp.moe_gated_backward(z(6, 4), pre, A, B)),
            (ValueError, lambda: sp.moe_gated_backward(dH, pre, A, B, work=pre.view(torch.uint8)))]:
        with pytest.raises(error):
            call()
    for call in (lambda: sp.moe_gemm(A, B, slots=0, src=z(6, dtype=torch.int32)), lambda: sp.rms_norm(x, eps=-1.0),
                 lambda: sp.rms_norm(x, eps=float("nan")), lambda: sp.moe_gated_backward(dH, pre, A, B, work=z(16, dtype=torch.uint8))):
        with pytest.raises(sp.SparseError):
            call()


def test_outputs_beside_inputs():
    """Outputs in other columns of one buffer's rows."""
    rng = rng_for("beside")
    buf = rows_tensor(rng, 70, 200, "f16")
    A, B = buf[:, :72], rows_tensor(rng, 40, 72, "f16")
    want = sp.moe_gemm(A.clone(), B)
    assert torch.equal(sp.moe_gemm(A, B, out=buf[:, 72:112]), want)
    y, s = sp.rms_norm(A.clone(), residual=A.clone())
    got = sp.rms_norm(A, residual=A, out=buf[:, 112:184])
    assert torch.equal(got[0], y) and torch.equal(got[1], s)

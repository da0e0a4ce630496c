"""Calls at the edges of the mixture-of-experts operators: operands on other streams, inside one buffer, scales and
sizes at the ends of their range, and launches with more work than workgroups."""
import numpy as np
import pytest
import torch

import spmm_csr_spmv_amd as sp
from gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def codes(g, *shape, most=127):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda", dtype=torch.int8)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ scales at the ends of the range
# one kernel each: 16 x 16, 16 x 32, 32 x 32, 32 x 64 tiles, 128 x 128 with four and two steps in LDS, 256 x 256, and
# rows of fewer than 16 bytes
@pytest.mark.parametrize("M,N,K", [(4, 40, 64), (8, 5000, 64), (20, 5000, 64), (60, 5000, 64), (700, 800, 64),
                                   (2100, 2100, 16), (5000, 5000, 16), (4, 40, 9)])
def test_large_scales_do_not_overflow_on_the_way(M, N, K):
    """Sums times a_scale beyond fp32's range, and a b_scale that brings the product back into it: three fp32
    roundings and nothing else.  The other way round, and both small, too."""
    say("large scales", M, N, K)
    g = gen(M)
    A, B = codes(g, M, K), codes(g, N, K)
    A[1], B[2] = 127, 127
    sa = torch.rand(M, generator=g, device="cuda") + 0.5
    sb = torch.rand(N, generator=g, device="cuda") + 0.5
    sums = A.double() @ B.double().t()
    for p, q in ((120.0, -60.0), (127.0, -30.0), (-60.0, 120.0), (-100.0, 30.0), (-126.0, 126.0), (-90.0, -40.0)):
        for rows in (slice(None), slice(0, M, 3)):  # all rows, and some among ordinary ones
            a = sa.clone()
            a[rows] *= 2.0 ** p
            b = sb * 2.0 ** q
            want = sums * a.double()[:, None] * b.double()
            got = sp.gemm_i8(A, a, B, b, dtype=torch.float32).double()
            big = want.abs() >= 2.0 ** 128 * (1 - 4 * U)
            assert not (got.isinf() & ~big).any() and not got.isnan().any()
            # below the normal range each of three roundings is off by half of 2^-149, what follows scales it by b
            tol = 3.001 * U * want.abs() + 2.0 ** -149 * (2 + b.double())
            assert ((got - want).abs() <= tol)[~big].all(), (p, q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(4, 4000, 64), (8, 5000, 64), (20, 5000, 64), (60, 5003, 64), (700, 1000, 64),
                                   (2100, 2100, 128), (3000, 5001, 16), (600, 2500, 9), (3000, 4000, 33)])
def test_products_are_rounded_alike_everywhere(M, N, K, dtype):
    """The float of a sum times a_scale times b_scale in fp32, then rounded: the same bits wherever in C a value stands,
    in whole tiles and at their edges, and beside rows with large scales."""
    say("rounding", M, N, K, dtype)
    g = gen(M)
    A, B = codes(g, M, K), codes(g, N, K)
    a = torch.randn(M, generator=g, device="cuda").exp()
    b = torch.randn(N, generator=g, device="cuda") * 0.01
    want = ((A.double() @ B.double().t()).float() * a[:, None] * b).to(dtype)
    assert torch.equal(sp.gemm_i8(A, a, B, b, dtype=dtype), want)
    a[M // 3] = 2.0 ** 110
    got = sp.gemm_i8(A, a, B, b, dtype=dtype)
    others = torch.arange(M, device="cuda") != M // 3
    assert torch.equal(got[others], want[others])


# ------------------------------------------------------------------ operands of another stream
def busy(stream):
    """Tens of milliseconds of work on `stream`."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)


def test_operands_of_a_side_stream_call_are_kept():
    """Memory of an operand that is dropped right after a call on a side stream is not handed out before the call has
    read it."""
    say("kept operands")
    T, k, E, H, F = 600, 2, 4, 256, 192
    rng = np.random.default_rng(3)
    ids0 = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    offsets, src, pos = sp.moe_sort(ids0, E)
    x0 = torch.randn(T, H, device="cuda")
    ys0 = torch.randn(T * k, H, device="cuda")
    w0 = torch.rand(T, k, device="cuda")
    q0, s0 = sp.quantize_rows_i8(x0)
    B0, b0 = codes(gen(4), E, F, H), torch.rand(E, F, device="cuda")
    many = torch.from_numpy(rng.integers(0, E, 9000).astype(np.int32)).cuda()
    work0 = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    calls = {
        "sort": (lambda s, i: sp.moe_sort(i, E, stream=s), (ids0,)),
        "sort's work": (lambda s, i, m: sp.moe_sort(i, E, work=m, stream=s), (many, work0)),
        "dispatch": (lambda s, x, p: sp.moe_dispatch(x, p, stream=s), (x0, pos)),
        "combine": (lambda s, y, p, w: sp.moe_combine(y, p, w, stream=s), (ys0, pos, w0)),
        "backward": (lambda s, g, y, p, w: sp.moe_combine_backward(g, y, p, w, stream=s), (x0, ys0, pos, w0)),
        "quantize": (lambda s, x: sp.quantize_rows_i8(x, stream=s), (x0,)),
        "gemm": (lambda s, q, a, B, b: sp.gemm_i8(q, a, B, b, stream=s), (q0, s0, B0[0], b0[0])),
        "experts": (lambda s, q, a, B, b, o, f: sp.moe_gemm_i8(q, a, B, b, o, src=f, slots=k, stream=s),
                    (q0, s0, B0, b0, offsets, src)),
    }
    side = torch.cuda.Stream()
    for name, (call, kept) in calls.items():
        want = call(None, *kept)
        args = [t.clone(memory_format=torch.contiguous_format) for t in kept]
        where = {t.data_ptr() for t in args}
        sizes = [(t.shape, t.dtype) for t in args]
        torch.cuda.synchronize()
        busy(side)
        got = call(side, *args)
        del args
        again = [torch.empty(s, dtype=d, device="cuda") for s, d in sizes]
        waiting = not side.query()
        handed_out = [t for t in again if t.data_ptr() in where]
        for t in again:
            t.zero_()
        torch.cuda.synchronize()
        assert waiting, "the side stream was done too early to show anything"
        assert not handed_out, name
        for u, v in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
            assert torch.equal(u, v), name


def test_stream_given_in_a_capture():
    """The operands of a call that is captured on the stream it is given, dropped and made anew between replays."""
    say("stream in a capture")
    T, k, E, H = 700, 2, 5, 160
    rng = np.random.default_rng(8)
    ids = torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)).cuda()
    x, w = torch.randn(T, H, device="cuda"), torch.rand(T, k, device="cuda")

    def step(stream):
        _, _, pos = sp.moe_sort(ids, E, stream=stream)
        rows = sp.moe_dispatch(x, pos, out=torch.zeros(T * k, H, device="cuda"), stream=stream)
        return sp.moe_combine(rows, pos, w, stream=stream)  # the rows' memory is free again after this

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        out = step(side)
    for n in range(4):
        x.normal_()
        ids.copy_(torch.from_numpy(rng.integers(-1, E, (T, k)).astype(np.int32)))
        want = step(None)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), n


# ------------------------------------------------------------------ operands inside one buffer
def test_operands_in_columns_of_one_buffer():
    """Inputs and outputs that are disjoint columns of one buffer do not overlap."""
    say("columns of one buffer")
    T, H = 40, 24
    pos = torch.arange(T, device="cuda", dtype=torch.int32).flip(0).view(T, 1).contiguous()
    w = torch.rand(T, 1, device="cuda")
    for a, b in ((0, H), (H + 3, 0)):  # input before the output and behind it
        whole = torch.randn(T, 2 * H + 3, device="cuda")
        x, out = whole[:, a:a + H], whole[:, b:b + H]
        xc, before = x.clone(), whole.clone()
        sp.moe_dispatch(x, pos, out=out)
        assert torch.equal(out, xc.flip(0))
        sp.moe_combine(x, pos, w, out=out)
        assert torch.equal(out, w * xc.flip(0))
        _, dw = sp.moe_combine_backward(x, xc, pos, w, dYs=out)
        assert torch.equal(out, (w * xc).flip(0))
        keep = torch.ones(2 * H + 3, dtype=torch.bool, device="cuda")
        keep[b:b + H] = False
        assert torch.equal(whole[:, keep], before[:, keep])
    both = torch.randint(-100, 101, (T, 64), device="cuda", dtype=torch.int8)
    A, B = both[:, :31], codes(gen(5), 16, 31)
    ones = torch.ones(T, device="cuda")
    want = A.double() @ B.double().t()
    sp.gemm_i8(A, ones, B, ones[:16], out=both.view(torch.float16)[:, 16:32])  # bytes 32 .. 63 of every row
    assert torch.equal(both.view(torch.float16)[:, 16:32], want.to(torch.float16))
    # codes beside the rows they are made of
    x = torch.randn(T, 16, device="cuda")
    wide = torch.zeros(T, 20, device="cuda")
    wide[:, :16] = x
    q, s = sp.quantize_rows_i8(wide[:, :16], q=wide.view(torch.int8)[:, 64:])
    assert torch.equal(q, sp.quantize_rows_i8(x)[0]) and torch.equal(wide[:, :16], x)


def test_operands_that_share_bytes_are_refused():
    say("shared bytes")
    T, H = 40, 24
    pos = torch.arange(T, device="cuda", dtype=torch.int32).view(T, 1)
    whole = torch.zeros(T, 2 * H, device="cuda")
    x = whole[:, :H]
    for out in (whole[:, H - 1:2 * H - 1],                       # one column of each row
                whole.view(-1)[5:5 + T * H].view(T, H),          # another row distance
                whole.view(-1).as_strided((T - 1, H), (2 * H, 1), 2 * H - 3)):  # over a row's end into the next
        with pytest.raises(ValueError, match="overlaps"):
            sp.moe_dispatch(x, pos, out=out)
    with pytest.raises(ValueError, match="overlaps"):  # the place list inside the output's rows
        ints = torch.zeros(T * H, dtype=torch.int32, device="cuda")
        sp.moe_combine(x, ints[:T].view(T, 1), out=ints.view(torch.float32).view(T, H))


# ------------------------------------------------------------------ numbers beyond 32 bits
def test_counts_beyond_32_bits_are_not_cut():
    say("counts")
    ids = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    for n in (2 ** 32 + 5, 2 ** 32, -2 ** 32 + 5, 2 ** 31):
        with pytest.raises(sp.SparseError) as e:
            sp.moe_sort(ids, n)
        assert e.value.code == 5
    A, s = torch.ones(3, 16, dtype=torch.int8, device="cuda"), torch.tensor([1.0, 2.0, 3.0], device="cuda")
    B, b = torch.ones(1, 4, 16, dtype=torch.int8, device="cuda"), torch.ones(1, 4, device="cuda")
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    src = torch.tensor([5, 4, 1], dtype=torch.int32, device="cuda")
    got = sp.moe_gemm_i8(A, s, B, b, off, src=src, slots=2 ** 32 + 2, dtype=torch.float32)
    assert (got == 16).all()  # src // slots is 0 everywhere
    with pytest.raises(sp.SparseError) as e:
        sp.moe_gemm_i8(A, s, B, b, off, src=src, slots=-2 ** 32 + 2)
    assert e.value.code == 2


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


# ------------------------------------------------------------------ more work than workgroups
# T behind 2^20 workgroups of 16, 4 and 1 tokens (the gradient: the same with twice the row), and rows of one element
@pytest.mark.parametrize("T,H,dtype", [((1 << 24) + 51, 4, torch.float32), ((1 << 24) + 33, 1, torch.bfloat16),
                                       ((1 << 22) + 77, 132, torch.float32), ((1 << 22) + 5, 137, torch.bfloat16),
                                       ((1 << 20) + 777, 516, torch.float32), ((1 << 20) + 1, 1040, torch.float16),
                                       ((1 << 20) + 300, 1088, torch.bfloat16)])
def test_rows_in_several_rounds(T, H, dtype):
    say("rows in rounds", T, H, dtype)
    g = gen(T)
    X = torch.randint(-8, 9, (T, H), generator=g, device="cuda", dtype=torch.int8).to(dtype)
    X[:, 0] = (torch.arange(T, device="cuda") % 61).to(dtype)  # neighbours, and rows a round apart, differ
    pos = torch.randperm(T, generator=g, device="cuda").to(torch.int32).view(T, 1)
    at = pos.view(-1).long()
    w = torch.randint(1, 4, (T, 1), generator=g, device="cuda").float()
    Xs = torch.full_like(X, -99)
    sp.moe_dispatch(X, pos, out=Xs)
    assert torch.equal(Xs[at], X)
    Y = torch.full_like(X, -99)
    sp.moe_combine(Xs, pos, w, out=Y)
    assert torch.equal(Y, w.to(dtype) * X)  # small whole numbers: exact
    dXs, dw = sp.moe_combine_backward(X, Xs, pos, w, dYs=Y)
    assert torch.equal(dXs[at], w.to(dtype) * X)
    for b in range(0, T, 1 << 22):  # sums below 2^24: exact
        x = X[b:b + (1 << 22)].float()
        assert torch.equal(dw[b:b + (1 << 22), 0], (x * x).sum(1)), b


# rows behind 2^20 workgroups of 16, 4 and 1 rows, in rows of a few elements, one chunk, held and read again
@pytest.mark.parametrize("rows,K,dtype", [((1 << 24) + 100, 1, torch.bfloat16), ((1 << 24) + 17, 11, torch.float32),
                                          ((1 << 22) + 9, 520, torch.bfloat16), ((1 << 20) + 555, 2056, torch.bfloat16),
                                          ((1 << 20) + 3, 4104, torch.float32)])
def test_quantised_rows_in_several_rounds(rows, K, dtype):
    say("quantise in rounds", rows, K, dtype)
    g = gen(K)
    X = torch.randint(-126, 127, (rows, K), generator=g, device="cuda", dtype=torch.int8).to(dtype)
    top = (127 * 2.0 ** (torch.arange(rows, device="cuda") % 5)).to(dtype)  # scales 1, 2, 4, 8, 16
    X[:, K // 2] = top
    q, s = sp.quantize_rows_i8(X)
    assert torch.equal(s, top.float() / 127)
    part = max(1, (1 << 28) // K)
    for b in range(0, rows, part):
        want = torch.round(X[b:b + part].float() / s[b:b + part, None])
        assert torch.equal(q[b:b + part].float(), want), b


@pytest.mark.parametrize("K", [1, 17])
def test_tiles_in_several_rounds(K):
    """More 128 x 128 tiles than workgroups: experts of one row, and a few of one and two blocks of 64."""
    say("tiles in rounds", K)
    E, N = 1024, 540000
    rows = np.ones(E, np.int64)
    rows[[3, 500]], rows[[0, 1023]], rows[7] = 100, 60, 0
    offsets = np.concatenate([[0], np.cumsum(rows)])
    S = int(offsets[-1])
    g = gen(K)
    A, B = codes(g, S, K), codes(g, E, N, K)
    ones = torch.ones(E, N, device="cuda")
    sa = torch.arange(S, device="cuda").float() % 3 + 1
    C = sp.moe_gemm_i8(A, sa, B, ones, torch.from_numpy(offsets.astype(np.int32)).cuda(), dtype=torch.float32)
    for e in range(E):
        a = slice(offsets[e], offsets[e + 1])
        want = (A[a].float() @ B[e].float().t()) * sa[a, None]  # whole numbers below 2^24: exact
        assert torch.equal(C[a], want), e


def test_one_row_of_more_tiles_than_workgroups():
    say("one row in rounds")
    N = (1 << 29) + 1000
    g = gen(9)
    B = codes(g, N, 1)
    A = torch.full((1, 1), 3, dtype=torch.int8, device="cuda")
    C = sp.gemm_i8(A, torch.ones(1, device="cuda"), B, torch.ones(N, device="cuda"), dtype=torch.float16)
    assert torch.equal(C[0], 3 * B[:, 0].half())


@pytest.mark.parametrize("S,N,K", [(300, 520, 40), (300, 520, 48), (9000, 300, 33), (9000, 600, 64)])
def test_overlapping_offsets_end(S, N, K):
    """Every other one of 1024 experts claims all rows: what C holds is unspecified, but the tiles are no more than the
    launch has room for and nothing around C is written."""
    say("overlapping offsets", S, N, K)
    E = 1024
    g = gen(K)
    A, B = codes(g, S, K), codes(g, E, N, K)
    offsets = torch.arange(E + 1, device="cuda", dtype=torch.int32) % 2 * S
    whole = torch.full((S + 2, N + 5), -7.0, device="cuda")
    out = whole[1:-1, 2:2 + N]
    sp.moe_gemm_i8(A, torch.ones(S, device="cuda"), B, torch.ones(E, N, device="cuda"), offsets, out=out)
    assert (out == out.round()).all()  # sums, or what was there
    out.fill_(-7.0)
    assert (whole == -7.0).all()

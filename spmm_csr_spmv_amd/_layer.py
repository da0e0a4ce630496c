"""ctypes binding of the norm, the gated products and the experts' products in 16 bits -- argument marshalling only.

In the manner of the mixture-of-experts calls: names of the C calls, checks of types,
shapes, devices, strides and overlaps, allocation of what is not given, SparseError
on a non-zero status, everything on `stream` (default: the current stream of the
tensors' device), nothing synchronises and nothing is recorded for autograd.
"""
import ctypes
import functools

import torch

from ._binding import SP_OK, SparseError, _sz, lib
from ._moe import (_F32, _I8, _I32, _TYPES, _apart, _call, _check, _int32, _operands, _product_out, _rows, _type, _want,
                   _whole)

_ACTS = {"silu": 0, "gelu_tanh": 1}
_16 = (torch.bfloat16, torch.float16)


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("act must be 'silu' or 'gelu_tanh', got %r" % (act,))
    return code


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ norm
# Each call tests its operands in a few expressions; what follows where one fails says what is wrong.
def _norm_rows(t, name, x, shape, device):
    """An operand of x's type and shape; its row distance."""
    if not (t.dtype is x.dtype and t.shape == shape and t.get_device() == device):
        _want(t, x.dtype, 2, name, device)
        raise ValueError("%s must have the rows' shape" % name)
    ld, step = t.stride()
    return ld if step == 1 and ld >= shape[1] > 0 else _rows(t, name)


def _norm_x(x, weight, name):
    """Type codes of the rows and of the weight (which may be None), the rows' shape, device and distance."""
    dtype = x.dtype
    code = _TYPES.get(dtype)
    device = x.get_device()
    if code is None or device < 0 or x.dim() != 2:
        _type(x, name)
        _want(x, dtype, 2, name)
    shape = x.shape
    H = shape[1]
    ld, step = x.stride()
    if step != 1 or ld < H or H == 0:
        ld = _rows(x, name)
    w_type = code
    if weight is not None:
        w = weight.dtype
        if not ((w is dtype or w is _F32) and weight.shape == (H,) and weight.get_device() == device
                and weight.is_contiguous()):
            _whole(weight, _F32 if w is _F32 else dtype, 1, "weight", device)
            raise ValueError("weight must have one entry per column")
        w_type = code if w is dtype else 0
    return code, w_type, shape, device, ld


def _like(x, ld, shape):
    """A contiguous buffer of x's type and shape, whose rows are ld apart."""
    return torch.empty_like(x) if ld == shape[1] and x.is_contiguous() else torch.empty(shape, dtype=x.dtype, device=x.device)


def _sum_out(x, residual, sum_out, weight, shape, device, ld_x):
    """The buffer of the sum (None without a residual), which may be x or the residual, and its row distance."""
    if sum_out is None:
        return (None, 0) if residual is None else (_like(x, ld_x, shape), shape[1])
    if residual is None:
        raise ValueError("sum_out is the sum with the residual, and there is none")
    ld = _norm_rows(sum_out, "sum_out", x, shape, device)
    _apart(sum_out, "sum_out", weight, *(t for t in (x, residual) if t.data_ptr() != sum_out.data_ptr()
                                         or t.stride() != sum_out.stride()))
    return sum_out, ld


def rms_norm(x, weight=None, residual=None, eps=1e-6, out=None, sum_out=None, stream=None):
    """Root-mean-square norm of the rows of x (rows x H, float32, bfloat16 or float16): s / sqrt(mean(s^2) + eps)
    * weight, in x's type.  With `residual` (x's type and shape) s = x + residual, rounded to that type, and the
    result is (norm, s); s goes to `sum_out`, which may be x or the residual.  weight: H values of x's type or
    float32; None: ones."""
    return _call(_rms_norm, x, stream, x, weight, residual, out, sum_out, eps, _norm_x(x, weight, "x"))


def _rms_norm(raw, x, weight, residual, out, sum_out, eps, of):
    code, w_type, shape, device, ld = of
    ld_r = 0 if residual is None else _norm_rows(residual, "residual", x, shape, device)
    total, ld_sum = _sum_out(x, residual, sum_out, weight, shape, device, ld)
    rows, H = shape
    if out is None:
        out, ld_out = _like(x, ld, shape), max(H, 1)
    else:
        ld_out = _norm_rows(out, "out", x, shape, device)
        _apart(out, "out", x, residual, weight, total)
    rc = lib().rms_norm(rows, H, code, x.data_ptr(), ld, None if residual is None else residual.data_ptr(), ld_r,
                        None if weight is None else weight.data_ptr(), w_type, eps,
                        None if total is None else total.data_ptr(), ld_sum, out.data_ptr(), ld_out, raw)
    if rc != SP_OK:
        raise SparseError("rms_norm", rc, lib())
    return out if residual is None else (out, total)


def rms_norm_i8(x, weight=None, residual=None, eps=1e-6, q=None, scale=None, sum_out=None, stream=None):
    """rms_norm with its result as int8 codes and one float32 scale per row, for gemm_i8, gated_i8 and the experts'
    products: (q, scale), with a residual (q, scale, s).  A q allocated here has its rows a multiple of 16 bytes apart."""
    return _call(_rms_norm_i8, x, stream, x, weight, residual, q, scale, sum_out, eps, _norm_x(x, weight, "x"))


def _rms_norm_i8(raw, x, weight, residual, q, scale, sum_out, eps, of):
    code, w_type, shape, device, ld = of
    ld_r = 0 if residual is None else _norm_rows(residual, "residual", x, shape, device)
    total, ld_sum = _sum_out(x, residual, sum_out, weight, shape, device, ld)
    rows, H = shape
    if q is None:
        ld_q = (H + 15) // 16 * 16
        q = torch.empty(rows, ld_q, dtype=_I8, device=x.device)
        if ld_q != H:
            q = q[:, :H]
    else:
        _want(q, _I8, 2, "q", device)
        if q.shape != shape:
            raise ValueError("q must have x's shape")
        _apart(q, "q", x, residual, weight, total)
        ld_q = _rows(q, "q")
    if scale is None:
        scale = torch.empty(rows, dtype=_F32, device=x.device)
    else:
        _whole(scale, _F32, 1, "scale", device)
        if scale.shape[0] != rows:
            raise ValueError("scale must have one entry per row")
        _apart(scale, "scale", x, residual, weight, total, q)
    rc = lib().rms_norm_i8(rows, H, code, x.data_ptr(), ld, None if residual is None else residual.data_ptr(), ld_r,
                           None if weight is None else weight.data_ptr(), w_type, eps,
                           None if total is None else total.data_ptr(), ld_sum, q.data_ptr(), max(ld_q, 1), scale.data_ptr(),
                           raw)
    if rc != SP_OK:
        raise SparseError("rms_norm_i8", rc, lib())
    return (q, scale) if residual is None else (q, scale, total)


@functools.lru_cache(maxsize=256)
def _bytes(name, *sizes):
    size = _sz()
    _check(name, getattr(lib(), name)(*sizes, ctypes.byref(size)))
    return size.value


def _work(work, need, device, *operands):
    """The workspace (allocated when None) and its size; refuses one that shares bytes with an operand."""
    if work is None:
        return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)
    if not (isinstance(work, torch.Tensor) and work.device == device and work.is_contiguous()):
        raise ValueError("work must be a contiguous tensor on %s" % device)
    _apart(work, "work", *operands)
    return work, work.nbytes


def rms_norm_backward(dy, s, weight=None, eps=1e-6, dsum=None, dx=None, dweight=None, work=None, stream=None):
    """Gradient of rms_norm: (dx, dweight).  s is the stored sum (x without a residual), dsum its own gradient where
    it is used elsewhere too; dx is the gradient of x and of the residual alike, dweight float32 (None without a
    weight).  `work` is a uint8 device tensor of rms_norm_backward_bufsize bytes (allocated when None)."""
    return _call(_rms_norm_backward, s, stream, dy, s, weight, dsum, dx, dweight, work, eps, _norm_x(s, weight, "s"))


def _rms_norm_backward(raw, dy, s, weight, dsum, dx, dweight, work, eps, of):
    code, w_type, shape, device, ld = of
    ld_dy = _norm_rows(dy, "dy", s, shape, device)
    ld_d = 0 if dsum is None else _norm_rows(dsum, "dsum", s, shape, device)
    rows, H = shape
    if dx is None:
        dx, ld_dx = _like(s, ld, shape), max(H, 1)
    else:
        ld_dx = _norm_rows(dx, "dx", s, shape, device)
        _apart(dx, "dx", dy, s, weight, dsum)
    if weight is None:
        if dweight is not None:
            raise ValueError("dweight is the weight's gradient, and there is none")
    elif dweight is None:
        dweight = torch.empty(H, dtype=_F32, device=s.device)
    else:
        _whole(dweight, _F32, 1, "dweight", device)
        if dweight.shape[0] != H:
            raise ValueError("dweight must have one entry per column")
        _apart(dweight, "dweight", dy, s, weight, dsum, dx)
    need = _bytes("rms_norm_backward_bufsize", rows, H, code) if dweight is not None else 0
    work, nbytes = _work(work, need, s.device, dy, s, weight, dsum, dx, dweight)
    rc = lib().rms_norm_backward(rows, H, code, dy.data_ptr(), ld_dy, s.data_ptr(), ld, _ptr(weight), w_type, eps,
                                 _ptr(dsum), ld_d, dx.data_ptr(), ld_dx, _ptr(dweight), _ptr(work), nbytes, raw)
    if rc != SP_OK:
        raise SparseError("rms_norm_backward", rc, lib())
    return dx, dweight


# ------------------------------------------------------------------ gated products in int8
def gated_i8(A, a_scale, B, b_scale, act="silu", out=None, dtype=torch.bfloat16, stream=None):
    """Gated product: out[m, n] = a(g) u of the products g and u that gemm_i8 gives at columns n and N + n; B int8
    2 N x K, the gate's N rows first, b_scale float32 [2 N].  act: "silu" or "gelu_tanh"."""
    _operands(A, a_scale, B, b_scale, 2)
    (M, K), rows = A.shape, B.shape[0]
    if B.shape[1] != K or rows % 2 or b_scale.shape[0] != rows:
        raise ValueError("B must be 2 N x K and b_scale have one entry per row of B")
    return _call(_gated_i8, A, stream, A, a_scale, B, b_scale, out, dtype, _act(act))


def _gated_i8(raw, A, a_scale, B, b_scale, out, dtype, act):
    (M, K), N = A.shape, B.shape[0] // 2
    out = _product_out(out, dtype, M, N, A, B, a_scale, b_scale)
    _check("gated_i8", lib().gated_i8(M, N, K, A.data_ptr(), _rows(A, "A"), a_scale.data_ptr(), B.data_ptr(),
                                      _rows(B, "B"), b_scale.data_ptr(), act, _TYPES[out.dtype], out.data_ptr(),
                                      _rows(out, "out"), raw))
    return out


def _matrices(B, name):
    """Row and expert distance of a tensor of matrices (the last two dimensions) with contiguous, disjoint rows."""
    shape, stride = B.shape, B.stride()
    N, K = shape[-2:]
    if K > 1 and stride[-1] != 1 or N > 1 and stride[-2] < K:
        raise ValueError("%s must have a contiguous last dimension and rows that do not overlap" % name)
    ld = max(stride[-2] if N > 1 else K, K, 1)
    return ld, stride[0] if len(shape) == 3 and shape[0] > 1 and N > 0 and K > 0 else N * ld


def moe_gated_i8(A, a_scale, B, b_scale, offsets, src=None, slots=1, act="silu", out=None, dtype=torch.bfloat16,
                 stream=None):
    """gated_i8 with one matrix per expert: B int8 E x 2 N x K, b_scale float32 E x 2 N; rows, offsets, src and slots
    as for moe_gemm_i8."""
    _operands(A, a_scale, B, b_scale, 3)
    _whole(offsets, _I32, 1, "offsets", A.get_device())
    E, rows, K = B.shape
    if A.shape[1] != K or rows % 2 or tuple(b_scale.shape) != (E, rows) or offsets.shape[0] != E + 1:
        raise ValueError("B must be E x 2 N x K, b_scale E x 2 N and offsets E + 1")
    if src is not None:
        _whole(src, _I32, 1, "src", A.get_device())
    return _call(_moe_gated_i8, A, stream, A, a_scale, B, b_scale, offsets, src, slots, out, dtype, _act(act))


def _moe_gated_i8(raw, A, a_scale, B, b_scale, offsets, src, slots, out, dtype, act):
    (a_rows, K), (E, rows, _) = A.shape, B.shape
    S, N = a_rows if src is None else src.shape[0], rows // 2
    ldb, strideb = _matrices(B, "B")
    out = _product_out(out, dtype, S, N, A, B, a_scale, b_scale, offsets, src)
    _check("moe_gated_i8",
           lib().moe_gated_i8(S, E, N, K, A.data_ptr(), a_rows, _rows(A, "A"), a_scale.data_ptr(), _ptr(src),
                              _int32(slots), B.data_ptr(), ldb, strideb, b_scale.data_ptr(), offsets.data_ptr(), act,
                              _TYPES[out.dtype], out.data_ptr(), _rows(out, "out"), raw))
    return out


# ------------------------------------------------------------------ products of experts in 16 bits
def _product_args(A, B, offsets, src, slots, gate):
    """S, E, N, K, type code and A .. offsets as the C calls take them, after the operands' checks."""
    device = A.get_device()
    dtype = A.dtype
    dim = 2 if offsets is None else 3
    if not (dtype in _16 and A.dim() == 2 and device >= 0 and B.dtype is dtype and B.dim() == dim
            and B.get_device() == device):
        if isinstance(A, torch.Tensor) and dtype not in _16:
            raise TypeError("A must be bfloat16 or float16, got %s" % dtype)
        _want(A, dtype, 2, "A")
        _want(B, dtype, dim, "B", device)
    a_rows, K = A.shape
    shape = B.shape
    N = shape[-2]
    if shape[-1] != K:
        raise ValueError("A and B must have rows of one length")
    E = 1
    if offsets is not None:
        E = shape[0]
        if not (offsets.dtype is _I32 and offsets.shape == (E + 1,) and offsets.get_device() == device
                and offsets.is_contiguous()):
            _whole(offsets, _I32, 1, "offsets", device)
            raise ValueError("offsets must be E + 1")
    S = a_rows
    if src is not None:
        _whole(src, _I32, 1, "src", device)
        S = src.shape[0]
    if gate:
        if N % 2:
            raise ValueError("B must have 2 N rows a matrix")
        N //= 2
    ld, step = A.stride()
    if step != 1 or ld < K or K == 0:
        ld = _rows(A, "A")
    return (S, E, N, K, _TYPES[dtype]), (A.data_ptr(), a_rows, ld, _ptr(src), _int32(slots), B.data_ptr(),
                                         *_matrices(B, "B"), _ptr(offsets))


def _rows_like(t, name, A, rows, columns):
    """A rows x columns operand of A's type; its row distance."""
    if not (t.dtype is A.dtype and t.shape == (rows, columns) and t.get_device() == A.get_device()):
        _want(t, A.dtype, 2, name, A.get_device())
        raise ValueError("%s must be %d x %d" % (name, rows, columns))
    ld, step = t.stride()
    return ld if step == 1 and ld >= columns > 0 else _rows(t, name)


def moe_gemm(A, B, offsets=None, src=None, slots=1, out=None, stream=None):
    """The experts' product in 16 bits: row p of out (S x N) in expert e's range is B[e] (N x K) times A's row p, or
    with src (moe_sort's, and its slots per token) A's row src[p] // slots.  A and B bfloat16 or float16, B E x N x K
    with offsets int32 [E + 1] (moe_sort); offsets None: one matrix, B N x K.  Rows behind the last expert's keep
    their contents (undefined where out is allocated here)."""
    return _call(_moe_gemm, A, stream, A, B, offsets, src, out, _product_args(A, B, offsets, src, slots, False))


def _moe_gemm(raw, A, B, offsets, src, out, of):
    sizes, operands = of
    if out is None:
        out, ld = torch.empty(sizes[0], sizes[2], dtype=A.dtype, device=A.device), max(sizes[2], 1)
    else:
        ld = _rows_like(out, "out", A, sizes[0], sizes[2])
        _apart(out, "out", A, B, offsets, src)
    rc = lib().moe_gemm(*sizes, *operands, out.data_ptr(), ld, raw)
    if rc != SP_OK:
        raise SparseError("moe_gemm", rc, lib())
    return out


def moe_gated(A, B, offsets=None, src=None, slots=1, act="silu", pre=None, out=None, stream=None):
    """The experts' gated product in 16 bits: out[p, n] = a(g) u of the products g and u with rows n and N + n of B[e]
    (2 N x K), operands as for moe_gemm; act: "silu" or "gelu_tanh".  `pre` (S x 2 N, A's type) receives the
    pre-activations [g u], which moe_gated_backward wants."""
    return _call(_moe_gated, A, stream, A, B, offsets, src, pre, out, _act(act),
                 _product_args(A, B, offsets, src, slots, True))


def _moe_gated(raw, A, B, offsets, src, pre, out, act, of):
    sizes, operands = of
    S, _, N = sizes[:3]
    ld_pre = 0
    if pre is not None:
        ld_pre = _rows_like(pre, "pre", A, S, 2 * N)
        _apart(pre, "pre", A, B, offsets, src)
    if out is None:
        out, ld = torch.empty(S, N, dtype=A.dtype, device=A.device), max(N, 1)
    else:
        ld = _rows_like(out, "out", A, S, N)
        _apart(out, "out", A, B, offsets, src, pre)
    rc = lib().moe_gated(*sizes, *operands, act, _ptr(pre), ld_pre, out.data_ptr(), ld, raw)
    if rc != SP_OK:
        raise SparseError("moe_gated", rc, lib())
    return out


def _gradients(sizes, A, B, dA, dB, *inputs):
    """The gradients' buffers, allocated where they are True; with their distances as the C calls take them."""
    S, K = sizes[0], sizes[3]
    if dA is True:
        dA = torch.empty(S, K, dtype=A.dtype, device=A.device)
    if dB is True:
        dB = torch.empty(B.shape, dtype=B.dtype, device=B.device)
    ld_a = ld_b = stride_b = 0
    if dA is not None:
        ld_a = _rows_like(dA, "dA", A, S, K)
        _apart(dA, "dA", A, B, *inputs)
    if dB is not None:
        if not (dB.dtype is B.dtype and dB.shape == B.shape and dB.get_device() == B.get_device()):
            _want(dB, B.dtype, B.dim(), "dB", B.get_device())
            raise ValueError("dB must have B's shape")
        ld_b, stride_b = _matrices(dB, "dB")
        _apart(dB, "dB", A, B, dA, *inputs)
    return dA, dB, (_ptr(dA), ld_a, _ptr(dB), ld_b, stride_b)


def moe_gemm_backward(dC, A, B, offsets=None, src=None, slots=1, dA=True, dB=True, work=None, stream=None):
    """Gradient of moe_gemm: (dA, dB), dA S x K by sorted row (with src, moe_combine adds up a token's), dB of B's
    shape, zeros for an expert without rows.  dA and dB are buffers, True: allocated here, None: not wanted.  Rows of
    dA behind the last expert's keep their contents (undefined where dA is allocated here).  `work` is a uint8 device
    tensor of moe_gemm_backward_bufsize bytes (allocated when None)."""
    return _call(_moe_gemm_backward, A, stream, dC, A, B, offsets, src, dA, dB, work,
                 _product_args(A, B, offsets, src, slots, False))


def _moe_gemm_backward(raw, dC, A, B, offsets, src, dA, dB, work, of):
    sizes, operands = of
    ld = _rows_like(dC, "dC", A, sizes[0], sizes[2])
    dA, dB, outputs = _gradients(sizes, A, B, dA, dB, dC, offsets, src)
    need = 0 if dA is None and dB is None else _bytes("moe_gemm_backward_bufsize", *sizes)
    work, nbytes = _work(work, need, A.device, dC, A, B, offsets, src, dA, dB)
    rc = lib().moe_gemm_backward(*sizes, dC.data_ptr(), ld, *operands, *outputs, _ptr(work), nbytes, raw)
    if rc != SP_OK:
        raise SparseError("moe_gemm_backward", rc, lib())
    return dA, dB


def moe_gated_backward(dout, pre, A, B, offsets=None, src=None, slots=1, act="silu", dA=True, dB=True, work=None,
                       stream=None):
    """Gradient of moe_gated: (dA, dB) as of moe_gemm_backward, from dout (S x N) and the pre-activations that
    moe_gated left in `pre` (S x 2 N).  `work`: moe_gated_backward_bufsize bytes."""
    return _call(_moe_gated_backward, A, stream, dout, pre, A, B, offsets, src, _act(act), dA, dB, work,
                 _product_args(A, B, offsets, src, slots, True))


def _moe_gated_backward(raw, dout, pre, A, B, offsets, src, act, dA, dB, work, of):
    sizes, operands = of
    ld = _rows_like(dout, "dout", A, sizes[0], sizes[2])
    ld_pre = _rows_like(pre, "pre", A, sizes[0], 2 * sizes[2])
    dA, dB, outputs = _gradients(sizes, A, B, dA, dB, dout, pre, offsets, src)
    need = 0 if dA is None and dB is None else _bytes("moe_gated_backward_bufsize", *sizes)
    work, nbytes = _work(work, need, A.device, dout, pre, A, B, offsets, src, dA, dB)
    rc = lib().moe_gated_backward(*sizes, act, dout.data_ptr(), ld, pre.data_ptr(), ld_pre, *operands, *outputs,
                                  _ptr(work), nbytes, raw)
    if rc != SP_OK:
        raise SparseError("moe_gated_backward", rc, lib())
    return dA, dB

"""ctypes binding of the mixture-of-experts entry points -- argument marshalling only.

Like the rest of the package: the functions have the names of the C calls, check
types, shapes, devices and strides, allocate what is not given, and raise
SparseError on a non-zero status.  Row tensors may have any row distance as long
as their last dimension is contiguous and rows do not overlap.  Everything is
enqueued on `stream` (default: the current stream of the tensors' device; with a
stream given the operands are marked as used there, so that their memory is not
handed out again before the call has read it), nothing synchronises, and nothing
here is recorded for autograd: gradients are calls of their own (moe_combine for
moe_dispatch's, moe_combine_backward for moe_combine's).
"""
import ctypes
import functools

import torch

from ._binding import SP_OK, SparseError, _on, _sz, _used_on, lib

_Tensor = torch.Tensor
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _check(fn, code):
    if code != SP_OK:
        raise SparseError(fn, code, lib())


# The calls take a few microseconds on the GPU at small sizes, so each tests its
# arguments in one expression first; _want and _whole, which say what is wrong,
# run where that fails.
_F32, _I32, _I8 = torch.float32, torch.int32, torch.int8


def _type(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    return code


def _want(t, dtype, dim, name, device=None):
    """Checks type, number of dimensions and device (a number; None: any)."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.is_cuda and t.dim() == dim and (
            device is None or t.get_device() == device):
        return
    if not isinstance(t, _Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise TypeError("%s must be a device tensor" % name)
    if t.dim() != dim:
        raise ValueError("%s must have %d dimensions, got %d" % (name, dim, t.dim()))
    raise ValueError("%s is on device %d, the others on %d" % (name, t.get_device(), device))


def _whole(t, dtype, dim, name, device=None):
    """_want, and contiguous."""
    _want(t, dtype, dim, name, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _rows(t, name):
    """Row distance of a 2-D tensor with contiguous, disjoint rows."""
    rows, cols = t.shape
    ld, step = t.stride()
    if step == 1 and ld >= cols > 0:
        return ld
    if cols > 1 and step != 1 or rows > 1 and ld < cols:
        raise ValueError("%s must have a contiguous last dimension and rows that do not overlap" % name)
    return max(ld, cols, 1)


def _reach(t):
    """Bytes from a tensor's first element to behind its last, gaps included."""
    if t.is_contiguous():
        return t.nbytes
    return (sum((n - 1) * d for n, d in zip(t.shape, t.stride())) + 1) * t.element_size() if t.numel() else 0


def _line(t):
    """(row distance, row length) in bytes of a tensor whose rows are contiguous, equally far apart and disjoint;
    (0, 0) where they are not."""
    ld, size = 0, t.element_size()
    for n, d in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n > 1:
            if ld and d % ld:
                return 0, 0
            ld = ld or d
    if t.dim() < 2 or (t.shape[-1] > 1 and t.stride(-1) != 1) or ld < t.shape[-1]:
        return 0, 0
    return ld * size, t.shape[-1] * size


def _columns_apart(a, b):
    """Whether two tensors lie in different columns of rows of one distance, as two parts of one buffer do."""
    (la, wa), (lb, wb) = _line(a), _line(b)
    between = (b.data_ptr() - a.data_ptr()) % la if la else 0
    return la == lb > 0 and between >= wa and between + wb <= la


def _apart(out, name, *inputs):
    """Refuses an output that may share bytes with an input."""
    lo = out.data_ptr()
    hi = lo + _reach(out)
    for t in inputs:
        if t is not None:
            b = t.data_ptr()
            if b < hi and lo < b + _reach(t) and not _columns_apart(out, t):
                raise ValueError("%s overlaps an input" % name)


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _call(body, t, stream, *args):
    """body(raw stream, *args) with t's device current and allocations on the stream."""
    device = t.get_device()
    if stream is None and device == _current_device():
        return body(_current_stream(device), *args)
    if stream is not None and stream.device.index != device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    with torch.cuda.device(device), _on(stream):
        result = body(_current_stream(device), *args)
    for a in args:
        if isinstance(a, _Tensor):
            _used_on(a, stream)
    return result


def _int32(v):
    """v as the C calls take it; what int32 cannot hold becomes its nearest end (ctypes would cut off the high bits)."""
    return max(-2 ** 31, min(int(v), 2 ** 31 - 1))


@functools.lru_cache(maxsize=256)
def _sort_bytes(n, num_experts):
    size = _sz()
    _check("moe_sort_bufsize", lib().moe_sort_bufsize(n, num_experts, ctypes.byref(size)))
    return size.value


def moe_sort(ids, num_experts, work=None, stream=None):
    """Stable sort of the slots ids (int32, any shape) by expert: (offsets int32
    [num_experts + 1], src int32 [n], pos int32 of ids' shape).  src[p] is the slot
    at place p (-1 from place offsets[-1] on), pos[f] the place of slot f; a slot
    whose id is outside [0, num_experts) is routed nowhere, its pos is -1.  `work` is
    a uint8 device tensor of moe_sort_bufsize bytes apart from ids (allocated when None)."""
    _whole(ids, _I32, ids.dim(), "ids")
    n, num_experts = ids.numel(), _int32(num_experts)
    need = _sort_bytes(n, num_experts)
    return _call(_sort, ids, stream, ids, n, num_experts, need, work)


def _sort(raw, ids, n, num_experts, need, work):
    device = ids.device
    offsets = torch.empty(num_experts + 1, dtype=_I32, device=device)
    src = torch.empty(n, dtype=_I32, device=device)
    pos = torch.empty(ids.shape, dtype=_I32, device=device)
    if work is None:
        work = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    elif work.device != device or not work.is_contiguous():
        raise ValueError("work must be a contiguous tensor on %s" % device)
    nbytes = 0 if work is None else work.nbytes
    rc = lib().moe_sort(n, num_experts, ids.data_ptr(), offsets.data_ptr(), src.data_ptr(), pos.data_ptr(),
                        work.data_ptr() if nbytes else None, nbytes, raw)
    if rc != SP_OK:
        raise SparseError("moe_sort", rc, lib())
    return offsets, src, pos


def moe_dispatch(X, pos, S=None, out=None, stream=None):
    """out[pos[t, j]] = X[t]: the rows of X (T x H) at their places, out S x H.  pos is
    int32 T x slots (moe_sort); S defaults to T * slots.  Rows that no slot names keep
    their contents (they are undefined where out is allocated here)."""
    code = _type(X, "X")
    device = X.get_device()
    if not (X.dim() == 2 and device >= 0 and pos.dtype is _I32 and pos.dim() == 2 and pos.get_device() == device
            and pos.is_contiguous()):
        _want(X, X.dtype, 2, "X")
        _whole(pos, _I32, 2, "pos", device)
    T, slots = pos.shape
    if X.shape[0] != T or slots < 1:
        raise ValueError("pos must be T x slots, slots at least 1")
    return _call(_dispatch, X, stream, code, X, pos, T, slots, S, out)


def _dispatch(raw, code, X, pos, T, slots, S, out):
    H = X.shape[1]
    if out is None:
        out = torch.empty(T * slots if S is None else int(S), H, dtype=X.dtype, device=X.device)
        ld_out = H
    else:
        _want(out, X.dtype, 2, "out", X.get_device())
        if out.shape[1] != H or (S is not None and out.shape[0] != S):
            raise ValueError("out must be S x H")
        _apart(out, "out", X, pos)
        ld_out = _rows(out, "out")
    rc = lib().moe_dispatch(T, slots, H, out.shape[0], code, X.data_ptr(), _rows(X, "X"), pos.data_ptr(),
                            out.data_ptr(), ld_out, raw)
    if rc != SP_OK:
        raise SparseError("moe_dispatch", rc, lib())
    return out


def moe_combine(Ys, pos, weights=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] Ys[pos[t, j]] (T x H); weights float32 T x slots, or
    None for all ones (then it is also the gradient of moe_dispatch)."""
    code = _type(Ys, "Ys")
    device = Ys.get_device()
    if not (Ys.dim() == 2 and device >= 0 and pos.dtype is _I32 and pos.dim() == 2 and pos.get_device() == device
            and pos.is_contiguous()):
        _want(Ys, Ys.dtype, 2, "Ys")
        _whole(pos, _I32, 2, "pos", device)
    if weights is not None and not (weights.dtype is _F32 and weights.shape == pos.shape
                                    and weights.get_device() == device and weights.is_contiguous()):
        _whole(weights, _F32, 2, "weights", device)
        raise ValueError("weights must have pos's shape")
    return _call(_combine, Ys, stream, code, Ys, pos, weights, out)


def _combine(raw, code, Ys, pos, weights, out):
    (T, slots), (S, H) = pos.shape, Ys.shape
    if slots < 1:
        raise ValueError("pos must be T x slots, slots at least 1")
    if out is None:
        out = torch.empty(T, H, dtype=Ys.dtype, device=Ys.device)
        ld_out = H
    else:
        _want(out, Ys.dtype, 2, "out", Ys.get_device())
        if tuple(out.shape) != (T, H):
            raise ValueError("out must be T x H")
        _apart(out, "out", Ys, pos, weights)
        ld_out = _rows(out, "out")
    rc = lib().moe_combine(T, slots, H, S, code, Ys.data_ptr(), _rows(Ys, "Ys"), pos.data_ptr(),
                           None if weights is None else weights.data_ptr(), out.data_ptr(), ld_out, raw)
    if rc != SP_OK:
        raise SparseError("moe_combine", rc, lib())
    return out


def moe_combine_backward(dY, Ys, pos, weights, dYs=None, dweights=None, stream=None):
    """Gradient of moe_combine: (dYs, dweights) with dYs[pos[t, j]] = weights[t, j] dY[t] (S x H;
    rows that no slot names keep their contents, undefined where dYs is allocated here)
    and dweights[t, j] = <dY[t], Ys[pos[t, j]]>, 0 where the slot is routed nowhere."""
    code = _type(Ys, "Ys")
    device = Ys.get_device()
    if not (Ys.dim() == 2 and device >= 0 and dY.dtype is Ys.dtype and dY.dim() == 2 and dY.get_device() == device
            and pos.dtype is _I32 and pos.dim() == 2 and pos.get_device() == device and pos.is_contiguous()
            and weights.dtype is _F32 and weights.get_device() == device and weights.is_contiguous()):
        _want(Ys, Ys.dtype, 2, "Ys")
        _want(dY, Ys.dtype, 2, "dY", device)
        _whole(pos, _I32, 2, "pos", device)
        _whole(weights, _F32, 2, "weights", device)
    T, slots = pos.shape
    if slots < 1 or weights.shape != pos.shape or dY.shape[0] != T or dY.shape[1] != Ys.shape[1]:
        raise ValueError("dY must be T x H, pos and weights T x slots, slots at least 1")
    return _call(_combine_backward, Ys, stream, code, dY, Ys, pos, weights, dYs, dweights)


def _combine_backward(raw, code, dY, Ys, pos, weights, dYs, dweights):
    (T, slots), (S, H) = pos.shape, Ys.shape
    if dYs is None:
        dYs = torch.empty(S, H, dtype=Ys.dtype, device=Ys.device)
    else:
        _want(dYs, Ys.dtype, 2, "dYs", Ys.get_device())
        if dYs.shape != Ys.shape:
            raise ValueError("dYs must be S x H")
        _apart(dYs, "dYs", dY, Ys, pos, weights)
    if dweights is None:
        dweights = torch.empty(T, slots, dtype=_F32, device=Ys.device)
    else:
        _whole(dweights, _F32, 2, "dweights", Ys.get_device())
        if dweights.shape != pos.shape:
            raise ValueError("dweights must have pos's shape")
        _apart(dweights, "dweights", dY, Ys, pos, weights, dYs)
    _check("moe_combine_backward",
           lib().moe_combine_backward(T, slots, H, S, code, dY.data_ptr(), _rows(dY, "dY"), Ys.data_ptr(),
                                      _rows(Ys, "Ys"), pos.data_ptr(), weights.data_ptr(), dYs.data_ptr(),
                                      _rows(dYs, "dYs"), dweights.data_ptr(), raw))
    return dYs, dweights


def quantize_rows_i8(X, q=None, scale=None, stream=None):
    """Rows of X (rows x K) as int8 codes and one float32 scale each: (q, scale), X about
    q * scale[:, None].  A q allocated here has its rows a multiple of 16 bytes apart, as
    the fast kernels of the products want them."""
    code = _type(X, "X")
    _want(X, X.dtype, 2, "X")
    return _call(_quantize, X, stream, code, X, q, scale)


def _quantize(raw, code, X, q, scale):
    rows, K = X.shape
    if q is None:
        q = torch.empty(rows, (K + 15) // 16 * 16, dtype=_I8, device=X.device)
        if q.shape[1] != K:
            q = q[:, :K]
    else:
        _want(q, _I8, 2, "q", X.get_device())
        if q.shape != X.shape:
            raise ValueError("q must have X's shape")
        _apart(q, "q", X)
    if scale is None:
        scale = torch.empty(rows, dtype=_F32, device=X.device)
    else:
        _whole(scale, _F32, 1, "scale", X.get_device())
        if scale.shape[0] != rows:
            raise ValueError("scale must have one entry per row")
        _apart(scale, "scale", X, q)
    _check("quantize_rows_i8", lib().quantize_rows_i8(rows, K, code, X.data_ptr(), _rows(X, "X"), q.data_ptr(),
                                                      _rows(q, "q"), scale.data_ptr(), raw))
    return q, scale


def _operands(A, a_scale, B, b_scale, dim):
    """Types, dimensions and devices of a product's operands (B has dim dimensions)."""
    device = A.get_device()
    if not (A.dtype is _I8 and A.dim() == 2 and device >= 0 and B.dtype is _I8 and B.dim() == dim
            and B.get_device() == device and a_scale.dtype is _F32 and a_scale.dim() == 1
            and a_scale.get_device() == device and a_scale.is_contiguous() and b_scale.dtype is _F32
            and b_scale.dim() == dim - 1 and b_scale.get_device() == device and b_scale.is_contiguous()):
        _want(A, _I8, 2, "A")
        _whole(a_scale, _F32, 1, "a_scale", device)
        _want(B, _I8, dim, "B", device)
        _whole(b_scale, _F32, dim - 1, "b_scale", device)
    if a_scale.shape[0] != A.shape[0]:
        raise ValueError("a_scale must have one entry per row of A")


def _product_out(out, dtype, rows, N, A, *inputs):
    if out is None:
        if dtype not in _TYPES:
            raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % (dtype,))
        return torch.empty(rows, N, dtype=dtype, device=A.device)
    _type(out, "out")
    _want(out, out.dtype, 2, "out", A.get_device())
    if tuple(out.shape) != (rows, N):
        raise ValueError("out must be %d x %d" % (rows, N))
    _apart(out, "out", A, *inputs)
    return out


def gemm_i8(A, a_scale, B, b_scale, out=None, dtype=torch.bfloat16, stream=None):
    """out[m, n] = a_scale[m] b_scale[n] sum_k A[m, k] B[n, k]: A int8 M x K, B int8 N x K, scales
    float32; out in `dtype` (float32, bfloat16 or float16) when it is allocated here."""
    _operands(A, a_scale, B, b_scale, 2)
    (M, K), N = A.shape, B.shape[0]
    if B.shape[1] != K or b_scale.shape[0] != N:
        raise ValueError("B must be N x K and b_scale have one entry per row of B")
    return _call(_gemm, A, stream, A, a_scale, B, b_scale, out, dtype)


def _gemm(raw, A, a_scale, B, b_scale, out, dtype):
    (M, K), N = A.shape, B.shape[0]
    out = _product_out(out, dtype, M, N, A, B, a_scale, b_scale)
    _check("gemm_i8", lib().gemm_i8(M, N, K, A.data_ptr(), _rows(A, "A"), a_scale.data_ptr(), B.data_ptr(),
                                    _rows(B, "B"), b_scale.data_ptr(), _TYPES[out.dtype], out.data_ptr(),
                                    _rows(out, "out"), raw))
    return out


def moe_gemm_i8(A, a_scale, B, b_scale, offsets, src=None, slots=1, out=None, dtype=torch.bfloat16, stream=None):
    """The product with one matrix per expert: B int8 E x N x K, b_scale float32 E x N, offsets
    int32 [E + 1] (moe_sort).  Row p of out in expert e's range is the product of A's row p, or
    with src (moe_sort's, and its slots per token) of A's row src[p] // slots.  Rows behind the
    last expert's keep their contents (undefined where out is allocated here)."""
    _operands(A, a_scale, B, b_scale, 3)
    _whole(offsets, _I32, 1, "offsets", A.get_device())
    (rows, K), (E, N, _) = A.shape, B.shape
    if B.shape[2] != K or tuple(b_scale.shape) != (E, N) or offsets.shape[0] != E + 1:
        raise ValueError("B must be E x N x K, b_scale E x N and offsets E + 1")
    if src is not None:
        _whole(src, _I32, 1, "src", A.get_device())
    S = rows if src is None else src.shape[0]
    if K > 1 and B.stride(2) != 1 or N > 1 and B.stride(1) < K:
        raise ValueError("B must have a contiguous last dimension and rows that do not overlap")
    ldb = max(B.stride(1), K, 1)
    strideb = B.stride(0) if K > 0 else N * ldb
    return _call(_moe_gemm, A, stream, A, a_scale, B, b_scale, offsets, src, slots, out, dtype, ldb, strideb)


def _moe_gemm(raw, A, a_scale, B, b_scale, offsets, src, slots, out, dtype, ldb, strideb):
    (rows, K), (E, N, _) = A.shape, B.shape
    S = rows if src is None else src.shape[0]
    out = _product_out(out, dtype, S, N, A, B, a_scale, b_scale, offsets, src)
    _check("moe_gemm_i8",
           lib().moe_gemm_i8(S, E, N, K, A.data_ptr(), rows, _rows(A, "A"), a_scale.data_ptr(),
                             src.data_ptr() if src is not None else None, _int32(slots), B.data_ptr(), ldb, strideb,
                             b_scale.data_ptr(), offsets.data_ptr(), _TYPES[out.dtype], out.data_ptr(),
                             _rows(out, "out"), raw))
    return out

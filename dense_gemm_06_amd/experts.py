"""Block-scaled 8-bit products, and the experts built on them, for torch tensors.

The functions mirror include/gemm_experts.h: they check the tensors, allocate the results
and pass pointers, strides and the current stream on; every step runs in the library's HIP
kernels. Results belong to the current stream of the tensors' device, and the calls can be
captured into a graph.

  gemm_block_quantize_tensors           values -> codes with block scales, as they are and transposed
  gemm_block_product_tensors            C = A B^T for block-scaled A and B
  gemm_experts_route_tensors            scores, choice of experts and their weights
  gemm_experts_route_backward_tensors   the logits' gradient
  gemm_experts_dispatch_tensors         the plan: every expert's rows
  gemm_experts_product_tensors          every row's product with its expert's matrix
  gemm_experts_gradient_tensors         that product's weight gradients
  gemm_experts_combine_tensors          the weighted sum of each token's rows
  gemm_experts_combine_backward_tensors its gradients

Tensors need unit stride along their last dimension (an operand's codes along either); other
strides are free. Results carry no gradient, also of tensors that require one: a training step
calls the gradients' operators itself (examples/experts_step.py) or from its own
torch.autograd.Function.
"""
from __future__ import annotations

import ctypes

import dense_gemm_06_amd as _dg

GEMM_E4M3, GEMM_E5M2 = 3, 4
GEMM_SCORE_SOFTMAX, GEMM_SCORE_SIGMOID = 0, 1
SCORE_CODE = {"softmax": GEMM_SCORE_SOFTMAX, "sigmoid": GEMM_SCORE_SIGMOID}
BLOCK = 128

_i64, _i32, _vp, _f = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float


class gemm_block_matrix(ctypes.Structure):
    """Codes and block scales of a matrix, or of a batch of them (see include/gemm_experts.h)."""
    _fields_ = [("data", _vp), ("scale", _vp), ("rows", _i64), ("cols", _i64), ("ld", _i64), ("scale_row", _i64),
                ("scale_block", _i64), ("stride", _i64), ("scale_stride", _i64), ("dtype", _i32),
                ("block_rows", _i32), ("op", _i32), ("reserved", _i32)]


class gemm_router(ctypes.Structure):
    """How experts are chosen (see include/gemm_experts.h)."""
    _fields_ = [("top_k", _i32), ("score", _i32), ("groups", _i32), ("top_groups", _i32), ("group_top", _i32),
                ("renorm", _i32), ("factor", _f)]


class gemm_expert_plan(ctypes.Structure):
    """The arrays of a plan (see include/gemm_experts.h)."""
    _fields_ = [("offsets", _vp), ("counts", _vp), ("rows", _vp), ("position", _vp), ("experts", _i64),
                ("tokens", _i64), ("top_k", _i64), ("capacity", _i64)]


def router(top_k, score="softmax", groups=1, top_groups=1, group_top=1, renorm=False, factor=1.0) -> gemm_router:
    return gemm_router(top_k, SCORE_CODE[score] if isinstance(score, str) else score, groups, top_groups, group_top,
                       int(renorm), factor)


def declare(lib):
    """The argument types of include/gemm_experts.h's functions."""
    c_int = ctypes.c_int
    mat, rt, pl = ctypes.POINTER(gemm_block_matrix), ctypes.POINTER(gemm_router), ctypes.POINTER(gemm_expert_plan)
    for name, args, res in (
            ("gemm_block_quantize", [_vp, _i64, _i64, _i64, c_int, _vp, _i64, mat, mat, _vp], c_int),
            ("gemm_block_product", [mat, mat, _vp, _i64, c_int, _vp, _i64, _vp], c_int),
            ("gemm_block_product_workspace", [_i64, _i64, _i64], _i64),
            ("gemm_experts_route", [_vp, _i64, _i64, _i64, c_int, rt, _vp, _vp, _vp, _vp], c_int),
            ("gemm_experts_route_backward", [_vp, _i64, _i64, _i64, c_int, rt, _vp, _vp, _vp, _i64, _vp], c_int),
            ("gemm_experts_capacity", [_i64, _i64, _i64, _i64], _i64),
            ("gemm_experts_dispatch", [_vp, _i64, pl, _vp, _i64, _vp], c_int),
            ("gemm_experts_dispatch_workspace", [_i64, _i64, _i64], _i64),
            ("gemm_experts_product", [mat, mat, pl, c_int, _vp, _i64, c_int, _vp], c_int),
            ("gemm_experts_gradient", [mat, mat, pl, _vp, _i64, _i64, c_int, _vp], c_int),
            ("gemm_experts_combine", [_vp, _i64, _i64, c_int, pl, _vp, _vp, _i64, _vp], c_int),
            ("gemm_experts_combine_backward", [_vp, _i64, _i64, c_int, pl, _vp, _vp, _i64, _vp, _i64, _vp, _vp],
             c_int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


class BlockTensor:
    """Codes and scales: data (..., R, K) float8_e4m3fn or float8_e5m2; scale (..., ceil(R / block_rows),
    ceil(K / 128)) float32, the number at (i, k) being data[i, k] * scale[i // block_rows, k // 128].
    Either of data's last two dimensions may be the contiguous one, so that codes in 128 x 128 blocks
    serve both ways (t())."""
    __slots__ = ("data", "scale", "block_rows")

    def __init__(self, data, scale, block_rows=1):
        self.data, self.scale, self.block_rows = data, scale, block_rows

    def t(self):
        """The transposed numbers, in the same memory (128 x 128 blocks only)."""
        if self.block_rows != BLOCK:
            raise ValueError("only codes in 128 x 128 blocks have a transpose")
        return BlockTensor(self.data.transpose(-1, -2), self.scale.transpose(-1, -2), BLOCK)


class ExpertPlan:
    """offsets (E + 1), counts (E), rows (P) and position (T, k), all int32 (see include/gemm_experts.h)."""
    __slots__ = ("offsets", "counts", "rows", "position", "align")

    def __init__(self, offsets, counts, rows, position, align=None):
        self.offsets, self.counts, self.rows, self.position, self.align = offsets, counts, rows, position, align


# ----------------------------------------------------------------------------- checks
# A call on a few tokens takes a few microseconds on the GPU, so what is looked up for every
# call is kept here: torch (imported with the first use) and its types' codes.
torch = None
_CODES, _WIDE = {}, {}
_raw_stream = _current_device = None


def _use_torch():
    global torch, _raw_stream, _current_device
    import torch as t
    _CODES.update({t.float8_e4m3fn: GEMM_E4M3, t.float8_e5m2: GEMM_E5M2})
    _WIDE.update({t.float32: _dg.GEMM_F32, t.float16: _dg.GEMM_F16, t.bfloat16: _dg.GEMM_BF16})
    _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: t.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t


def _code_type(dtype, what):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{what}: {dtype} is not float8_e4m3fn or float8_e5m2")
    return code


def _wide_type(dtype, what):
    code = _WIDE.get(dtype)
    if code is None:
        raise TypeError(f"{what}: {dtype} is not float32, float16 or bfloat16")
    return code


def _ld(shape, strides, what):
    """Leading dimension of rows that have to be contiguous: the last two dimensions of shape and strides."""
    cols = shape[-1]
    if strides[-1] != 1 and cols > 1:
        raise ValueError(f"{what} needs unit stride along its last dimension, not {tuple(strides)}")
    if shape[-2] <= 1:
        return cols or 1
    if strides[-2] < cols:
        raise ValueError(f"{what}: rows overlap (strides {tuple(strides)})")
    return strides[-2] or 1


def _matrix(t, what):
    """Leading dimension of a 2-D tensor with contiguous rows."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be 2-D, not {tuple(shape)}")
    return _ld(shape, t.stride(), what)


def _array(t, what, dtype, shape):
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous of shape {tuple(shape)}, not {tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _device(*tensors):
    """The index of the tensors' common GPU."""
    at = tensors[0].get_device()
    for t in tensors:
        if not t.is_cuda or t.get_device() != at:
            raise ValueError(f"tensors must be on one GPU, not {', '.join(str(t.device) for t in tensors)}")
    return at


def _block(b, what, dims=2):
    """A BlockTensor as the library takes it."""
    if not isinstance(b, BlockTensor):
        raise TypeError(f"{what} must be a BlockTensor, not {type(b).__name__}")
    data, scale, rows = b.data, b.scale, b.block_rows
    code = _CODES.get(data.dtype) or _code_type(data.dtype, f"{what}.data")
    shape, strides = data.shape, data.stride()
    if len(shape) != dims:
        raise ValueError(f"{what}.data must be {dims}-D, not {tuple(shape)}")
    R, K = shape[-2], shape[-1]
    op = 0
    if strides[-1] == 1 and strides[-2] >= K > 0 and R > 1:
        ld = strides[-2]
    elif (strides[-2] == 1 or R == 1) and strides[-1] != 1 and K > 1:
        ld, op = _ld((K, R), (strides[-1], 1), f"{what}.data"), 1
    else:
        ld = _ld(shape, strides, f"{what}.data")
    if rows != 1 and rows != BLOCK:
        raise ValueError(f"{what}.block_rows must be 1 or {BLOCK}, not {rows}")
    if scale.dtype != torch.float32:
        raise TypeError(f"{what}.scale must be float32, not {scale.dtype}")
    have = scale.shape
    if len(have) != dims or have[-2] != (R + rows - 1) // rows or have[-1] != (K + 127) // 128 or (
            dims == 3 and have[0] != shape[0]):
        want = (*shape[:-2], -(-R // rows), -(-K // BLOCK))
        raise ValueError(f"{what}.scale must have shape {want}, not {tuple(have)}")
    at = scale.stride()
    if dims == 3:
        return gemm_block_matrix(data.data_ptr(), scale.data_ptr(), R, K, ld, at[-2], at[-1], strides[0], at[0], code,
                                 rows, op, 0)
    return gemm_block_matrix(data.data_ptr(), scale.data_ptr(), R, K, ld, at[-2], at[-1], 0, 0, code, rows, op, 0)


def _plan(plan):
    """An ExpertPlan as the library takes it."""
    if not isinstance(plan, ExpertPlan):
        raise TypeError(f"plan must be an ExpertPlan, not {type(plan).__name__}")
    offsets, counts, rows, position = plan.offsets, plan.counts, plan.rows, plan.position
    if position.dim() != 2 or counts.dim() != 1 or rows.dim() != 1:
        raise ValueError("plan: position must be 2-D, counts and rows 1-D")
    i32 = torch.int32
    T, k = position.shape
    E, P = counts.shape[0], rows.shape[0]
    return gemm_expert_plan(_array(offsets, "plan.offsets", i32, (E + 1,)), _array(counts, "plan.counts", i32, (E,)),
                            _array(rows, "plan.rows", i32, (P,)), _array(position, "plan.position", i32, (T, k)),
                            E, T, k, P)


def _call(name, device, *args):
    """The library function on the current stream of GPU `device`."""
    fn = getattr(_dg._lib or _dg.library(), name)
    if device == _current_device():
        st = fn(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(device))
    if st:
        _dg._check(st, name)


# ----------------------------------------------------------------------------- block-scaled products
def _new_block(rows, cols, dtype, code, block_rows, device):
    """An empty BlockTensor, its scales laid out with the rows adjacent, and as the library takes it."""
    data = torch.empty((rows, cols), dtype=dtype, device=device)
    r = (rows + block_rows - 1) // block_rows
    scale = torch.empty_strided((r, (cols + 127) // 128), (1, r), dtype=torch.float32, device=device)
    return BlockTensor(data, scale, block_rows), gemm_block_matrix(
        data.data_ptr(), scale.data_ptr(), rows, cols, cols or 1, 1, r, 0, 0, code, block_rows, 0, 0)


def gemm_block_quantize_tensors(x, dtype, block_rows=1, natural=True, transposed=False, rows=None):
    """x (M, K) as (natural, transposed) BlockTensors of the float8 `dtype`, either None where not asked for.

    rows (int32, any length R): row i of the result is row rows[i] of x, zeros where rows[i] is negative
    or at least M.
    """
    if torch is None:
        _use_torch()
    ld = _matrix(x, "x")
    code, wide = _code_type(dtype, "dtype"), _wide_type(x.dtype, "x")
    if block_rows != 1 and block_rows != BLOCK:
        raise ValueError(f"block_rows must be 1 or {BLOCK}, not {block_rows}")
    if not natural and not transposed:
        raise ValueError("neither natural nor transposed is asked for")
    M, K = x.shape
    R, gather = M, None
    if rows is not None:
        R = rows.numel()
        gather = _array(rows, "rows", torch.int32, (R,))
        at = _device(x, rows)
    else:
        at = _device(x)
    dev = x.device
    q, nat = _new_block(R, K, dtype, code, block_rows, dev) if natural else (None, None)
    t, tr = _new_block(K, R, dtype, code, block_rows, dev) if transposed else (None, None)
    if R and K:
        _call("gemm_block_quantize", at, x.data_ptr(), M, K, ld, wide, gather, R, nat, tr)
    return q, t


def gemm_block_product_tensors(a, b, dtype=None):
    """C (M, N) = A B^T for BlockTensors a (M, K) and b (N, K), stored as `dtype` (bfloat16 by default)."""
    if torch is None:
        _use_torch()
    dtype = dtype or torch.bfloat16
    out = _wide_type(dtype, "dtype")
    A, B = _block(a, "a"), _block(b, "b")
    M, N, K = A.rows, B.rows, A.cols
    if K != B.cols:
        raise ValueError(f"shape mismatch: a {tuple(a.data.shape)}, b {tuple(b.data.shape)}")
    at = _device(a.data, a.scale, b.data, b.scale)
    dev = a.data.device
    c = torch.empty((M, N), dtype=dtype, device=dev)
    if M and N:
        n = (_dg._lib or _dg.library()).gemm_block_product_workspace(M, N, K)
        work = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        _call("gemm_block_product", at, A, B, c.data_ptr(), N, out, work.data_ptr() if n else None, n)
    return c


# ----------------------------------------------------------------------------- experts
def _logits(logits, router):
    if not isinstance(router, gemm_router):
        raise TypeError(f"router must be a gemm_router, not {type(router).__name__}")
    return _matrix(logits, "logits"), _wide_type(logits.dtype, "logits")


def gemm_experts_route_tensors(logits, router, bias=None):
    """(index, weight), int32 and float32 (T, k), of logits (T, E); bias: float32 (E), for the choice only."""
    if torch is None:
        _use_torch()
    ld, code = _logits(logits, router)
    T, E = logits.shape
    k = max(router.top_k, 0)
    b = None
    if bias is not None:
        b = _array(bias, "bias", torch.float32, (E,))
        at = _device(logits, bias)
    else:
        at = _device(logits)
    dev = logits.device
    index = torch.empty((T, k), dtype=torch.int32, device=dev)
    weight = torch.empty((T, k), dtype=torch.float32, device=dev)
    _call("gemm_experts_route", at, logits.data_ptr(), T, E, ld, code, router, b, index.data_ptr(), weight.data_ptr())
    return index, weight


def gemm_experts_route_backward_tensors(logits, router, index, weight_grad):
    """The gradient of the logits (their type) from that of the weights, the choice held fixed."""
    if torch is None:
        _use_torch()
    ld, code = _logits(logits, router)
    T, E = logits.shape
    i = _array(index, "index", torch.int32, (T, router.top_k))
    g = _array(weight_grad, "weight_grad", torch.float32, (T, router.top_k))
    at = _device(logits, index, weight_grad)
    grad = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
    _call("gemm_experts_route_backward", at, logits.data_ptr(), T, E, ld, code, router, i, g, grad.data_ptr(), E or 1)
    return grad


def gemm_experts_dispatch_tensors(index, experts, align=1):
    """The ExpertPlan of index (T, k): every expert's (token, slot) pairs in their order, an expert's
    first row at a multiple of `align` (128 where a gradient of the weights is wanted)."""
    if torch is None:
        _use_torch()
    if index.dim() != 2:
        raise ValueError(f"index must be 2-D, not {tuple(index.shape)}")
    T, k = index.shape
    i = _array(index, "index", torch.int32, (T, k))
    if experts < 1 or align < 1:
        raise ValueError(f"experts = {experts} and align = {align} must be positive")
    at = _device(index)
    dev = index.device
    lib = _dg._lib or _dg.library()
    P, n = lib.gemm_experts_capacity(T, k, experts, align), lib.gemm_experts_dispatch_workspace(T, k, experts)
    # the plan's arrays in one allocation; the workspace behind them
    E1, head = experts + 1, 2 * experts + 1
    buf = torch.empty(head + P + T * k + n // 4, dtype=torch.int32, device=dev)
    p0 = buf.data_ptr()
    offsets, counts, rows, position, _ = buf.split_with_sizes((E1, experts, P, T * k, n // 4))
    plan = ExpertPlan(offsets, counts, rows, position.view(T, k), align)
    c = gemm_expert_plan(p0, p0 + 4 * E1, p0 + 4 * head, p0 + 4 * (head + P), experts, T, k, P)
    _call("gemm_experts_dispatch", at, i, align, c, p0 + 4 * (head + P + T * k) if n else None, n)
    return plan


def gemm_experts_product_tensors(a, b, plan, dtype=None, gather=True):
    """C (P, N): each row of the plan times its expert's matrix, zeros in padding rows. b (E, N, K); a holds
    the tokens' rows (T, K) with gather, the plan's (P, K) without."""
    if torch is None:
        _use_torch()
    dtype = dtype or torch.bfloat16
    out = _wide_type(dtype, "dtype")
    A, B, p = _block(a, "a"), _block(b, "b", 3), _plan(plan)
    if A.cols != B.cols or b.data.shape[0] != p.experts or A.rows != (p.tokens if gather else p.capacity):
        raise ValueError(f"shape mismatch: a {tuple(a.data.shape)}, b {tuple(b.data.shape)}, plan of {p.experts} "
                         f"experts, {p.tokens} tokens and {p.capacity} rows")
    at = _device(a.data, a.scale, b.data, b.scale, plan.offsets, plan.counts, plan.rows)
    P, N = p.capacity, B.rows
    c = torch.empty((P, N), dtype=dtype, device=a.data.device)
    if P and N:
        _call("gemm_experts_product", at, A, B, p, int(gather), c.data_ptr(), N, out)
    return c


def gemm_experts_gradient_tensors(a, b, plan, dtype=None):
    """C (E, M, N) = A_e B_e^T over each expert's rows, for a (M, P) and b (N, P) with the plan's rows along
    their columns and zeros in padding, as gemm_block_quantize_tensors(..., transposed=True, rows=plan.rows)
    makes them. The plan's align has to be a multiple of 128; float32 by default."""
    if torch is None:
        _use_torch()
    dtype = dtype or torch.float32
    out = _wide_type(dtype, "dtype")
    A, B, p = _block(a, "a"), _block(b, "b"), _plan(plan)
    if A.cols != p.capacity or B.cols != p.capacity:
        raise ValueError(f"shape mismatch: a {tuple(a.data.shape)}, b {tuple(b.data.shape)}, plan of {p.capacity} rows")
    if plan.align is not None and plan.align % BLOCK:
        raise ValueError(f"the plan's align is {plan.align}, not a multiple of {BLOCK}")
    at = _device(a.data, a.scale, b.data, b.scale, plan.offsets)
    M, N = A.rows, B.rows
    c = torch.empty((p.experts, M, N), dtype=dtype, device=a.data.device)
    if p.experts and M and N:
        _call("gemm_experts_gradient", at, A, B, p, c.data_ptr(), N, M * N, out)
    return c


def _combine(y, plan, weight):
    p = _plan(plan)
    ld, code = _matrix(y, "y"), _wide_type(y.dtype, "y")
    if y.shape[0] != p.capacity:
        raise ValueError(f"y has {y.shape[0]} rows, the plan {p.capacity}")
    return p, ld, code, _array(weight, "weight", torch.float32, (p.tokens, p.top_k))


def gemm_experts_combine_tensors(y, plan, weight):
    """out (T, N) = the sum of each token's rows of y (P, N), weighted by weight (T, k) float32."""
    if torch is None:
        _use_torch()
    p, ld, code, w = _combine(y, plan, weight)
    at = _device(y, plan.position, weight)
    T, N = p.tokens, y.shape[1]
    out = torch.empty((T, N), dtype=y.dtype, device=y.device)
    if T and N:
        _call("gemm_experts_combine", at, y.data_ptr(), N, ld, code, p, w, out.data_ptr(), N)
    return out


def gemm_experts_combine_backward_tensors(y, plan, weight, grad):
    """(y_grad (P, N) of y's type, weight_grad (T, k) float32) from grad (T, N)."""
    if torch is None:
        _use_torch()
    p, ld, code, w = _combine(y, plan, weight)
    ldg = _matrix(grad, "grad")
    if grad.dtype != y.dtype or grad.shape != (p.tokens, y.shape[1]):
        raise ValueError(f"grad must be {y.dtype} of shape {(p.tokens, y.shape[1])}, not {grad.dtype} {tuple(grad.shape)}")
    at = _device(y, plan.position, plan.rows, weight, grad)
    N = y.shape[1]
    y_grad = torch.empty((p.capacity, N), dtype=y.dtype, device=y.device)
    weight_grad = torch.empty((p.tokens, p.top_k), dtype=torch.float32, device=y.device)
    _call("gemm_experts_combine_backward", at, y.data_ptr(), N, ld, code, p, w, grad.data_ptr(), ldg,
          y_grad.data_ptr(), N or 1, weight_grad.data_ptr())
    return y_grad, weight_grad

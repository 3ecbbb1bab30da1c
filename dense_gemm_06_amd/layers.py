"""Operators around a layer's dense products, for torch tensors.

The functions mirror include/gemm_layers.h: they check the tensors, allocate the results and
the workspace and pass pointers, strides and the current stream on; every step runs in the
library's HIP kernels. Results belong to the current stream of the tensors' device, and the
calls can be captured into a graph.

  gemm_adapters_tensors             x w^T with a low-rank term of each row's own adapter
  gemm_adapters_backward_tensors    its gradients
  gemm_loss_tensors                 softmax cross entropy of x w^T over a vocabulary
  gemm_loss_backward_tensors        its gradients, in pieces of the vocabulary
  gemm_activation_tensors           an activation, with or without a gate, and its input in 8 bits
  gemm_activation_backward_tensors  its gradient from the 8-bit codes
  gemm_activation_value_tensors     the activation again from the codes

Tensors need unit stride along their last dimension; other strides are free. Results carry no
gradient, also of tensors that require one: a training step calls the gradients' operators
itself (examples/adapter_step.py) or from its own torch.autograd.Function.
"""
from __future__ import annotations

import ctypes
import functools

import dense_gemm_06_amd as _dg

from . import experts as _ex
from .experts import (BlockTensor, _array, _block, _call, _device, _ld, _matrix, _new_block, _plan, _wide_type,
                      gemm_block_matrix, gemm_expert_plan)

GEMM_ACT_SILU = 3
_ACT_CODE = {"relu": _dg.GEMM_ACT_RELU, "gelu_tanh": _dg.GEMM_ACT_GELU_TANH, "silu": GEMM_ACT_SILU}

_i64, _vp = ctypes.c_int64, ctypes.c_void_p


class gemm_adapter_set(ctypes.Structure):
    """The adapters' matrices (see include/gemm_layers.h)."""
    _fields_ = [("a", _vp), ("b", _vp), ("scale", _vp), ("adapters", _i64), ("rank", _i64), ("lda", _i64),
                ("stride_a", _i64), ("ldb", _i64), ("stride_b", _i64)]


def declare(lib):
    """The argument types of include/gemm_layers.h's functions."""
    c_int = ctypes.c_int
    mat, ad, pl = ctypes.POINTER(gemm_block_matrix), ctypes.POINTER(gemm_adapter_set), ctypes.POINTER(gemm_expert_plan)
    for name, args, res in (
            ("gemm_adapters_product", [_vp, _i64, _i64, _i64, _vp, _i64, _i64, c_int, ad, _vp, _vp, _i64, _vp, _vp,
                                       _i64, _vp], c_int),
            ("gemm_adapters_workspace", [_i64, _i64, _i64, _i64, c_int], _i64),
            ("gemm_adapters_backward", [_vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, c_int, ad, _vp, pl,
                                        _vp, _i64, _vp, _vp, _vp, _i64, _vp], c_int),
            ("gemm_adapters_backward_workspace", [_i64, _i64, _i64, _i64, _i64, c_int], _i64),
            ("gemm_loss", [_vp, _i64, _i64, _i64, _vp, _i64, _i64, c_int, _vp, _vp, _vp, _vp, _i64, _vp], c_int),
            ("gemm_loss_workspace", [_i64, _i64, _i64, c_int], _i64),
            ("gemm_loss_backward", [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, c_int, _vp, _vp, _vp, _i64, _vp, _i64,
                                    _i64, _vp, _i64, _vp], c_int),
            ("gemm_loss_backward_workspace", [_i64, _i64, _i64, c_int, c_int, c_int, _i64], _i64),
            ("gemm_activation_forward", [_vp, _i64, _i64, _i64, c_int, c_int, c_int, _vp, _i64, mat, _vp], c_int),
            ("gemm_activation_backward", [mat, _vp, _i64, _i64, _i64, c_int, c_int, c_int, _vp, _i64, _vp, _i64, _vp],
             c_int)):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


torch = None


def _use_torch():
    global torch
    if _ex.torch is None:
        _ex._use_torch()
    torch = _ex.torch


def _lib():
    return _dg._lib or _dg.library()


@functools.lru_cache(maxsize=1024)
def _bytes(name, *sizes):
    """A workspace's size, which the call's sizes and type alone tell."""
    return getattr(_lib(), name)(*sizes)


def _work(n, device):
    """A workspace of n bytes, which the caller keeps until the call is made (None for 0), and its address."""
    if not n:
        return None, None
    work = torch.empty(n, dtype=torch.uint8, device=device)
    return work, work.data_ptr()


def _same(t, what, dtype, shape):
    """Leading dimension of a matrix of a given type and shape."""
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return _matrix(t, what)


# ----------------------------------------------------------------------------- adapters
def _batch(t, what):
    """Leading dimension and batch stride of a 3-D tensor."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{what} must be 3-D, not {tuple(shape)}")
    ld = strides[1] if strides[2] == 1 and strides[1] >= shape[2] > 0 and shape[1] > 1 else _ld(shape, strides, what)
    return ld, strides[0] if shape[0] > 1 else 0


def _adapters(x, w, a, b, index, scale):
    """The call's type, leading dimensions of x and w, the set, index's pointer and the sizes."""
    dt = x.dtype
    code = _wide_type(dt, "x")
    if w.dtype != dt or a.dtype != dt or b.dtype != dt:
        raise TypeError(f"x, w, a and b must share one dtype, not {dt}, {w.dtype}, {a.dtype} and {b.dtype}")
    ldx, ldw = _matrix(x, "x"), _matrix(w, "w")
    (lda, sa), (ldb, sb) = _batch(a, "a"), _batch(b, "b")
    (T, K), N = x.shape, w.shape[0]
    R, rank, Ka = a.shape
    if w.shape[1] != K or Ka != K or b.shape != (R, N, rank):
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}, a {tuple(a.shape)}, b {tuple(b.shape)}")
    i = _array(index, "index", torch.int32, (T,))
    if scale is None:
        s, at = None, _device(x, w, a, b, index)
    else:
        s, at = _array(scale, "scale", torch.float32, (R,)), _device(x, w, a, b, index, scale)
    adapters = gemm_adapter_set(a.data_ptr(), b.data_ptr(), s, R, rank, lda, sa, ldb, sb)
    return code, ldx, ldw, adapters, i, at, (T, N, K, R, rank)


def gemm_adapters_tensors(x, w, a, b, index, scale=None, keep=False):
    """y (T, N) = x w^T + scale_i (x a_i^T) b_i^T for x (T, K), w (N, K) and the adapter i = index[t] (int32, T) of
    each row, none where it lies outside 0 .. R-1. a (R, rank, K), b (R, N, rank), scale float32 (R) or None.
    With keep: (y, u), u (T, rank) float32 = x a_i^T, which the backward pass takes."""
    if torch is None:
        _use_torch()
    code, ldx, ldw, adapters, i, at, (T, N, K, R, rank) = _adapters(x, w, a, b, index, scale)
    dev = x.device
    y = torch.empty((T, N), dtype=x.dtype, device=dev)
    u = torch.empty((T, rank), dtype=torch.float32, device=dev) if keep else None
    if T:
        n = _bytes("gemm_adapters_workspace", T, N, K, rank, code)
        head = 0 if keep else -(-T * rank // 64) * 256  # u lies before the workspace where it is not kept
        work, wp = _work(head + n, dev)
        _call("gemm_adapters_product", at, x.data_ptr(), T, K, ldx, w.data_ptr(), N, ldw, code, adapters, i,
              y.data_ptr(), N or 1, u.data_ptr() if keep else wp, wp + head if n else None, n)
    return (y, u) if keep else y


def gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, plan, scale=None, x_grad=True):
    """(x_grad, a_grad, b_grad) of gemm_adapters_tensors(..., keep=True) from the gradient of y, x_grad None where
    not wanted. plan: gemm_experts_dispatch_tensors(index[:, None], R), which serves every layer of a batch (not read
    without adapters)."""
    if torch is None:
        _use_torch()
    code, ldx, ldw, adapters, i, at, (T, N, K, R, rank) = _adapters(x, w, a, b, index, scale)
    ldg = _same(grad, "grad", x.dtype, (T, N))
    up = _array(u, "u", torch.float32, (T, rank))
    p = None
    if R:
        p = _plan(plan)
        if p.experts != R or p.tokens != T or p.top_k != 1:
            raise ValueError(f"plan of {p.experts} experts, {p.tokens} tokens and top_k {p.top_k}, not of {R} "
                             f"adapters, {T} tokens and 1")
        _device(x, grad, u, plan.offsets, plan.counts, plan.rows)
    else:
        _device(x, grad, u)
    dev = x.device
    xg = torch.empty((T, K), dtype=x.dtype, device=dev) if x_grad else None
    ag = torch.empty((R, rank, K), dtype=x.dtype, device=dev)
    bg = torch.empty((R, N, rank), dtype=x.dtype, device=dev)
    n = _bytes("gemm_adapters_backward_workspace", T, N, K, R, rank, code)
    work, wp = _work(n, dev)
    _call("gemm_adapters_backward", at, grad.data_ptr(), T, N, ldg, x.data_ptr(), K, ldx, up, w.data_ptr(), ldw, code,
          adapters, i, p, xg.data_ptr() if x_grad else None, K or 1, ag.data_ptr(), bg.data_ptr(), wp, n)
    return xg, ag, bg


# ----------------------------------------------------------------------------- loss over a vocabulary
def _head(x, w, target):
    code = _wide_type(x.dtype, "x")
    ldx, ldw = _matrix(x, "x"), _matrix(w, "w")
    if w.dtype != x.dtype:
        raise TypeError(f"x and w must share one dtype, not {x.dtype} and {w.dtype}")
    if w.shape[1] != x.shape[1]:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}")
    return code, ldx, ldw, _array(target, "target", torch.int64, (x.shape[0],))


def gemm_loss_tensors(x, w, target):
    """(loss, lse), float32 (T): the softmax cross entropy of the logits x w^T for x (T, K), w (V, K) and target
    (T) int64, and the logarithm of their exponentials' sum. A target outside 0 .. V-1 gives loss 0. The logits
    are not kept."""
    if torch is None:
        _use_torch()
    code, ldx, ldw, t = _head(x, w, target)
    at = _device(x, w, target)
    (T, K), V, dev = x.shape, w.shape[0], x.device
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    if T:
        n = _bytes("gemm_loss_workspace", T, V, K, code)
        work, wp = _work(n, dev)
        _call("gemm_loss", at, x.data_ptr(), T, K, ldx, w.data_ptr(), V, ldw, code, t, loss.data_ptr(),
              lse.data_ptr(), wp, n)
    return loss, lse


def gemm_loss_backward_tensors(grad, x, w, target, lse, x_grad=True, w_grad=True, piece=0):
    """(x_grad, w_grad) from grad (T) float32, the gradient of gemm_loss_tensors' loss, and its lse; either is None
    where not wanted. The logits are computed again, `piece` columns of the vocabulary at a time (0: the library's
    choice)."""
    if torch is None:
        _use_torch()
    code, ldx, ldw, t = _head(x, w, target)
    (T, K), V, dev = x.shape, w.shape[0], x.device
    g, l = _array(grad, "grad", torch.float32, (T,)), _array(lse, "lse", torch.float32, (T,))
    at = _device(x, w, target, grad, lse)
    if piece < 0:
        raise ValueError(f"piece = {piece} must be non-negative")
    xg = torch.empty((T, K), dtype=x.dtype, device=dev) if x_grad else None
    wg = torch.empty((V, K), dtype=x.dtype, device=dev) if w_grad else None
    n = _bytes("gemm_loss_backward_workspace", T, V, K, code, int(x_grad), int(w_grad), piece)
    work, wp = _work(n, dev)
    _call("gemm_loss_backward", at, g, x.data_ptr(), T, K, ldx, w.data_ptr(), V, ldw, code, t, l,
          xg.data_ptr() if x_grad else None, K or 1, wg.data_ptr() if w_grad else None, K or 1, piece,
          wp, n)
    return xg, wg


# ----------------------------------------------------------------------------- activations
def _activation(activation):
    code = _ACT_CODE.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(_ACT_CODE)}, not {activation!r}")
    return code


def gemm_activation_tensors(z, activation, gated=False, dtype=None):
    """(y, codes): y = f(z), or f(z1) * z2 for gated z = [z1 | z2] along the columns, and z as a BlockTensor of the
    float8 `dtype` with block_rows 1 (None: codes is None). f: "relu", "gelu_tanh" or "silu"."""
    if torch is None:
        _use_torch()
    ld, wide, act = _matrix(z, "z"), _wide_type(z.dtype, "z"), _activation(activation)
    T, Z = z.shape
    if gated and Z % 2:
        raise ValueError(f"a gated z has an even number of columns, not {Z}")
    F = Z // 2 if gated else Z
    at, dev = _device(z), z.device
    y = torch.empty((T, F), dtype=z.dtype, device=dev)
    codes = c = None
    if dtype is not None:
        codes, c = _new_block(T, Z, dtype, _ex._code_type(dtype, "dtype"), 1, dev)
    if T and F:
        _call("gemm_activation_forward", at, z.data_ptr(), T, F, ld, wide, act, int(gated), y.data_ptr(), F, c)
    return y, codes


def gemm_activation_backward_tensors(grad, codes, activation, gated=False, value=True):
    """(z_grad, y) from grad (T, F), the gradient of y, and gemm_activation_tensors' codes: the gradient of z and
    y computed again from the codes (None without value), both of grad's type."""
    if torch is None:
        _use_torch()
    ld, wide, act = _matrix(grad, "grad"), _wide_type(grad.dtype, "grad"), _activation(activation)
    c = _block(codes, "codes")
    T, F = grad.shape
    Z = 2 * F if gated else F
    if (c.rows, c.cols) != (T, Z):
        raise ValueError(f"codes must be {(T, Z)} for grad {(T, F)}, not {(c.rows, c.cols)}")
    at, dev = _device(grad, codes.data, codes.scale), grad.device
    zg = torch.empty((T, Z), dtype=grad.dtype, device=dev)
    y = torch.empty((T, F), dtype=grad.dtype, device=dev) if value else None
    if T and F:
        _call("gemm_activation_backward", at, c, grad.data_ptr(), T, F, ld, wide, act, int(gated), zg.data_ptr(), Z,
              y.data_ptr() if value else None, F)
    return zg, y


def gemm_activation_value_tensors(codes, activation, gated=False, dtype=None):
    """y (T, F) computed again from gemm_activation_tensors' codes, of type dtype (bfloat16 by default): as the
    backward pass gives it, for where it is needed before the gradient of y is known."""
    if torch is None:
        _use_torch()
    dtype = dtype or torch.bfloat16
    wide, act, c = _wide_type(dtype, "dtype"), _activation(activation), _block(codes, "codes")
    T, Z = c.rows, c.cols
    if gated and Z % 2:
        raise ValueError(f"codes of a gated activation have an even number of columns, not {Z}")
    F = Z // 2 if gated else Z
    at, dev = _device(codes.data, codes.scale), codes.data.device
    y = torch.empty((T, F), dtype=dtype, device=dev)
    if T and F:
        _call("gemm_activation_backward", at, c, None, T, F, 0, wide, act, int(gated), None, 0, y.data_ptr(), F)
    return y

"""CPU tests of include/gemm_layers.h and its torch front: exported symbols, refusals before any
device access, host-side sizes. No kernel is launched."""
import ctypes
import os
import re

import pytest
import torch

import dense_gemm_06_amd as dg
from dense_gemm_06_amd import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4 = torch.float8_e4m3fn
OK, INVALID, NULL, UNSUPPORTED = 0, 1, 2, 3
G = 1 << 30  # distance between the made-up addresses: nothing overlaps


def lib():
    return dg.library()


def test_header_symbols_exported():
    src = open(os.path.join(ROOT, "include", "gemm_layers.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*(?:int|int64_t)\s+(gemm_\w+)\s*\(", src, flags=re.M))
    assert names == {"gemm_adapters_product", "gemm_adapters_workspace", "gemm_adapters_backward",
                     "gemm_adapters_backward_workspace", "gemm_loss", "gemm_loss_workspace", "gemm_loss_backward",
                     "gemm_loss_backward_workspace", "gemm_activation_forward", "gemm_activation_backward"}
    for n in names:
        assert hasattr(lib(), n), n


def adapters(**kw):
    s = dg.gemm_adapter_set(3 * G, 4 * G, 5 * G, 2, 16, 64, 16 * 64, 16, 32 * 16)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def forward(**kw):
    v = dict(x=G, T=8, K=64, ldx=64, w=2 * G, N=32, ldw=64, dtype=dg.GEMM_BF16, set=adapters(), index=6 * G, y=7 * G,
             ldy=32, u=8 * G, ws=9 * G, n=G)
    v.update(kw)
    s = ctypes.byref(v["set"]) if v["set"] is not None else None
    return lib().gemm_adapters_product(v["x"], v["T"], v["K"], v["ldx"], v["w"], v["N"], v["ldw"], v["dtype"], s,
                                       v["index"], v["y"], v["ldy"], v["u"], v["ws"], v["n"], None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(y=None)), (NULL, dict(u=None)), (NULL, dict(index=None)),
    (NULL, dict(set=None)), (NULL, dict(ws=None)), (INVALID, dict(n=16, dtype=dg.GEMM_F32)),
    (INVALID, dict(ws=9 * G + 4)),
    (INVALID, dict(dtype=3)), (INVALID, dict(ldx=63)), (INVALID, dict(ldw=63)), (INVALID, dict(ldy=31)),
    (INVALID, dict(T=-1)), (UNSUPPORTED, dict(T=1 << 31)), (UNSUPPORTED, dict(K=1 << 31)), (INVALID, dict(y=G)),
    (INVALID, dict(u=7 * G + 16)), (INVALID, dict(ws=2 * G)), (INVALID, dict(u=4 * G)), (INVALID, dict(y=6 * G)),
    (INVALID, dict(set=adapters(rank=0))), (INVALID, dict(set=adapters(rank=-1))),
    (UNSUPPORTED, dict(set=adapters(rank=129))), (NULL, dict(set=adapters(a=None))),
    (NULL, dict(set=adapters(b=None))), (INVALID, dict(set=adapters(lda=63))), (INVALID, dict(set=adapters(ldb=15))),
    (INVALID, dict(set=adapters(stride_a=-1))), (INVALID, dict(set=adapters(adapters=-1))), (UNSUPPORTED, dict(set=adapters(adapters=32769)))])
def test_adapters_refusals(want, kw):
    assert forward(**kw) == want
    assert dg.gemm_last_error()


def backward(**kw):
    v = dict(grad=G, T=8, N=32, ldg=32, x=2 * G, K=64, ldx=64, u=10 * G, w=11 * G, ldw=64, dtype=dg.GEMM_BF16,
             set=adapters(), index=6 * G, plan=dg.gemm_expert_plan(12 * G, 13 * G, 14 * G, 15 * G, 2, 8, 1, 8),
             x_grad=16 * G, ldxg=64, a_grad=17 * G, b_grad=18 * G, ws=19 * G, n=G)
    v.update(kw)
    p = ctypes.byref(v["plan"]) if v["plan"] is not None else None
    return lib().gemm_adapters_backward(v["grad"], v["T"], v["N"], v["ldg"], v["x"], v["K"], v["ldx"], v["u"], v["w"],
                                        v["ldw"], v["dtype"], ctypes.byref(v["set"]), v["index"], p, v["x_grad"],
                                        v["ldxg"], v["a_grad"], v["b_grad"], v["ws"], v["n"], None)


def plan(offsets=12 * G, counts=13 * G, rows=14 * G, experts=2, tokens=8, top_k=1, capacity=8):
    return dg.gemm_expert_plan(offsets, counts, rows, 15 * G, experts, tokens, top_k, capacity)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(grad=None)), (NULL, dict(x=None)), (NULL, dict(u=None)), (NULL, dict(w=None)), (NULL, dict(index=None)),
    (NULL, dict(plan=None)), (NULL, dict(a_grad=None)), (NULL, dict(b_grad=None)), (NULL, dict(ws=None)),
    (NULL, dict(plan=plan(offsets=None))), (NULL, dict(plan=plan(counts=None))), (NULL, dict(plan=plan(rows=None))),
    (INVALID, dict(plan=plan(experts=3))), (INVALID, dict(plan=plan(tokens=9))), (INVALID, dict(plan=plan(top_k=2))),
    (INVALID, dict(plan=plan(capacity=-1))), (INVALID, dict(plan=plan(capacity=9))), (INVALID, dict(n=16)), (INVALID, dict(ldg=31)), (INVALID, dict(ldxg=63)),
    (INVALID, dict(x_grad=G)), (INVALID, dict(a_grad=18 * G)), (INVALID, dict(b_grad=14 * G)), (INVALID, dict(ws=16 * G))])
def test_adapters_backward_refusals(want, kw):
    assert backward(**kw) == want
    assert dg.gemm_last_error()


def loss(**kw):
    v = dict(x=G, T=8, K=64, ldx=64, w=2 * G, V=100, ldw=64, dtype=dg.GEMM_F16, target=3 * G, loss=4 * G, lse=5 * G,
             ws=6 * G, n=G)
    v.update(kw)
    return lib().gemm_loss(v["x"], v["T"], v["K"], v["ldx"], v["w"], v["V"], v["ldw"], v["dtype"], v["target"],
                           v["loss"], v["lse"], v["ws"], v["n"], None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(target=None)), (NULL, dict(loss=None)), (NULL, dict(lse=None)),
    (NULL, dict(ws=None)), (INVALID, dict(n=0)), (INVALID, dict(ws=6 * G + 8)), (INVALID, dict(dtype=-1)),
    (INVALID, dict(ldx=1)), (INVALID, dict(ldw=1)), (INVALID, dict(V=-1)), (UNSUPPORTED, dict(V=1 << 31)),
    (INVALID, dict(lse=4 * G + 16)), (INVALID, dict(loss=3 * G)), (INVALID, dict(ws=2 * G))])
def test_loss_refusals(want, kw):
    assert loss(**kw) == want
    assert dg.gemm_last_error()


def loss_backward(**kw):
    v = dict(grad=10 * G, x=G, T=8, K=64, ldx=64, w=2 * G, V=100, ldw=64, dtype=dg.GEMM_F16, target=3 * G, lse=5 * G,
             x_grad=7 * G, ldxg=64, w_grad=8 * G, ldwg=64, piece=0, ws=6 * G, n=G)
    v.update(kw)
    return lib().gemm_loss_backward(v["grad"], v["x"], v["T"], v["K"], v["ldx"], v["w"], v["V"], v["ldw"], v["dtype"],
                                    v["target"], v["lse"], v["x_grad"], v["ldxg"], v["w_grad"], v["ldwg"], v["piece"],
                                    v["ws"], v["n"], None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(grad=None)), (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(target=None)), (NULL, dict(lse=None)),
    (NULL, dict(ws=None)), (INVALID, dict(n=64)), (INVALID, dict(piece=-1)), (INVALID, dict(ldxg=63)),
    (INVALID, dict(ldwg=63)), (INVALID, dict(x_grad=8 * G)), (INVALID, dict(w_grad=2 * G)), (INVALID, dict(ws=G))])
def test_loss_backward_refusals(want, kw):
    assert loss_backward(**kw) == want
    assert dg.gemm_last_error()


def mat(rows, cols, **kw):
    m = dg.gemm_block_matrix(2 * G, 3 * G, rows, cols, cols, 1, rows, 0, 0, dg.GEMM_E4M3, 1)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


def act(**kw):
    v = dict(z=G, T=8, F=64, ldz=128, dtype=dg.GEMM_BF16, act=3, gated=1, y=4 * G, ldy=64, codes=mat(8, 128))
    v.update(kw)
    c = ctypes.byref(v["codes"]) if v["codes"] is not None else None
    return lib().gemm_activation_forward(v["z"], v["T"], v["F"], v["ldz"], v["dtype"], v["act"], v["gated"], v["y"],
                                         v["ldy"], c, None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(z=None)), (NULL, dict(y=None)), (INVALID, dict(act=0)), (INVALID, dict(act=4)), (INVALID, dict(dtype=9)),
    (INVALID, dict(ldz=127)), (INVALID, dict(ldy=63)), (INVALID, dict(codes=mat(8, 64))), (INVALID, dict(codes=mat(9, 128))),
    (INVALID, dict(codes=mat(8, 128, block_rows=128))), (UNSUPPORTED, dict(codes=mat(8, 128, op=1))),
    (NULL, dict(codes=mat(8, 128, data=None))), (INVALID, dict(y=G)), (INVALID, dict(y=2 * G)), (INVALID, dict(y=3 * G)),
    (UNSUPPORTED, dict(F=(1 << 30) + 1, ldz=1 << 32, ldy=1 << 32)), (INVALID, dict(T=-1))])
def test_activation_refusals(want, kw):
    assert act(**kw) == want
    assert dg.gemm_last_error()


def act_backward(**kw):
    v = dict(codes=mat(8, 128), grad=G, T=8, F=64, ldg=64, dtype=dg.GEMM_BF16, act=3, gated=1, z_grad=4 * G, ldzg=128,
             y=5 * G, ldy=64)
    v.update(kw)
    c = ctypes.byref(v["codes"]) if v["codes"] is not None else None
    return lib().gemm_activation_backward(c, v["grad"], v["T"], v["F"], v["ldg"], v["dtype"], v["act"], v["gated"],
                                          v["z_grad"], v["ldzg"], v["y"], v["ldy"], None)


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(codes=None)), (NULL, dict(grad=None)), (NULL, dict(z_grad=None)), (INVALID, dict(ldg=63)),
    (INVALID, dict(ldzg=127)), (INVALID, dict(ldy=63)), (INVALID, dict(y=4 * G)), (INVALID, dict(z_grad=G)),
    (INVALID, dict(z_grad=2 * G)), (INVALID, dict(codes=mat(8, 64))), (INVALID, dict(codes=mat(8, 128, dtype=0)))])
def test_activation_backward_refusals(want, kw):
    assert act_backward(**kw) == want
    assert dg.gemm_last_error()


def test_empty_calls_need_no_device():
    assert forward(T=0, x=None, y=None) == OK
    assert loss(T=0) == OK and loss_backward(K=0, ldx=64) == OK and loss_backward(x_grad=None, w_grad=None) == OK
    assert act(T=0, codes=mat(0, 128)) == OK


@pytest.mark.parametrize("call,kw", [(c, kw) for c, names in (
    (forward, ("ldx", "ldw")), (backward, ("ldg", "ldx", "ldw")), (loss, ("ldx", "ldw")), (loss_backward, ("ldx", "ldw")))
    for kw in [{n: 1 << 23} for n in names] + [{"T": 1 << 30}, {"K": 1 << 30, "ldx": 1 << 30, "ldw": 1 << 30, "ldxg": 1 << 30, "ldwg": 1 << 30, "set": adapters(lda=1 << 30)}]])
def test_product_limits(call, kw):
    """Operands whose rows lie too far apart for the products' 32-bit offsets, whatever form would take them."""
    for T in (8, 100, 5000):
        assert call(**{"T": T, "n": 1 << 60, **kw}) == UNSUPPORTED
        assert "2^" in dg.gemm_last_error()


def test_adapter_limits():
    for call in (forward, backward):
        assert call(set=adapters(lda=1 << 23)) == call(set=adapters(ldb=1 << 23)) == UNSUPPORTED
    assert loss_backward(T=(1 << 23) - 31) == UNSUPPORTED and "w_grad" in dg.gemm_last_error()


def test_workspaces():
    assert lib().gemm_loss_workspace(-1, 5, 5, 0) == 0 and lib().gemm_adapters_workspace(1, 1, 1, 1, 7) == 0
    small = lib().gemm_loss_backward_workspace(4096, 65536, 1024, dg.GEMM_BF16, 1, 1, 1024)
    large = lib().gemm_loss_backward_workspace(4096, 65536, 1024, dg.GEMM_BF16, 1, 1, 65536)
    assert 0 < small < large
    # far less than the logits in fp32 hold
    assert lib().gemm_loss_workspace(32768, 262144, 1024, dg.GEMM_BF16) < 32768 * 262144 * 4 // 8


# ----------------------------------------------------------------------------- the torch front
def test_front_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    a, b, index = torch.zeros(2, 3, 8), torch.zeros(2, 6, 3), torch.zeros(4, dtype=torch.int32)
    call = dg.gemm_adapters_tensors
    with pytest.raises(ValueError, match="one GPU"):
        call(x, w, a, b, index)
    with pytest.raises(TypeError, match="share one dtype"):
        call(x, w.half(), a, b, index)
    with pytest.raises(ValueError, match="shape mismatch"):
        call(x, w, a, torch.zeros(2, 5, 3), index)
    with pytest.raises(TypeError, match="int32"):
        call(x, w, a, b, index.long())
    with pytest.raises(ValueError, match="unit stride"):
        call(torch.zeros(8, 4).t(), w, a, b, index)
    with pytest.raises(TypeError, match="float32"):
        call(x, w, a, b, index, torch.ones(2, dtype=torch.float64))
    with pytest.raises(TypeError, match="int64"):
        dg.gemm_loss_tensors(x, w, index)
    with pytest.raises(ValueError, match="one GPU"):
        dg.gemm_loss_tensors(x, w, index.long())
    with pytest.raises(ValueError, match="shape mismatch"):
        dg.gemm_loss_tensors(x, torch.zeros(6, 7), index.long())
    with pytest.raises(ValueError, match="activation"):
        dg.gemm_activation_tensors(x, "tanh")
    with pytest.raises(ValueError, match="even"):
        dg.gemm_activation_tensors(torch.zeros(4, 7), "silu", True)
    with pytest.raises(TypeError, match="float8"):
        dg.gemm_activation_tensors(x.cuda() if torch.cuda.is_available() else x, "silu", True, torch.int8) \
            if torch.cuda.is_available() else layers._ex._code_type(torch.int8, "dtype")
    with pytest.raises(TypeError, match="BlockTensor"):
        dg.gemm_activation_backward_tensors(x, x, "silu")

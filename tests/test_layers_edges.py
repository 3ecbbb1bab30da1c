"""CPU tests of include/gemm_layers.h at the edges of its sizes and arguments. No kernel is launched; a
call that would be made gives GEMM_ERR_DEVICE where there is no GPU, and is not made where there is one."""
import ctypes

import pytest
import torch

import dense_gemm_06_amd as dg

OK, INVALID, NULL, UNSUPPORTED, DEVICE = 0, 1, 2, 3, 4
TYPES = (dg.GEMM_F32, dg.GEMM_F16, dg.GEMM_BF16)
G = 1 << 40  # distance between the made-up addresses: nothing overlaps


def lib():
    return dg.library()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0, 1, 16, 17, 20, 64, 65, 300, 5000])
def test_adapters_workspaces_of_empty_sizes(T, dtype):
    for N in (0, 1, 64):
        for K in (0, 1, 8, 64):
            for R, rank in ((0, 0), (0, 5), (1, 1), (3, 16), (2, 128)):
                assert lib().gemm_adapters_workspace(T, N, K, rank, dtype) >= 0
                assert lib().gemm_adapters_backward_workspace(T, N, K, R, rank, dtype) >= 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [0, 1, 65, 300])
def test_loss_workspaces_of_empty_sizes(T, dtype):
    for V in (0, 1, 7, 300):
        for K in (0, 1, 8, 64):
            assert lib().gemm_loss_workspace(T, V, K, dtype) >= 0
            for want in ((0, 0), (0, 1), (1, 0), (1, 1)):
                for piece in (0, 1, 1000):
                    assert lib().gemm_loss_backward_workspace(T, V, K, dtype, *want, piece) >= 0


def adapters_backward(**kw):
    v = dict(T=8, N=32, K=64, ld=64, dtype=dg.GEMM_BF16, x_grad=None, a_grad=7 * G, b_grad=8 * G, R=2, rank=16)
    v.update(kw)
    s = dg.gemm_adapter_set(G, 2 * G, None, v["R"], v["rank"], v["ld"], 0, v["ld"], 0)
    plan = dg.gemm_expert_plan(3 * G, 4 * G, 5 * G, 6 * G, v["R"], v["T"], 1, v["T"])
    return lib().gemm_adapters_backward(9 * G, v["T"], v["N"], v["ld"], 10 * G, v["K"], v["ld"], 11 * G, 12 * G, v["ld"],
                                        v["dtype"], ctypes.byref(s), 13 * G, ctypes.byref(plan), v["x_grad"], v["ld"],
                                        v["a_grad"], v["b_grad"], 14 * G, G, None)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_of_the_adapters_gradients_missing(dtype):
    """Also beside an empty one, whose pointer may be anything."""
    for kw in (dict(a_grad=None), dict(b_grad=None), dict(a_grad=None, N=0), dict(b_grad=None, K=0)):
        assert adapters_backward(dtype=dtype, **kw) == NULL, kw
        assert "come together" in dg.gemm_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("dtype", TYPES)
def test_an_empty_gradient_needs_no_pointer(dtype):
    for kw in (dict(a_grad=None, K=0), dict(b_grad=None, N=0)):
        assert adapters_backward(dtype=dtype, **kw) == DEVICE, kw


def adapters_forward(**kw):
    v = dict(T=8, N=32, K=64, ld=64, dtype=dg.GEMM_BF16, R=2, rank=16)
    v.update(kw)
    s = dg.gemm_adapter_set(G, 2 * G, None, v["R"], v["rank"], v["ld"], 0, v["ld"], 0)
    return lib().gemm_adapters_product(9 * G, v["T"], v["K"], v["ld"], 12 * G, v["N"], v["ld"], v["dtype"], ctypes.byref(s),
                                       13 * G, 10 * G, v["N"], 11 * G, 14 * G, G, None)


def test_more_threads_than_a_launch_holds():
    """Refused before anything is enqueued: 16 tokens to 512 threads for rows of odd lengths, 32 tokens by 64
    columns to 256, 16 columns to 512 for few tokens."""
    for call, kw in ((adapters_forward, dict(T=1 << 27, K=9, ld=65)), (adapters_backward, dict(T=1 << 27, N=9, ld=65, a_grad=None, b_grad=None)),
                     (adapters_forward, dict(T=1 << 20, N=1 << 15, rank=65, ld=72)),
                     (adapters_backward, dict(T=1 << 20, K=1 << 15, rank=65, ld=1 << 15, x_grad=15 * G)),
                     (adapters_forward, dict(T=1, N=1 << 27, ld=65))):
        assert call(**kw) == UNSUPPORTED, kw
        assert "threads" in dg.gemm_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
@pytest.mark.parametrize("dtype", TYPES)
def test_many_tokens_of_a_high_rank(dtype):
    """What a launch holds is not refused: a million tokens of rank 64, and y of 2^35 elements in tiles."""
    assert adapters_forward(T=1 << 20, rank=64, dtype=dtype) == DEVICE
    assert adapters_backward(T=1 << 20, rank=64, dtype=dtype, x_grad=15 * G) == DEVICE
    assert adapters_forward(T=1 << 20, N=1 << 15, rank=64, dtype=dtype) == DEVICE


def test_workspace_of_the_adapters_backward_pass():
    """x's gradient in fp32 once, not once for every slice of k that only the forward pass cuts."""
    T, N, K, rank = 512, 8192, 2048, 16
    rest = lib().gemm_adapters_backward_workspace(T, N, 0, 4, rank, dg.GEMM_BF16)  # without x's gradient and a's
    whole = lib().gemm_adapters_backward_workspace(T, N, K, 4, rank, dg.GEMM_BF16)
    slots = 4 + T // 64
    assert whole - rest <= T * K * 4 + 4 * K * rank * 2 + slots * rank * K * 4 + 4096


def test_workspaces_of_the_largest_sizes():
    """No wrap at the largest sizes that the calls take, and 0 for sizes that they refuse."""
    L = lib()
    top, over = (1 << 30) - 1, 1 << 30
    for dtype in TYPES:
        ad, back = L.gemm_adapters_workspace, L.gemm_adapters_backward_workspace
        assert ad(top, top, top, 128, dtype) > (0 if dtype == dg.GEMM_F32 else top)  # fp32: the product's alone
        assert back(top, top, top, 32768, 128, dtype) > 128 * top
        for T, N, K in ((over, 1, 1), (1, over, 1), (1, 1, over), (-1, 1, 1)):
            assert ad(T, N, K, 1, dtype) == back(T, N, K, 1, 1, dtype) == 0
            assert L.gemm_loss_workspace(T, N, K, dtype) == L.gemm_loss_backward_workspace(T, N, K, dtype, 1, 1, 0) == 0
        assert ad(1, 1, 1, 129, dtype) == ad(1, 1, 1, 2 ** 31 - 1, dtype) == ad(1, 1, 1, -1, dtype) == 0
        assert back(top, top, top, 2 ** 31 - 1, 2 ** 31 - 1, dtype) == back(1, 1, 1, 32769, 1, dtype) == 0
        assert L.gemm_loss_workspace(top, top, top, dtype) > top
        assert L.gemm_loss_backward_workspace(top, top, top, dtype, 1, 0, 0) > top
        assert L.gemm_loss_backward_workspace(top, top, top, dtype, 1, 1, 2 ** 31 - 1) > top
        assert L.gemm_loss_backward_workspace(1, 1, 1, dtype, 1, 1, -1) == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [65537, 70000, 131073, 140000, 262145, 1000001])
def test_pieces_of_many_tokens(T, dtype):
    """A piece of the vocabulary has 256 columns at least, however many tokens there are."""
    V, K, es = 50000, 8, 4 if dtype == dg.GEMM_F32 else 2
    d = T * 256 * es
    assert lib().gemm_loss_backward_workspace(T, V, K, dtype, 1, 0, 0) >= d
    assert lib().gemm_loss_workspace(T, V, 4, dtype) >= T * 256 * 4  # the logits' own piece


def test_batches_of_single_rows():
    """The stride of a matrix's only row is anything: adapters of rank 1 stored as 1 x R x K."""
    a = torch.empty(1, 3, 2 ** 22, device="meta").transpose(0, 1)
    assert a.stride(1) > 2 ** 23 and dg.layers._batch(a, "a") == (2 ** 22, 2 ** 22)
    b = torch.empty(4, 1, 8)
    assert dg.layers._batch(b, "b") == (8, 8)

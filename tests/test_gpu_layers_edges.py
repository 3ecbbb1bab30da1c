"""The adapters, the loss and the activations on the GPU at the edges of what their documentation
allows: sets without adapters in every form, small and large numbers, infinities and NaN."""
import pytest
import torch

import dense_gemm_06_amd as dg
import layer_util as lu

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, size=1.0, dt=F32):
    return (torch.randn(*shape, generator=g) * size).to(dt).cuda()


# ----------------------------------------------------------------------------- adapters
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("rank", [0, 8])
@pytest.mark.parametrize("T,N,K", [(20, 96, 64), (2049, 4096, 64), (2049, 64, 4096)])
def test_no_adapters_in_any_form(T, N, K, rank, dt):
    """A set without adapters, of rank 0 too, in tiles of y and of x's gradient: the shared product alone."""
    g = gen(T + N)
    x, w, grad = normal(g, T, K, dt=dt), normal(g, N, K, size=0.05, dt=dt), normal(g, T, N, size=0.1, dt=dt)
    a, b = torch.zeros(0, rank, K, dtype=dt).cuda(), torch.zeros(0, N, rank, dtype=dt).cuda()
    index = torch.randint(-1, 3, (T,), generator=g, dtype=torch.int32).cuda()
    y, u = dg.gemm_adapters_tensors(x, w, a, b, index, None, keep=True)
    ref, err, _, _ = lu.adapters(x, w, a, b, index, None)
    lu.check(y, ref, err, "y")
    assert u.shape == (T, rank) and not u.any()
    xg, ag, bg = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, None)
    lu.check(xg, *lu.adapters_backward(grad, x, u, w, a, b, index, None)[0], "x_grad")
    assert ag.shape == a.shape and bg.shape == b.shape


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T", [1, 16, 20, 64, 70])
def test_adapters_without_columns(T, dt):
    """An empty y: u is written all the same."""
    g = gen(T)
    x, w, a, b = normal(g, T, 64, dt=dt), normal(g, 0, 64, dt=dt), normal(g, 3, 16, 64, dt=dt), normal(g, 3, 0, 16, dt=dt)
    index = torch.randint(-1, 3, (T,), generator=g, dtype=torch.int32).cuda()
    y, u = dg.gemm_adapters_tensors(x, w, a, b, index, None, keep=True)
    _, _, ref, err = lu.adapters(x, w, a, b, index, None)
    assert y.shape == (T, 0)
    lu.check(u, ref, err, "u")


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_adapters_of_a_million_tokens(dt):
    """2^20 tokens of rank 64: what one launch with a wave to each token and rank number would not hold."""
    T, N, K, R, rank = 2 ** 20, 8, 8, 2, 64
    g = gen(1)
    x, w, grad = normal(g, T, K, dt=dt), normal(g, N, K, dt=dt), normal(g, T, N, size=0.1, dt=dt)
    a, b = normal(g, R, rank, K, size=0.3, dt=dt), normal(g, R, N, rank, size=0.3, dt=dt)
    index = torch.randint(-1, R, (T,), generator=g, dtype=torch.int32).sort().values.cuda()
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), R)
    y, u = dg.gemm_adapters_tensors(x, w, a, b, index, None, keep=True)
    ref, err, _, _ = lu.adapters(x, w, a, b, index, None)
    lu.check(y, ref, err, "y")
    got = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, plan)
    for name, have, (ref, err) in zip(("x_grad", "a_grad", "b_grad"), got,
                                      lu.adapters_backward(grad, x, u, w, a, b, index, None)):
        lu.check(have, ref, err, name)


def kept_to(of):
    """How far a number v held as two fp16 numbers after a power of two may be off: 2^-22 of itself and half of
    fp16's smallest step, 2^-25, of a unit that brings the largest number that shares it to 2^14 .. 2^15 (`of` gives
    that number for each v): 2^-39 of it. Numbers brought to a common unit afterwards round hi and lo twice more."""
    return lambda v, dt: v.abs() * 2.0 ** -21 + of(v.abs()) * 2.0 ** -37


ROW = kept_to(lambda v: v.amax(1, keepdim=True))   # a token's own unit
ALL = kept_to(lambda v: v.amax())                  # one unit for an adapter's tokens


@pytest.mark.parametrize("T,N,K,R,rank", [(1, 256, 256, 2, 16), (20, 256, 264, 3, 3), (100, 256, 264, 3, 16),
                                          (100, 256, 264, 2, 40), (70, 256, 256, 2, 100), (700, 256, 256, 3, 16),
                                          (700, 251, 203, 3, 33), (700, 256, 256, 2, 128), (2100, 4096, 64, 3, 24),
                                          (2100, 64, 4096, 3, 64)])
@pytest.mark.parametrize("x,a,b,g", [(1.0, 0.06, 1e-4, 1e-3), (1.0, 0.06, 1e-4, 2.0 ** -12), (1e-3, 1e-5, 100.0, 100.0),
                                     (100.0, 50.0, 1e-5, 1e-4)])
@pytest.mark.parametrize("mixed", [False, True])
def test_adapters_of_small_and_large_numbers_in_fp16(x, a, b, g, T, N, K, R, rank, mixed, monkeypatch):
    """u and v far outside of what fp16 holds, and tokens of very different sizes side by side, keep their digits."""
    r = gen(T + rank)
    size = 2.0 ** -torch.randint(0, 12, (T, 1), generator=r).float() if mixed else torch.ones(T, 1)
    X = (torch.randn(T, K, generator=r) * x * size).half().cuda()
    G = (torch.randn(T, N, generator=r) * g * size.flip(0)).half().cuda()
    W, A, B = normal(r, N, K, size=0.05, dt=F16), normal(r, R, rank, K, size=a, dt=F16), normal(r, R, N, rank, size=b, dt=F16)
    scale = torch.rand(R, generator=r).cuda() + 0.5
    index = torch.randint(-1, R, (T,), generator=r, dtype=torch.int32)
    index = (index.sort().values if T > 1000 else index).cuda()
    y, u = dg.gemm_adapters_tensors(X, W, A, B, index, scale, keep=True)
    monkeypatch.setattr(lu, "kept_as", ROW)
    ref, err, u_ref, u_err = lu.adapters(X, W, A, B, index, scale)
    lu.check(u, u_ref, u_err, "u")
    lu.check(y, ref, err, "y")
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), R)
    xg, ag, bg = dg.gemm_adapters_backward_tensors(G, X, u, W, A, B, index, plan, scale)
    lu.check(xg, *lu.adapters_backward(G, X, u, W, A, B, index, scale)[0], "x_grad")
    monkeypatch.setattr(lu, "kept_as", ALL)
    _, wa, wb = lu.adapters_backward(G, X, u, W, A, B, index, scale)
    lu.check(ag, *wa, "a_grad")
    lu.check(bg, *wb, "b_grad")


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,N,K,rank", [(1, 256, 256, 16), (40, 256, 264, 12), (40, 255, 131, 12), (100, 256, 264, 16),
                                        (700, 256, 256, 16), (700, 251, 203, 33), (700, 256, 256, 128), (2100, 4096, 64, 24),
                                        (2100, 64, 4096, 64)])
def test_infinities_of_adapters(T, N, K, rank, dt):
    """An infinite weight of an adapter, or element of x or of y's gradient, makes results infinite, with the sign of
    what it is multiplied by, and leaves the others as they were."""
    R, g, inf = 2, gen(T + rank), float("inf")
    x, w, grad = normal(g, T, K, dt=dt), normal(g, N, K, size=0.05, dt=dt), normal(g, T, N, size=0.1, dt=dt)
    a, b = normal(g, R, rank, K, size=0.1, dt=dt), normal(g, R, N, rank, size=0.1, dt=dt)
    index = (torch.arange(T) * 3 // T - 1).abs().int().cuda()  # runs of adapters 1, 0 and 1
    scale = torch.tensor([0.75, 1.5]).cuda()
    mine = index == 1
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), R)
    y, u = dg.gemm_adapters_tensors(x, w, a, b, index, scale, keep=True)
    grads = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, plan, scale)
    v = grad.double() @ b[1].double()
    j = rank - 1

    def check(have, plain, where, of, what):
        want = plain.clone()
        want[where] = (of.sign() * inf).to(dt)
        assert torch.equal(have, want), what

    b2 = b.clone()
    b2[1, N - 2, j] = inf
    at = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    at[mine, N - 2] = True
    have, u2 = dg.gemm_adapters_tensors(x, w, a, b2, index, scale, keep=True)
    check(have, y, at, u[mine, j], "y")
    assert torch.equal(u2, u)

    a2 = a.clone()
    a2[1, j, K - 3] = -inf
    at = torch.zeros(T, K, dtype=torch.bool, device="cuda")
    at[mine, K - 3] = True
    have = dg.gemm_adapters_backward_tensors(grad, x, u, w, a2, b, index, plan, scale)
    check(have[0], grads[0], at, -v[mine, j], "x_grad")
    assert torch.equal(have[1], grads[1]) and torch.equal(have[2], grads[2])

    t = int(mine.nonzero()[0])
    x2 = x.clone()
    x2[t, K - 3] = inf
    at = torch.zeros(R, rank, K, dtype=torch.bool, device="cuda")
    at[1, :, K - 3] = True
    have = dg.gemm_adapters_backward_tensors(grad, x2, u, w, a, b, index, plan, scale)
    check(have[1], grads[1], at, v[t], "a_grad")
    assert torch.equal(have[0], grads[0]) and torch.equal(have[2], grads[2])

    grad2 = grad.clone()
    grad2[t, N - 2] = -inf
    at = torch.zeros(R, N, rank, dtype=torch.bool, device="cuda")
    at[1, N - 2] = True
    have = dg.gemm_adapters_backward_tensors(grad2, x, u, w, a, b, index, plan, scale)
    check(have[2], grads[2], at, -u[t], "b_grad")


# ----------------------------------------------------------------------------- loss
@pytest.mark.parametrize("T,dt", [(66001, F32), (131101, BF16)])
def test_loss_of_many_tokens(T, dt):
    """So many tokens that a piece of the vocabulary is a single block of columns."""
    V, K = 270, 8
    g = gen(2)
    x, w = normal(g, T, K, dt=dt), normal(g, V, K, dt=dt)
    target, grad = torch.randint(-9, V, (T,), generator=g).cuda(), torch.rand(T, generator=g).cuda()
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    ref, err, lse_ref, lse_err, _, _ = lu.loss(x, w, target)
    lu.check(lse, lse_ref, lse_err, "lse")
    lu.check(loss, ref, err, "loss")
    for name, have, (ref, err) in zip(("x_grad", "w_grad"), dg.gemm_loss_backward_tensors(grad, x, w, target, lse),
                                      lu.loss_backward(grad, x, w, target, lse)):
        lu.check(have, ref, err, name)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,V,K", [(0, 9, 8), (0, 0, 8), (0, 9, 0), (5, 9, 0), (5, 0, 8), (5, 0, 0), (70, 9, 0), (70, 0, 64)])
def test_loss_of_empty_sizes(T, V, K, dt):
    """Without a sum's terms every logit is 0; without words lse is -inf and no target counts."""
    x, w = torch.zeros(T, K, dtype=dt, device="cuda"), torch.zeros(V, K, dtype=dt, device="cuda")
    target, grad = torch.arange(T).cuda() % 5, torch.ones(T, device="cuda")
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    want = torch.logsumexp(torch.zeros(T, V, dtype=torch.float64), 1)
    # a logarithm of a whole number: four steps of it
    lu.check(lse, want, want.abs().nan_to_num(posinf=0) * 4 * lu.F32, "lse")
    lu.check(loss, want if V else torch.zeros(T).double(), want.abs().nan_to_num(posinf=0) * 4 * lu.F32, "loss")
    for name, have, like in zip(("x_grad", "w_grad"), dg.gemm_loss_backward_tensors(grad, x, w, target, lse), (x, w)):
        assert have.shape == like.shape and have.dtype == dt and not have.any(), name


# ----------------------------------------------------------------------------- activations
@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("kind", ["relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_activation_of_a_nan(gated, kind, dt):
    """A NaN in z is one in y, and one in the codes in everything that is computed from them."""
    F = 256
    z = normal(gen(3), 5, 2 * F if gated else F, dt=dt)
    plain, _ = dg.gemm_activation_tensors(z, kind, gated, torch.float8_e4m3fn)
    z[1, 7] = float("nan")
    y, codes = dg.gemm_activation_tensors(z, kind, gated, torch.float8_e4m3fn)
    same = torch.ones_like(y, dtype=torch.bool)
    same[1, 7] = False
    assert y[1, 7].isnan() and torch.equal(y[same], plain[same])
    held = codes.data.float()[:, :F].isnan()
    assert held[1, 7] and not held[0].any()
    grad = normal(gen(4), 5, F, dt=dt)
    zg, again = dg.gemm_activation_backward_tensors(grad, codes, kind, gated)
    assert torch.equal(again.isnan(), held) and torch.equal(zg[:, :F].isnan(), held)
    assert torch.equal(dg.gemm_activation_value_tensors(codes, kind, gated, dt).isnan(), held)


def test_relu_of_infinities():
    z = torch.tensor([[float("inf"), float("-inf"), 0.0, -1.0, 2.0]]).cuda()
    assert torch.equal(dg.gemm_activation_tensors(z, "relu")[0].cpu(), torch.tensor([[float("inf"), 0.0, 0.0, 0.0, 2.0]]))


@pytest.mark.parametrize("kind", ["relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_slope_of_huge_values(kind, dt):
    """Slopes of 1 and 0 far out, where squares of the values leave fp32."""
    z = torch.tensor([[s * 2.0 ** e for s in (1, -1)] for e in (6, 12, 20, 40, 62, 64, 65, 80, 100, 120, 126)])
    z = z.reshape(-1, 1).to(dt).cuda()  # a row, and a scale, to each
    y, codes = dg.gemm_activation_tensors(z, kind, False, torch.float8_e5m2)
    grad = torch.full_like(z, 3.0)
    zg, again = dg.gemm_activation_backward_tensors(grad, codes, kind)
    up = (z > 0).to(dt)
    # silu and its slope at -64, the only value between: -64 e^-64 and -63 e^-64, of which e^-64 < 2^-92
    for have, want in ((zg, 3 * up), (y, z * up), (again, z * up)):
        assert ((have - want).abs() <= 64 * 3 * 2.0 ** -92).all() and torch.equal(have[2:], want[2:])

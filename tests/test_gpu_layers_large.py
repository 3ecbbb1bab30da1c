"""The adapters, the loss and the activations where offsets pass 32 bits, and small forms that other
files leave out."""
import pytest
import torch

import dense_gemm_06_amd as dg
import layer_util as lu

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LD = 2 ** 23 - 8


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def far(t):
    """t's values as rows of the widest leading dimension, so that the last ones lie past 2^31 elements."""
    rows, cols = t.shape
    assert (rows - 1) * LD > 2 ** 31
    wide = torch.empty(rows * LD, dtype=t.dtype, device="cuda").as_strided((rows, cols), (LD, 1))
    wide.copy_(t)
    return wide


def adapters(T, N, K, R, rank, dt, seed):
    g = gen(seed)
    def normal(*shape, size=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * size).to(dt)
    index = torch.randint(-1, R, (T,), generator=g, device="cuda", dtype=torch.int32)
    return (normal(T, K), normal(N, K, size=0.05), normal(R, rank, K, size=K ** -0.5), normal(R, N, rank, size=0.2),
            index, torch.rand(R, generator=g, device="cuda") + 0.5, normal(T, N, size=0.1))


def check(got, want, names):
    for have, (ref, err), name in zip(got, want, names):
        lu.check(have, ref, err, name)


@pytest.mark.parametrize("T,dt", [(9, BF16), (64, F16), (300, F16), (1100, BF16), (270, F32)])
def test_adapters_far_rows(T, dt):
    x, w, a, b, index, scale, grad = adapters(T, 320, 256, 3, 16, dt, T)
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), 3)
    ref, err, u_ref, u_err = lu.adapters(x, w, a, b, index, scale)
    u = dg.gemm_adapters_tensors(x, w, a, b, index, scale, keep=True)[1]
    want = lu.adapters_backward(grad, x, u, w, a, b, index, scale)
    for name in ("x", "w", "grad"):
        q = dict(x=x, w=w, grad=grad)
        if len(q[name]) <= 2 ** 31 // LD + 1:
            continue
        q[name] = far(q[name])
        check(dg.gemm_adapters_tensors(q["x"], q["w"], a, b, index, scale, keep=True), ((ref, err), (u_ref, u_err)),
              (f"y, far {name}", f"u, far {name}"))
        check(dg.gemm_adapters_backward_tensors(q["grad"], q["x"], u, q["w"], a, b, index, plan, scale), want,
              (f"x_grad, far {name}", f"a_grad, far {name}", f"b_grad, far {name}"))


@pytest.mark.parametrize("T,dt", [(5, BF16), (300, BF16), (5, F32)])
def test_many_long_adapters(T, dt):
    """The last adapters of a set of more than 2^31 numbers."""
    R, rank, K, N = 1024, 128, 16640, 128
    x, w, a3, b3, index, scale3, grad = adapters(T, N, K, 3, rank, dt, T)
    index[:] = torch.arange(T, device="cuda") % 3
    a = torch.zeros(R, rank, K, dtype=dt, device="cuda")
    b = torch.zeros(R, N, rank, dtype=dt, device="cuda")
    scale = torch.ones(R, device="cuda")
    at = torch.tensor([0, R - 2, R - 1], device="cuda")
    a[at], b[at], scale[at] = a3, b3, scale3
    there = at[index.long()].int()
    y, u = dg.gemm_adapters_tensors(x, w, a, b, there, scale, keep=True)
    ref, err, u_ref, u_err = lu.adapters(x, w, a3, b3, index, scale3)
    check((y, u), ((ref, err), (u_ref, u_err)), ("y", "u"))
    plan = dg.gemm_experts_dispatch_tensors(there[:, None].contiguous(), R)
    xg, ag, bg = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, there, plan, scale)
    check((xg, ag[at], bg[at]), lu.adapters_backward(grad, x, u, w, a3, b3, index, scale3), ("x_grad", "a_grad", "b_grad"))
    assert not ag[1:R - 2].any() and not bg[1:R - 2].any()


@pytest.mark.parametrize("T,K,dt", [(9, 256, BF16), (300, 256, F16), (300, 4, BF16), (270, 64, F32)])
def test_loss_far_rows(T, K, dt):
    g = gen(T)
    x = torch.randn(T, K, generator=g, device="cuda").to(dt)
    w = (torch.randn(700, K, generator=g, device="cuda") * 0.1).to(dt)
    target = torch.randint(0, 700, (T,), generator=g, device="cuda")
    grad = torch.rand(T, generator=g, device="cuda")
    lse = dg.gemm_loss_tensors(x, w, target)[1]
    ref, err, lse_ref, lse_err, _, _ = lu.loss(x, w, target)
    want = lu.loss_backward(grad, x, w, target, lse)
    for name in ("w", "x") if T > 256 else ("w",):
        x2, w2 = (far(x), w) if name == "x" else (x, far(w))
        check(dg.gemm_loss_tensors(x2, w2, target), ((ref, err), (lse_ref, lse_err)),
              (f"loss, far {name}", f"lse, far {name}"))
        check(dg.gemm_loss_backward_tensors(grad, x2, w2, target, lse), want, (f"x_grad, far {name}", f"w_grad, far {name}"))


def test_loss_of_a_large_vocabulary():
    """A vocabulary matrix, and its gradient, of more than 2^31 numbers: words that no one's logit is near
    stay at zero, the last ones get theirs."""
    T, K, V = 70, 4096, 530000
    g = gen(3)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    w = torch.zeros(V, K, dtype=BF16, device="cuda")
    tail = (torch.randn(300, K, generator=g, device="cuda") * 0.3).to(BF16)
    w[-300:] = tail
    target = V - 1 - torch.randint(0, 300, (T,), generator=g, device="cuda")
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    l = x.double() @ tail.double().t()
    ref = torch.logsumexp(torch.cat([l, torch.zeros(T, 1, device="cuda").double() + torch.log(torch.tensor(V - 300.0)).cuda()], 1), 1)
    # logits are off by (K + 1) roundings of their terms, the sum by V
    err = (x.abs().double() @ tail.abs().double().t()).amax(1) * (K + 1) * lu.F32 + (V + 200) * lu.F32
    assert ((lse.double() - ref).abs() <= err).all()
    grad = torch.ones(T, device="cuda")
    xg, wg = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    p = torch.exp(l - lse.double()[:, None])
    d = p - torch.nn.functional.one_hot(target - (V - 300), 300)
    half = lu.HALF[BF16]
    bound = ((d.abs() * half + p * err[:, None] * 1.01).t() @ x.abs().double()) * 1.02 + (d.t() @ x.double()).abs() * half
    assert ((wg[-300:].double() - d.t() @ x.double()).abs() <= bound + 1e-6).all()
    # the other words all have the same gradient
    assert (wg[:-300:1000] == wg[0]).all()
    assert torch.equal(wg[V - 301], wg[0])


@pytest.mark.parametrize("gated", [False, True])
def test_activation_of_many_rows(gated):
    T, F = 70000, 16384 if gated else 32768
    piece = torch.randn(1000, 32768, generator=gen(1), device="cuda").to(BF16)
    z = piece.repeat(70, 1)
    assert z.numel() > 2 ** 31
    y, codes = dg.gemm_activation_tensors(z, "silu", gated, torch.float8_e4m3fn)
    y1, codes1 = dg.gemm_activation_tensors(piece, "silu", gated, torch.float8_e4m3fn)
    assert torch.equal(y[:1000], y1) and torch.equal(y[-1000:], y1)
    assert torch.equal(codes.data.view(torch.uint8)[-1000:], codes1.data.view(torch.uint8))
    del z
    zg, y2 = dg.gemm_activation_backward_tensors(y, codes, "silu", gated)
    zg1, y3 = dg.gemm_activation_backward_tensors(y1, codes1, "silu", gated)
    assert torch.equal(zg[-1000:], zg1) and torch.equal(y2[-1000:], y3)
    assert torch.equal(dg.gemm_activation_value_tensors(codes, "silu", gated)[-1000:], y3)


@pytest.mark.parametrize("kind", ["relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,F,dt", [(1, 1, BF16), (3, 130, F16), (65, 1003, F32), (300, 4096, BF16)])
def test_activation_value_alone(kind, gated, T, F, dt):
    z = torch.randn(T, 2 * F if gated else F, generator=gen(F), device="cuda").to(dt)
    _, codes = dg.gemm_activation_tensors(z, kind, gated, torch.float8_e4m3fn)
    grad = torch.randn(T, F, generator=gen(F + 1), device="cuda").to(dt)
    zg, y = dg.gemm_activation_backward_tensors(grad, codes, kind, gated)
    assert torch.equal(dg.gemm_activation_value_tensors(codes, kind, gated, dt), y)
    alone, none = dg.gemm_activation_backward_tensors(grad, codes, kind, gated, value=False)
    assert none is None and torch.equal(alone, zg)


@pytest.mark.parametrize("T", [1, 17, 64, 90])
def test_no_adapters(T):
    """A set without adapters, of rank 0 too, leaves the shared product, as does index -1 everywhere."""
    for dt in (BF16, F16, F32):
        x, w, a, b, index, scale, grad = adapters(T, 192, 256, 2, 8, dt, T)
        y = dg.gemm_adapters_tensors(x, w, a, b, index.fill_(-1), scale)
        none = dg.gemm_adapters_tensors(x, w, a[:0], b[:0], index, scale[:0])
        flat = dg.gemm_adapters_tensors(x, w, a[:0, :0], b[:0, :, :0], index, None)
        assert torch.equal(y, none) and torch.equal(y, flat)
        ref, err, _, _ = lu.adapters(x, w, a, b, index, scale)
        lu.check(y, ref, err, "y")


@pytest.mark.parametrize("T", [1, 16, 33, 64])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_few_tokens_of_unaligned_rows(T, dt):
    """Rows one element off 16-byte boundaries give what aligned copies give, to their roundings."""
    x, w, a, b, index, scale, grad = adapters(T, 200, 260, 3, 12, dt, T)
    x1, w1 = (torch.empty(t.shape[0], t.shape[1] + 3, dtype=dt, device="cuda")[:, 1:-2].copy_(t) for t in (x, w))
    y = dg.gemm_adapters_tensors(x1, w1, a, b, index, scale)
    ref, err, _, _ = lu.adapters(x, w, a, b, index, scale)
    lu.check(y, ref, err, "y")
    target = torch.arange(T, device="cuda") * 3
    loss, lse = dg.gemm_loss_tensors(x1, w1, target)
    ref, err, lse_ref, lse_err, _, _ = lu.loss(x, w, target)
    lu.check(lse, lse_ref, lse_err, "lse")
    lu.check(loss, ref, err, "loss")


@pytest.mark.parametrize("T", [1, 15, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("V,K,dt", [(130, 72, BF16), (6150, 64, F16), (6147, 40, BF16), (33000, 16, BF16)])
def test_loss_gradients_of_few_tokens(T, V, K, dt):
    """Every form of d for few tokens, in one piece and in pieces whose last words are odd."""
    g = gen(T + V)
    x = torch.randn(T, K, generator=g, device="cuda").to(dt)
    w = (torch.randn(V, K, generator=g, device="cuda") * 0.3).to(dt)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[T // 2:: 5] = V - 1
    target[1::7] = -100
    grad = torch.rand(T, generator=g, device="cuda") - 0.5
    lse = dg.gemm_loss_tensors(x, w, target)[1]
    want = lu.loss_backward(grad, x, w, target, lse)
    for piece in (0, V // 2 + 1):
        check(dg.gemm_loss_backward_tensors(grad, x, w, target, lse, piece=piece), want, ("x_grad", "w_grad"))

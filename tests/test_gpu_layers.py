"""The adapters, the loss over a vocabulary and the 8-bit activations on the GPU against their
definitions in 64 bits, at the sizes, layouts and values where they can go wrong."""
import pytest
import torch

import block_util as bu
import dense_gemm_06_amd as dg
import layer_util as lu

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, pad):
    """t on the GPU as rows of a wider buffer filled with NaN."""
    if pad == 0:
        return t.cuda()
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    wide[..., :t.shape[-1]] = t.cuda()
    return wide[..., :t.shape[-1]]


# ----------------------------------------------------------------------------- adapters
def adapter_inputs(T, N, K, R, rank, dt, pad=0, seed=0, runs=False):
    g = gen(seed)
    x = torch.randn(T, K, generator=g).to(dt)
    w = (torch.randn(N, K, generator=g) * 0.05).to(dt)
    a = (torch.randn(R, rank, K, generator=g) * max(K, 1) ** -0.5).to(dt)
    b = (torch.randn(R, N, rank, generator=g) * 0.2).to(dt)
    scale = torch.rand(R, generator=g) + 0.5
    index = torch.randint(-1, R + 1, (T,), generator=g, dtype=torch.int32)  # -1 and R: no adapter
    if runs:
        index = index.sort().values
    return [strided(t, pad) for t in (x, w, a, b)] + [index.cuda(), scale.cuda()]


def check_adapters(x, w, a, b, index, scale, backward=True, grad_pad=0, seed=5):
    y, u = dg.gemm_adapters_tensors(x, w, a, b, index, scale, keep=True)
    ref, err, u_ref, u_err = lu.adapters(x, w, a, b, index, scale)
    lu.check(u, u_ref, u_err, "u")
    lu.check(y, ref, err, "y")
    assert y.dtype == x.dtype
    if not backward:
        return
    grad = strided((torch.randn(y.shape, generator=gen(seed)) * 0.1).to(x.dtype), grad_pad)
    R = a.shape[0]
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), R) if R else None
    got = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, plan, scale)
    want = lu.adapters_backward(grad, x, u, w, a, b, index, scale)
    for name, have, (ref, err) in zip(("x_grad", "a_grad", "b_grad"), got, want):
        lu.check(have, ref, err, name)
    again = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, plan, scale)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    none, ag, bg = dg.gemm_adapters_backward_tensors(grad, x, u, w, a, b, index, plan, scale, x_grad=False)
    assert none is None and torch.equal(ag, got[1]) and torch.equal(bg, got[2])


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,N,K,R,rank", [
    (1, 128, 256, 3, 16), (1, 1, 1, 1, 1), (2, 40, 7, 2, 3), (5, 264, 520, 4, 8), (17, 129, 131, 5, 12),
    (33, 256, 384, 6, 32), (64, 512, 512, 8, 16), (65, 500, 256, 2, 33), (130, 257, 264, 3, 64), (300, 272, 272, 9, 128)])
def test_adapters(T, N, K, R, rank, dt):
    check_adapters(*adapter_inputs(T, N, K, R, rank, dt, seed=T + N))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 8])
def test_adapters_strided(pad, dt):
    check_adapters(*adapter_inputs(70, 136, 200, 4, 16, dt, pad=pad, runs=True), grad_pad=pad)


@pytest.mark.parametrize("dt", [BF16, F16])
def test_adapters_tiles(dt):
    """Whole and cut 256 x 256 tiles, runs that end inside a tile, sizes at which every compute unit has one."""
    check_adapters(*adapter_inputs(1000, 1032, 520, 5, 24, dt, runs=True, seed=2))
    check_adapters(*adapter_inputs(2100, 4096, 512, 7, 16, dt, runs=True, seed=3))


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("pad", [0, 1])
def test_adapters_tiles_of_odd_rows(pad, dt):
    """Tiles whose rows start at any even byte, forward (many columns of y) and backward (of x)."""
    check_adapters(*adapter_inputs(2100, 4099, 203, 5, 20, dt, pad=pad, runs=True, seed=4), grad_pad=pad)
    check_adapters(*adapter_inputs(2100, 203, 4099, 5, 20, dt, pad=pad, runs=True, seed=5), grad_pad=pad)


def test_adapters_many_in_a_tile():
    """Every row of a tile another adapter's, and ranks on both sides of what the tiles hold."""
    for rank in (64, 65):
        x, w, a, b, index, scale = adapter_inputs(2050, 4096, 64, 40, rank, BF16, seed=rank)
        check_adapters(x, w, a, b, index, scale, backward=rank == 64)


def test_adapters_without_scale_and_without_rows():
    x, w, a, b, index, scale = adapter_inputs(40, 128, 128, 4, 16, BF16, seed=4)
    index = torch.where(index == 2, 1, index)  # adapter 2 has no rows
    check_adapters(x, w, a, b, index, None)
    index = torch.full_like(index, -1)         # nor has any
    check_adapters(x, w, a, b, index, scale)
    far = torch.full_like(index, 2 ** 31 - 1)
    check_adapters(x, w, a, b, far, scale)


def test_adapters_empty():
    for T, N, K, R, rank in ((0, 16, 16, 2, 4), (5, 0, 16, 2, 4), (5, 16, 0, 2, 4), (5, 16, 16, 0, 4), (5, 16, 16, 0, 0)):
        x, w, a, b, index, scale = adapter_inputs(T, N, K, R, rank, BF16)
        check_adapters(x, w, a, b, index, scale)


def test_adapters_special_values():
    """A NaN or an infinity stays in its own row, and in its own adapter's gradient."""
    x, w, a, b, index, scale = adapter_inputs(64, 96, 128, 3, 8, BF16, seed=6)
    index = (torch.arange(64, dtype=torch.int32) % 3).cuda()
    plain = dg.gemm_adapters_tensors(x, w, a, b, index, scale)
    x2 = x.clone()
    x2[7, 3], x2[20, 5] = float("nan"), float("inf")
    got, u = dg.gemm_adapters_tensors(x2, w, a, b, index, scale, keep=True)
    keep = [t for t in range(64) if t not in (7, 20)]
    assert torch.equal(got[keep], plain[keep]) and got[7].isnan().all() and not got[20].isfinite().any()
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), 3)
    _, ag, bg = dg.gemm_adapters_backward_tensors(plain, x2, u, w, a, b, index, plan, scale)
    assert ag[0].isfinite().all() and bg[0].isfinite().all()  # rows 7 and 20 are of adapters 1 and 2
    assert ag[1, :, 3].isnan().all() and not ag[2, :, 5].isfinite().any()
    a2 = a.clone()
    a2[1] = float("nan")  # an adapter that other rows do not use
    other = dg.gemm_adapters_tensors(x, w, a2, b, index, scale)
    use = (index != 1).cpu()
    assert torch.equal(other[use], plain[use]) and other[~use].isnan().all()


def test_adapters_differences():
    """The gradients against differences of the forward pass in fp32."""
    x, w, a, b, index, scale = adapter_inputs(9, 12, 10, 2, 3, F32, seed=8)
    weight = torch.randn(9, 12, generator=gen(1), dtype=torch.float64)
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), 2)
    u = dg.gemm_adapters_tensors(x, w, a, b, index, scale, keep=True)[1]
    grads = dg.gemm_adapters_backward_tensors(weight.float().cuda(), x, u, w, a, b, index, plan, scale)
    f = lambda: float((dg.gemm_adapters_tensors(x, w, a, b, index, scale).cpu().double() * weight).sum())  # noqa: E731
    for t, have in zip((x, a, b), grads):
        flat = t.view(-1)
        for at in range(0, flat.numel(), max(1, flat.numel() // 7)):
            old, step = flat[at].item(), 2.0 ** -5
            flat[at] = old + step
            up = f()
            flat[at] = old - step
            down = f()
            flat[at] = old
            # the pass is linear in each element: only fp32 roundings of about 108 terms are left
            assert abs((up - down) / (2 * step) - have.view(-1)[at].item()) < 108 * 4 * 20 * lu.F32 / step


# ----------------------------------------------------------------------------- loss
def loss_inputs(T, V, K, dt, pad=0, seed=0, size=1.0):
    g = gen(seed)
    x = (torch.randn(T, K, generator=g) * size).to(dt)
    w = (torch.randn(V, K, generator=g) * 2 * max(K, 1) ** -0.5).to(dt)
    target = torch.randint(0, max(V, 1), (T,), generator=g)
    target = torch.where(torch.rand(T, generator=g) < 0.15, torch.tensor([-100, V, -1, 2 ** 40])[
        torch.randint(0, 4, (T,), generator=g)], target)
    return strided(x, pad), strided(w, pad), target.cuda(), (torch.randn(T, generator=g) / max(T, 1)).cuda()


def check_loss(x, w, target, grad, **kw):
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    ref, err, lse_ref, lse_err, _, _ = lu.loss(x, w, target)
    lu.check(lse, lse_ref, lse_err, "lse")
    lu.check(loss, ref, err, "loss")
    (xr, xe), (wr, we) = lu.loss_backward(grad, x, w, target, lse)
    xg, wg = dg.gemm_loss_backward_tensors(grad, x, w, target, lse, **kw)
    assert xg.dtype == wg.dtype == x.dtype
    lu.check(xg, xr, xe, "x_grad")
    lu.check(wg, wr, we, "w_grad")
    only_x, none = dg.gemm_loss_backward_tensors(grad, x, w, target, lse, w_grad=False, **kw)
    assert none is None
    lu.check(only_x, xr, xe, "x_grad alone")
    none, only_w = dg.gemm_loss_backward_tensors(grad, x, w, target, lse, x_grad=False, **kw)
    assert none is None
    lu.check(only_w, wr, we, "w_grad alone")
    again = dg.gemm_loss_tensors(x, w, target)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    xg2, wg2 = dg.gemm_loss_backward_tensors(grad, x, w, target, lse, **kw)
    assert torch.equal(xg, xg2) and torch.equal(wg, wg2)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T,V,K", [
    (1, 1, 1), (1, 1000, 64), (1, 257, 8), (3, 2, 5), (16, 512, 256), (31, 1003, 72), (64, 256, 128), (65, 511, 200),
    (257, 770, 136), (300, 1029, 264)])
def test_loss(T, V, K, dt):
    check_loss(*loss_inputs(T, V, K, dt, seed=T + V))


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("piece", [1, 100, 256, 1000])
def test_loss_pieces(piece, dt):
    check_loss(*loss_inputs(37, 600 if piece > 1 else 9, 64, dt, seed=piece), piece=piece)


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 8])
def test_loss_strided(pad, dt):
    check_loss(*loss_inputs(40, 300, 96, dt, pad=pad, seed=pad))


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_tiles(dt):
    check_loss(*loss_inputs(520, 9000, 256, dt, seed=1))
    check_loss(*loss_inputs(1024, 4096, 512, dt, seed=2))


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_wide_and_narrow_tiles(dt):
    """A whole round of wide tiles and the rest in narrow ones."""
    check_loss(*loss_inputs(2041, 9003, 64, dt, seed=8))


@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("T,V,K,pad", [(100, 520, 77, 0), (300, 1029, 80, 1), (513, 300, 131, 3)])
def test_loss_odd_rows(T, V, K, pad, dt):
    check_loss(*loss_inputs(T, V, K, dt, pad=pad, seed=T))


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_loss_far_logits(dt):
    """Logits of hundreds: the maximum keeps the exponentials in range."""
    check_loss(*loss_inputs(50, 700, 64, dt, seed=3, size=100.0))


def test_loss_empty():
    for T, V, K in ((0, 9, 8), (5, 9, 0), (0, 0, 8)):
        check_loss(*loss_inputs(T, V, K, BF16)) if T else None
    x, w, target, grad = loss_inputs(0, 9, 8, BF16)
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    xg, wg = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    assert loss.numel() == 0 and xg.shape == (0, 8) and torch.equal(wg, torch.zeros_like(wg))
    x, w, target, grad = loss_inputs(5, 0, 8, F16)
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    xg, wg = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    assert (loss == 0).all() and (lse == float("-inf")).all()
    assert torch.equal(xg, torch.zeros_like(xg)) and wg.shape == (0, 8)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_loss_ignored_rows(dt):
    """Rows without a target: loss 0, gradients 0, also where the row holds a NaN."""
    x, w, target, grad = loss_inputs(40, 300, 64, dt, seed=4)
    target = torch.full_like(target, -100)
    x[3, 5] = float("nan")
    loss, lse = dg.gemm_loss_tensors(x, w, target)
    assert torch.equal(loss, torch.zeros_like(loss)) and lse[3].isnan() and lse.isnan().sum() == 1
    xg, wg = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    assert torch.equal(xg, torch.zeros_like(xg))
    clean = [c for c in range(64) if c != 5]
    assert (wg[:, clean] == 0).all()


@pytest.mark.parametrize("dt", [BF16, F16, F32])
def test_loss_special_values(dt):
    """Infinite logits: a word that cannot follow (-inf), and NaN kept to its row."""
    x, w, target, grad = loss_inputs(20, 300, 64, dt, seed=5)
    target = torch.arange(20, device="cuda")
    x[:, 0] = 1
    w2 = w.clone()
    w2[250, 0] = float("-inf")
    loss, lse = dg.gemm_loss_tensors(x, w2, target)
    ref = lu.loss(x, w2[torch.arange(300) != 250], target)
    lu.check(lse, ref[2], ref[3], "lse")
    lu.check(loss, ref[0], ref[1], "loss")
    x[4, 1] = float("nan")
    loss2, lse2 = dg.gemm_loss_tensors(x, w2, target)
    keep = [t for t in range(20) if t != 4]
    assert torch.equal(loss2[keep], loss[keep]) and loss2[4].isnan() and lse2[4].isnan()


@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 8])
def test_loss_gradient_scales(size):
    """fp16 gradients of small and large upstream gradients keep their digits; rows of grad 0 give 0."""
    x, w, target, grad = loss_inputs(60, 400, 64, F16, seed=6, size=30.0)
    grad = (grad * 0 + 2.0 ** -6) * size
    grad[5] = 0
    check_loss(x, w * 0.03125, target, grad)
    lse = dg.gemm_loss_tensors(x, w, target)[1]
    assert (dg.gemm_loss_backward_tensors(grad, x, w, target, lse)[0][5] == 0).all()


@pytest.mark.parametrize("dt", [BF16, F16])
def test_loss_rows_of_no_gradient(dt):
    """Tokens of gradient 0, or of one that the fp16 scale brings to 0, add nothing to the word that is
    their target, whatever the workspace held before."""
    x, w, target, grad = loss_inputs(70, 300, 64, dt, seed=9)
    target[::2] = 7
    grad[::4], grad[1], grad[2] = 0, 2.0 ** 100, 2.0 ** -140
    lse = dg.gemm_loss_tensors(x, w, target)[1]
    held = [torch.full((2 ** k,), float("nan"), device="cuda") for k in range(8, 22) for _ in range(2)]
    del held
    _, wg = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    xg, only = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    (xr, xe), (wr, we) = lu.loss_backward(grad, x, w, target, lse)
    lu.check(xg, xr, xe, "x_grad")
    lu.check(wg, wr, we, "w_grad")
    assert torch.equal(wg, only) and (xg[::4] == 0).all()


def test_loss_differences():
    x, w, target, grad = loss_inputs(6, 11, 5, F32, seed=7)
    lse = dg.gemm_loss_tensors(x, w, target)[1]
    grads = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    f = lambda: float((dg.gemm_loss_tensors(x, w, target)[0].cpu().double() * grad.cpu().double()).sum())  # noqa: E731
    for t, have in zip((x, w), grads):
        flat = t.view(-1)
        for at in range(0, flat.numel(), max(1, flat.numel() // 7)):
            old, step = flat[at].item(), 2.0 ** -7
            flat[at] = old + step
            up = f()
            flat[at] = old - step
            down = f()
            flat[at] = old
            # the cubic term of a difference is step^2 / 6 of a third derivative of at most a few
            # |w|^3 |grad|; the losses' roundings are 2^-22 each, over the step
            bound = step ** 2 * 4 * float(grad.abs().sum()) * 8 + 6 * 2.0 ** -20 / step * float(grad.abs().max())
            assert abs((up - down) / (2 * step) - have.view(-1)[at].item()) < bound


# ----------------------------------------------------------------------------- activations
def check_activation(z, kind, gated, code, grad_pad=0):
    y, codes = dg.gemm_activation_tensors(z, kind, gated, code)
    lu.check(y, *lu.activation(z, kind, gated), "y")
    alone, none = dg.gemm_activation_tensors(z, kind, gated)
    assert none is None and torch.equal(alone, y)
    q, _ = dg.gemm_block_quantize_tensors(z, code)
    assert torch.equal(q.data.view(torch.uint8), codes.data.view(torch.uint8)) and torch.equal(q.scale, codes.scale)
    grad = strided((torch.randn(y.shape, generator=gen(9)) * 0.1).to(z.dtype), grad_pad)
    zg, y2 = dg.gemm_activation_backward_tensors(grad, codes, kind, gated)
    (zr, ze), (yr, ye) = lu.activation_backward(grad, bu.values(codes.data, codes.scale, 1), kind, gated)
    lu.check(zg, zr, ze, "z_grad")
    lu.check(y2, yr, ye, "y again")
    only, none = dg.gemm_activation_backward_tensors(grad, codes, kind, gated, value=False)
    assert none is None and torch.equal(only, zg)


@pytest.mark.parametrize("kind", ["relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,F,dt,code", [
    (1, 1, BF16, E4), (1, 128, F16, E4), (3, 7, F32, E5), (5, 130, BF16, E4), (16, 256, BF16, E5), (33, 515, F16, E4),
    (70, 384, F32, E4), (129, 1000, BF16, E4)])
def test_activation(kind, gated, T, F, dt, code):
    z = (torch.randn(T, 2 * F if gated else F, generator=gen(T + F)) * 3).to(dt)
    check_activation(z.cuda(), kind, gated, code)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("F", [128, 203])
def test_activation_strided(gated, F):
    z = torch.randn(40, 2 * F if gated else F, generator=gen(F)).to(BF16)
    check_activation(strided(z, 3), "silu", gated, E4, grad_pad=5)


@pytest.mark.parametrize("kind", ["gelu_tanh", "silu"])
def test_activation_far_values(kind):
    """Values at which the exponential over- and underflows, in 32 bits."""
    z = torch.linspace(-120, 120, 4001)[None, :].repeat(2, 1)
    check_activation(z.cuda(), kind, False, E5)


def test_activation_special_values():
    """Zeros; a NaN or an infinity reaches its own element of y only."""
    z = torch.zeros(4, 512, dtype=BF16, device="cuda")
    y, codes = dg.gemm_activation_tensors(z, "silu", True, E4)
    assert (y == 0).all() and (codes.data.float() == 0).all() and codes.scale.isfinite().all()
    z = torch.randn(4, 512, generator=gen(1)).to(BF16).cuda()
    plain = dg.gemm_activation_tensors(z, "silu", True, E4)[0]
    z2 = z.clone()
    z2[1, 7], z2[2, 300] = float("nan"), float("inf")
    y, codes = dg.gemm_activation_tensors(z2, "silu", True, E4)
    q, _ = dg.gemm_block_quantize_tensors(z2, E4)
    assert torch.equal(q.data.view(torch.uint8), codes.data.view(torch.uint8))
    same = torch.ones_like(y, dtype=torch.bool)
    same[1, 7] = same[2, 300 - 256] = False
    assert torch.equal(y[same], plain[same]) and y[1, 7].isnan() and y[2, 44].isinf()


def test_activation_empty():
    for shape in ((0, 64), (5, 0)):
        z = torch.zeros(shape, dtype=BF16, device="cuda")
        y, codes = dg.gemm_activation_tensors(z, "relu", True, E4)
        zg, _ = dg.gemm_activation_backward_tensors(y, codes, "relu", True)
        assert y.shape == (shape[0], shape[1] // 2) and zg.shape == z.shape


def test_activation_codes_in_square_blocks():
    """The backward pass reads codes of 128 x 128 blocks too."""
    z = torch.randn(200, 300, generator=gen(2)).to(BF16).cuda()
    codes, _ = dg.gemm_block_quantize_tensors(z, E4, 128)
    grad = torch.randn(200, 300, generator=gen(3)).to(BF16).cuda()
    zg, y = dg.gemm_activation_backward_tensors(grad, codes, "gelu_tanh")
    (zr, ze), (yr, ye) = lu.activation_backward(grad, bu.values(codes.data, codes.scale, 128), "gelu_tanh", False)
    lu.check(zg, zr, ze, "z_grad")
    lu.check(y, yr, ye, "y")

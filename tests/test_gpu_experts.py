"""GPU tests of the experts' operators against their definitions in 64 bits on the CPU."""
import pytest
import torch

import dense_gemm_06_amd as dg
from block_util import BLOCK, HALF, TINY, blocks, check_product, codes, dispatch, route, scores, values

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def choice(g, T, E, k):
    return torch.topk(torch.randn(T, E, generator=g) + torch.randn(1, E, generator=g), k, dim=1).indices.to(torch.int32)


# ----------------------------------------------------------------------------- route
ROUTES = [dict(E=8, k=2), dict(E=64, k=4, renorm=True), dict(E=60, k=6, bias=True),
          dict(E=256, k=8, score="sigmoid", groups=8, top_groups=4, group_top=2, bias=True, renorm=True, factor=2.5),
          dict(E=160, k=6, groups=4, top_groups=2, group_top=1), dict(E=1, k=1), dict(E=65, k=65 and 32),
          dict(E=1000, k=3, score="sigmoid", bias=True), dict(E=1024, k=32, groups=128, top_groups=7, group_top=4),
          dict(E=12, k=3, groups=4, top_groups=1, group_top=3, bias=True), dict(E=300, k=5, groups=100, top_groups=3)]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(f"{a}{b}" for a, b in c.items()))
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_route(case, dtype):
    g = gen(case["E"])
    r = dict(score="softmax", groups=1, top_groups=1, group_top=1, renorm=False, factor=1.0)
    r.update({a: b for a, b in case.items() if a in r})
    for T in (1, 3, 70):
        x = (torch.randn(T, case["E"], generator=g) * 2).to(dtype)
        bias = torch.randn(case["E"], generator=g) * 0.1 if case.get("bias") else None
        index, weight = dg.gemm_experts_route_tensors(x.cuda(), dg.router(case["k"], **r),
                                                      bias.cuda() if bias is not None else None)
        i, w = route(x, bias, case["k"], r["score"], r["groups"], r["top_groups"], r["group_top"], r["renorm"],
                     r["factor"])
        assert torch.equal(index.cpu(), i)
        assert ((weight.cpu().double() - w).abs() <= w.abs() * (2.0 ** -24 + 2.0 ** -45) + 2.0 ** -149).all()


def test_route_ties_take_the_lowest_index():
    x = torch.zeros(5, 100)
    x[1, 40:] = 1
    x[2, ::2] = -3
    x[3] = 200.0       # sigmoid scores all 1 in 64 bits
    x[4] = -0.0
    x[4, 50] = 0.0
    for score in ("softmax", "sigmoid"):
        index, _ = dg.gemm_experts_route_tensors(x.cuda(), dg.router(4, score))
        assert index.cpu().tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [1, 3, 5, 7], [0, 1, 2, 3], [0, 1, 2, 3]]
        index, _ = dg.gemm_experts_route_tensors(x.cuda(), dg.router(4, score, groups=10, top_groups=2, group_top=2))
        assert index.cpu().tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [1, 3, 5, 7], [0, 1, 2, 3], [0, 1, 2, 3]]


def test_route_close_scores():
    """Differences that fp32 scores lose: logits one step apart far out on the sigmoid, biases one step apart."""
    x = torch.full((2, 64), 17.0)
    x[0, 33] = torch.nextafter(torch.tensor(17.0), torch.tensor(18.0))
    x[1, 5] = torch.nextafter(torch.tensor(17.0), torch.tensor(0.0))
    index, _ = dg.gemm_experts_route_tensors(x.cuda(), dg.router(2, "sigmoid"))
    assert index.cpu().tolist() == [[33, 0], [0, 1]]
    bias = torch.full((64,), 0.25)
    bias[50] = torch.nextafter(torch.tensor(0.25), torch.tensor(1.0))
    index, _ = dg.gemm_experts_route_tensors(torch.zeros(1, 64).cuda(), dg.router(2, "sigmoid"), bias.cuda())
    assert index.cpu().tolist() == [[50, 0]]


def test_route_masked_and_nan_logits():
    x = torch.randn(4, 70, generator=gen(0))
    x[0, 3:] = -float("inf")                       # fewer live experts than choices
    x[1, :] = torch.finfo(torch.float32).min
    x[2, 60] = float("nan")
    x[3, 10] = float("nan")
    index, weight = dg.gemm_experts_route_tensors(x.cuda(), dg.router(5, "softmax"))
    live = sorted(range(3), key=lambda e: -x[0, e].item())
    assert index[0].tolist() == live + [3, 4] and weight[0, 3:].tolist() == [0.0, 0.0]
    assert index[1].tolist() == [0, 1, 2, 3, 4]
    assert index[2].tolist() == [0, 1, 2, 3, 4] and torch.isnan(weight[2]).all()   # softmax: the whole row is NaN
    index, weight = dg.gemm_experts_route_tensors(x.cuda(), dg.router(5, "sigmoid"))
    assert index[3, 0].item() == 10 and torch.isnan(weight[3, 0]) and torch.isfinite(weight[3, 1:]).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_route_backward(score, renorm, dtype):
    for T, E, k in ((1, 1, 1), (5, 8, 2), (33, 64, 4), (20, 130, 8), (9, 1024, 32)):
        g = gen(T * E)
        x = torch.randn(T, E, generator=g).to(dtype)
        r = dg.router(k, score, renorm=renorm, factor=1.5)
        wg = torch.randn(T, k, generator=g)
        index, _ = dg.gemm_experts_route_tensors(x.cuda(), r)
        got = dg.gemm_experts_route_backward_tensors(x.cuda(), r, index, wg.cuda())
        z = x.double().requires_grad_(True)
        s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
        p = s.gather(1, index.cpu().long())
        (((p / p.sum(1, keepdim=True) if renorm else p) * 1.5) * wg.double()).sum().backward()
        # one rounding, and 64-bit roundings of sums whose terms are at most |wg| * factor / sum of the chosen
        size = wg.double().abs().amax(1, keepdim=True) * 1.5 * k * (1 / p.detach().sum(1, keepdim=True) if renorm else 1)
        bound = z.grad.abs() * HALF[dtype] * (1 + 2.0 ** -9) + size * 2.0 ** -44 + TINY[dtype]
        assert got.dtype == dtype and ((got.cpu().double() - z.grad).abs() <= bound).all()


def test_route_backward_against_differences():
    """The gradient times a small step, against the change of the weights (64-bit weights of the definition)."""
    g = gen(3)
    for score, renorm in (("softmax", True), ("sigmoid", True), ("softmax", False), ("sigmoid", False)):
        x, wg, d = torch.randn(4, 16, generator=g), torch.randn(4, 3, generator=g), torch.randn(4, 16, generator=g)
        r = dg.router(3, score, renorm=renorm)
        index, _ = dg.gemm_experts_route_tensors(x.cuda(), r)
        grad = dg.gemm_experts_route_backward_tensors(x.cuda(), r, index, wg.cuda()).cpu().double()

        def loss(z):
            p = scores(z, score).gather(1, index.cpu().long())
            return ((p / p.sum(1, keepdim=True) if renorm else p) * wg.double()).sum(1)

        h = 2.0 ** -14
        change = (loss(x.double() + h * d.double()) - loss(x.double() - h * d.double())) / (2 * h)
        # third-derivative term h^2 |d|^3, and the fp32 rounding of the gradient
        bound = h * h * d.double().abs().sum(1) ** 3 * wg.double().abs().sum(1) + (grad.abs() * d.double().abs()).sum(1) * 2.0 ** -23
        assert ((change - (grad * d.double()).sum(1)).abs() <= bound).all()


def test_route_backward_bad_index():
    """Choices outside 0 .. E-1 carry nothing; a repeated one counts twice."""
    x = torch.randn(2, 70, generator=gen(1))
    index = torch.tensor([[-1, 70, 3], [5, 5, 1 << 30]], dtype=torch.int32)
    wg = torch.randn(2, 3, generator=gen(2))
    got = dg.gemm_experts_route_backward_tensors(x.cuda(), dg.router(3, "sigmoid"), index.cuda(), wg.cuda()).cpu()
    s = torch.sigmoid(x.double())
    want = torch.zeros(2, 70, dtype=torch.float64)
    want[0, 3], want[1, 5] = wg[0, 2].double(), wg[1, 0].double() + wg[1, 1].double()
    want = want * s * (1 - s)
    assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -23).all()


# ----------------------------------------------------------------------------- dispatch
@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 8), (16, 4, 64), (300, 6, 60), (1025, 1, 1024), (700, 8, 256),
                                   (5000, 2, 8)])
@pytest.mark.parametrize("align", [1, 128, 24])
def test_dispatch(T, k, E, align):
    index = choice(gen(T + E), T, E, k) if T else torch.empty(0, k, dtype=torch.int32)
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, align)
    want = dispatch(index, E, align, plan.rows.numel())
    for got, w in zip((plan.offsets, plan.counts, plan.rows, plan.position), want):
        assert torch.equal(got.cpu(), w)


def test_dispatch_one_expert_takes_all_and_bad_indices():
    index = torch.full((3000, 2), 5, dtype=torch.int32)
    index[::7, 1] = -3
    index[::11, 0] = 9
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), 9, 128)
    want = dispatch(index, 9, 128, plan.rows.numel())
    for got, w in zip((plan.offsets, plan.counts, plan.rows, plan.position), want):
        assert torch.equal(got.cpu(), w)


# ----------------------------------------------------------------------------- products
def expert_values(b):
    return torch.stack([values(b[0][e], b[1][e], BLOCK) for e in range(b[0].shape[0])])


def check_experts(c, a, b, plan, dtype, gather):
    """a (rows, K), b (E, N, K) in 64 bits."""
    off, cnt, rows = plan.offsets.tolist(), plan.counts.tolist(), plan.rows.cpu().long()
    out = c.cpu()
    live = torch.zeros(len(rows), dtype=torch.bool)
    for e in range(len(cnt)):
        lo, hi = off[e], off[e] + cnt[e]
        live[lo:hi] = True
        if hi > lo:
            check_product(out[lo:hi], a[rows[lo:hi]] if gather else a[lo:hi], b[e], dtype, e)
    assert (out[~live] == 0).all()


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 16, 128), (1, 2, 8, 256, 256), (16, 4, 64, 256, 512), (5, 3, 7, 100, 130),
                                       (64, 2, 4, 130, 384), (200, 2, 8, 256, 256), (333, 6, 10, 264, 400),
                                       (600, 4, 6, 300, 77), (1500, 2, 4, 512, 256)])
@pytest.mark.parametrize("align", [1, 128])
def test_experts_product(T, k, E, N, K, align):
    g = gen(T + N)
    plan = dg.gemm_experts_dispatch_tensors(choice(g, T, E, k).cuda(), E, align)
    for i, (ta, tb) in enumerate(((E4, E4), (E5, E4), (E4, E5), (E5, E5))):
        out = (BF16, F32, F16)[(i + T) % 3]
        a, b = codes(g, T, K, ta, 1), codes(g, N, K, tb, BLOCK, batch=E)
        B = dg.BlockTensor(b[0].cuda(), b[1].cuda(), BLOCK)
        c = dg.gemm_experts_product_tensors(dg.BlockTensor(a[0].cuda(), a[1].cuda(), 1), B, plan, out)
        check_experts(c, values(*a, 1), expert_values(b), plan, out, True)
    P = plan.rows.numel()
    a = codes(g, P, K, E4, 1)
    b = codes(g, N, K, E4, BLOCK, batch=E)
    c = dg.gemm_experts_product_tensors(dg.BlockTensor(a[0].cuda(), a[1].cuda(), 1),
                                        dg.BlockTensor(b[0].cuda(), b[1].cuda(), BLOCK), plan, F32, gather=False)
    check_experts(c, values(*a, 1), expert_values(b), plan, F32, False)


def test_experts_product_empty_experts_and_nan_padding():
    """Experts without rows; NaN codes in the row that padding would read stay out of the padding rows."""
    g = gen(4)
    for T in (4, 300):
        index = torch.where(torch.rand(T, 2, generator=g) < 0.5, 1, 6).to(torch.int32)
        index[0] = -1
        plan = dg.gemm_experts_dispatch_tensors(index.cuda(), 8, 128)
        a, b = codes(g, T, 256, E4, 1), codes(g, 160, 256, E4, BLOCK, batch=8)
        a[0][0] = float("nan")                      # token 0 goes to no expert
        c = dg.gemm_experts_product_tensors(dg.BlockTensor(a[0].cuda(), a[1].cuda(), 1),
                                            dg.BlockTensor(b[0].cuda(), b[1].cuda(), BLOCK), plan, F32)
        check_experts(c, values(*a, 1), expert_values(b), plan, F32, True)


def test_experts_product_without_tokens():
    """A plan with rows, and no token for them to name: zeros, and A is not read."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = codes(gen(1), 64, 128, E4, BLOCK, batch=2)
    B = dg.BlockTensor(b[0].cuda(), b[1].cuda(), BLOCK)
    a = dg.BlockTensor(torch.empty(0, 128, device="cuda").to(E4), torch.empty(0, 1, device="cuda"), 1)
    for P in (8, 300):
        plan = dg.ExpertPlan(i32(0, 2, P), i32(2, P - 2), torch.zeros(P, dtype=torch.int32, device="cuda"),
                             torch.empty(0, 2, dtype=torch.int32, device="cuda"))
        assert (dg.gemm_experts_product_tensors(a, B, plan, F32) == 0).all()


def test_experts_product_many_experts():
    g = gen(6)
    plan = dg.gemm_experts_dispatch_tensors(choice(g, 90, 200, 3).cuda(), 200, 1)
    a, b = codes(g, 90, 128, E4, 1), codes(g, 48, 128, E4, BLOCK, batch=200)
    c = dg.gemm_experts_product_tensors(dg.BlockTensor(a[0].cuda(), a[1].cuda(), 1),
                                        dg.BlockTensor(b[0].cuda(), b[1].cuda(), BLOCK), plan, F32)
    check_experts(c, values(*a, 1), expert_values(b), plan, F32, True)


@pytest.mark.parametrize("T,k,E,M,N", [(1, 1, 2, 64, 64), (40, 2, 4, 100, 130), (300, 3, 6, 256, 128), (200, 2, 3, 500, 77),
                                       (900, 4, 5, 300, 600)])
def test_experts_gradient(T, k, E, M, N):
    """Through the quantizer's transposed, gathered form, as a training step has it; ragged M and N."""
    g = gen(T)
    index = choice(g, T, E, k)
    index[index == E - 1] = 0                        # the last expert has no rows
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, BLOCK)
    x, y = torch.randn(T, M, generator=g).to(BF16).cuda(), torch.randn(T, N, generator=g).to(BF16).cuda()
    off = plan.offsets.tolist()
    for ta, tb, rows_b, out in ((E5, E4, 1, F32), (E4, E4, BLOCK, BF16), (E4, E5, 1, F16), (E5, E5, 1, F32)):
        _, a = dg.gemm_block_quantize_tensors(x, ta, natural=False, transposed=True, rows=plan.rows)
        _, b = dg.gemm_block_quantize_tensors(y, tb, rows_b, natural=False, transposed=True, rows=plan.rows)
        c = dg.gemm_experts_gradient_tensors(a, b, plan, out)
        A, B = values(a.data, a.scale, 1), values(b.data, b.scale, rows_b)
        for e in range(E):
            check_product(c[e], A[:, off[e]:off[e + 1]], B[:, off[e]:off[e + 1]], out, e)


@pytest.mark.parametrize("T,M,N", [(70, 64, 128), (300, 130, 200)])
def test_experts_operands_with_adjacent_rows(T, M, N):
    """The gradient of codes stored (P, N); the data gradient through the experts' own matrices, turned."""
    g = gen(T)
    plan = dg.gemm_experts_dispatch_tensors(choice(g, T, 4, 2).cuda(), 4, BLOCK)
    P, off = plan.rows.numel(), plan.offsets.tolist()
    a, b = codes(g, M, P, E5, 1), codes(g, N, P, E4, 1)
    want_a, want_b = values(*a, 1), values(*b, 1)
    flip = lambda x: x.cuda().t().contiguous().t()  # noqa: E731
    for fa, fb in ((False, True), (True, False), (True, True)):
        A = dg.BlockTensor(flip(a[0]) if fa else a[0].cuda(), a[1].cuda(), 1)
        B = dg.BlockTensor(flip(b[0]) if fb else b[0].cuda(), b[1].cuda(), 1)
        c = dg.gemm_experts_gradient_tensors(A, B, plan)
        for e in range(4):
            check_product(c[e], want_a[:, off[e]:off[e + 1]], want_b[:, off[e]:off[e + 1]], F32, e)
    w = codes(g, N, M, E4, BLOCK, batch=4)
    W = dg.BlockTensor(w[0].cuda(), w[1].cuda(), BLOCK)
    x = codes(g, T, N, E5, 1)
    c = dg.gemm_experts_product_tensors(dg.BlockTensor(x[0].cuda(), x[1].cuda(), 1), W.t(), plan, BF16)
    check_experts(c, values(*x, 1), expert_values(w).transpose(1, 2).contiguous(), plan, BF16, True)


def test_experts_gradient_rows_inside_a_block_are_nan():
    plan = dg.gemm_experts_dispatch_tensors(torch.tensor([[0], [1]], dtype=torch.int32).cuda(), 2, 64)
    P = plan.rows.numel()
    z = dg.BlockTensor(torch.zeros(32, P, device="cuda").to(E4), torch.ones(32, blocks(P), device="cuda"), 1)
    plan.align = None
    c = dg.gemm_experts_gradient_tensors(z, z, plan)
    assert (c[0] == 0).all() and torch.isnan(c[1]).all()


# ----------------------------------------------------------------------------- combine
@pytest.mark.parametrize("T,k,E,N", [(1, 1, 1, 1), (1, 8, 8, 256), (16, 4, 64, 2048), (33, 6, 60, 100), (257, 2, 8, 4100),
                                     (40, 3, 5, 2049)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("align", [1, 128])
def test_combine(T, k, E, N, dtype, align):
    g = gen(T * N)
    index = choice(g, T, E, k)
    if T > 3:
        index[2] = -1                                # a token without rows
        index[3, 0] = E
    plan = dg.gemm_experts_dispatch_tensors(index.cuda(), E, align)
    P = plan.rows.numel()
    y = torch.randn(P, N, generator=g).to(dtype)
    w, grad = torch.rand(T, k, generator=g), torch.randn(T, N, generator=g).to(dtype)
    out = dg.gemm_experts_combine_tensors(y.cuda(), plan, w.cuda())
    y_grad, w_grad = dg.gemm_experts_combine_backward_tensors(y.cuda(), plan, w.cuda(), grad.cuda())
    at, there = plan.position.cpu().long().clamp(min=0), (plan.position.cpu() >= 0).double()
    Y, G, W = y.double(), grad.double(), w.double() * there
    picked = Y[at.reshape(-1)].reshape(T, k, N)
    ref, size = (picked * W[:, :, None]).sum(1), (picked.abs() * W[:, :, None]).sum(1)
    assert ((out.cpu().double() - ref).abs() <= size * k * 2.0 ** -24 + ref.abs() * HALF[dtype] * (1 + 2.0 ** -9) + TINY[dtype]).all()
    ref, size = (picked * G[:, None, :]).sum(2) * there, (picked * G[:, None, :]).abs().sum(2)
    assert ((w_grad.cpu().double() - ref).abs() <= size * (N + 1) * 2.0 ** -24).all()
    ref = torch.zeros(P, N, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if there[t, j]:
                ref[plan.position[t, j].item()] = W[t, j] * G[t]
    bound = ref.abs() * (HALF[dtype] * (1 + 2.0 ** -9) + 2.0 ** -24) + TINY[dtype]
    assert ((y_grad.cpu().double() - ref).abs() <= bound).all()
    assert (y_grad.cpu()[plan.rows.cpu() < 0] == 0).all()


def test_combine_rows_past_32_bits():
    """Rows of y whose byte offsets pass 2^32."""
    P, N = 70000, 32768
    y = torch.empty(P, N, dtype=BF16, device="cuda")
    at = torch.tensor([[3, P - 1], [P - 2, 40000], [35000, -1]], dtype=torch.int32)
    g = gen(5)
    part = torch.randn(6, N, generator=g).to(BF16)
    for i, p in enumerate(at.reshape(-1).tolist()):
        if p >= 0:
            y[p] = part[i].cuda()
    rows = torch.full((P,), -1, dtype=torch.int32)
    for t in range(3):
        for p in at[t].tolist():
            if p >= 0:
                rows[p] = t
    i32 = lambda *x: torch.zeros(*x, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = dg.ExpertPlan(i32(2), i32(1), rows.cuda(), at.cuda())
    w, grad = torch.rand(3, 2, generator=g), torch.randn(3, N, generator=g).to(BF16)
    out = dg.gemm_experts_combine_tensors(y, plan, w.cuda()).cpu().double()
    yg, wg = dg.gemm_experts_combine_backward_tensors(y, plan, w.cuda(), grad.cuda())
    W = w.double() * (at >= 0)
    terms = part.double().reshape(3, 2, N) * W[:, :, None]
    ref = terms.sum(1)
    assert ((out - ref).abs() <= terms.abs().sum(1) * 2 * 2.0 ** -24 + ref.abs() * HALF[BF16] * (1 + 2.0 ** -9) + TINY[BF16]).all()
    for t in range(3):
        for j in range(2):
            p = at[t, j].item()
            if p < 0:
                assert wg[t, j].item() == 0
                continue
            want = W[t, j] * grad[t].double()
            assert ((yg[p].cpu().double() - want).abs() <= want.abs() * (HALF[BF16] * (1 + 2.0 ** -9) + 2.0 ** -24) + TINY[BF16]).all()
            size = (part[2 * t + j].double() * grad[t].double()).abs().sum()
            assert abs(wg[t, j].item() - (part[2 * t + j].double() * grad[t].double()).sum()) <= size * (N + 1) * 2.0 ** -24
    assert (yg[P - 3] == 0).all() and (yg[0] == 0).all()


def test_combine_backward_against_differences():
    g = gen(12)
    plan = dg.gemm_experts_dispatch_tensors(choice(g, 6, 5, 2).cuda(), 5, 1)
    y, w = torch.randn(12, 9, generator=g), torch.rand(6, 2, generator=g)
    grad, dy, dw = torch.randn(6, 9, generator=g), torch.randn(12, 9, generator=g), torch.randn(6, 2, generator=g)
    yg, wg = dg.gemm_experts_combine_backward_tensors(y.cuda(), plan, w.cuda(), grad.cuda())
    at = plan.position.cpu().long()

    def loss(a, b):
        return ((a[at.reshape(-1)].reshape(6, 2, 9) * b[:, :, None]).sum(1) * grad.double()).sum()

    h = 2.0 ** -10
    change = (loss(y.double() + h * dy.double(), w.double() + h * dw.double())
              - loss(y.double() - h * dy.double(), w.double() - h * dw.double())) / (2 * h)
    told = (yg.cpu().double() * dy.double()).sum() + (wg.cpu().double() * dw.double()).sum()
    # the loss is bilinear: central differences are exact but for 64-bit roundings over h
    size = (yg.cpu().double() * dy.double()).abs().sum() + (y.abs().sum() * grad.abs().max() * dw.abs().max()).double()
    assert (change - told).abs() <= size * (12 * 2.0 ** -24)


def test_whole_layer_on_a_graph():
    """Routing to combining, captured and replayed with new inputs, against eager calls."""
    g = gen(21)
    T, E, k, N, K = 48, 16, 4, 256, 384
    b = codes(g, N, K, E4, BLOCK, batch=E)
    B = dg.BlockTensor(b[0].cuda(), b[1].cuda(), BLOCK)
    x, logits = torch.randn(T, K, generator=g).to(BF16).cuda(), torch.randn(T, E, generator=g).cuda()
    r = dg.router(k, renorm=True)

    def layer():
        index, weight = dg.gemm_experts_route_tensors(logits, r)
        plan = dg.gemm_experts_dispatch_tensors(index, E, 128)
        a, _ = dg.gemm_block_quantize_tensors(x, E4)
        y = dg.gemm_experts_product_tensors(a, B, plan)
        out = dg.gemm_experts_combine_tensors(y, plan, weight)
        yg, wg = dg.gemm_experts_combine_backward_tensors(y, plan, weight, out)
        return out, yg, dg.gemm_experts_route_backward_tensors(logits, r, index, wg)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = layer()
    for _ in range(3):
        x.copy_(torch.randn(T, K, generator=g).to(BF16))
        logits.copy_(torch.randn(T, E, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        for a, b2 in zip(kept, layer()):
            assert torch.equal(a, b2)


def test_training_step_example():
    """The example's step against full precision: the only differences are the codes' roundings. A code is off by at
    most 2^-4 (e4m3) or 2^-3 (e5m2) of its value, so a product of two by less than (1 + 2^-4)(1 + 2^-3) - 1 = 0.2 of
    the terms' 2-norm; the out's gradient meets one more rounding to 16 bits."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts_step.py")
    spec = importlib.util.spec_from_file_location("experts_step", path)
    step = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(step)
    off = step.main(tokens=300, experts=6, top_k=2, inputs=256, outputs=384, repeat=1)
    assert off["out"] < 0.13 and off["x_grad"] < 0.2 and off["W_grad"] < 0.2 and off["logits_grad"] < 0.2, off

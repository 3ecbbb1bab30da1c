"""The adapters, the activations and the loss together, as a fine-tuning step uses them; captured
into graphs, on other streams and from several threads."""
import importlib.util
import os
import threading

import pytest
import torch

import block_util as bu
import dense_gemm_06_amd as dg
import layer_util as lu

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
E4 = torch.float8_e4m3fn


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapter_step.py")
    spec = importlib.util.spec_from_file_location("adapter_step", path)
    step = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(step)
    return step


def inputs(T, width, inner, words, R, rank, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    normal = lambda size, *s: (torch.randn(*s, generator=g) * size).to(dt).cuda()  # noqa: E731
    p = {"w_in": normal(width ** -0.5, 2 * inner, width), "w_out": normal(inner ** -0.5, width, inner),
         "a_in": normal(width ** -0.5, R, rank, width), "b_in": normal(rank ** -0.5, R, 2 * inner, rank),
         "a_out": normal(inner ** -0.5, R, rank, inner), "b_out": normal(rank ** -0.5, R, width, rank),
         "scale": torch.rand(R, generator=g).cuda() + 0.5, "head": normal(width ** -0.5, words, width)}
    x = normal(1.0, T, width)
    index = torch.randint(-1, R, (T,), generator=g, dtype=torch.int32).cuda()
    target = torch.randint(-3, words, (T,), generator=g).cuda()
    grad = torch.rand(T, generator=g).cuda() / T
    return x, p, index, target, grad


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_step_stage_by_stage(T, dt):
    """Each operator of the step against its definition on the very inputs that the step gave it."""
    x, p, index, target, grad = inputs(T, 136, 200, 515, 5, 12, dt, seed=T)
    step = example()
    loss, saved = step.forward(x, p, index, target)
    _, _, _, _, u_in, codes, u_out, h, lse = saved
    z, u = dg.gemm_adapters_tensors(x, p["w_in"], p["a_in"], p["b_in"], index, p["scale"], keep=True)
    assert torch.equal(u, u_in)
    ref, err, u_ref, u_err = lu.adapters(x, p["w_in"], p["a_in"], p["b_in"], index, p["scale"])
    lu.check(z, ref, err, "z")
    lu.check(u_in, u_ref, u_err, "u_in")
    y, again = dg.gemm_activation_tensors(z, "silu", True, E4)
    assert torch.equal(again.data.view(torch.uint8), codes.data.view(torch.uint8)) and torch.equal(again.scale, codes.scale)
    lu.check(y, *lu.activation(z, "silu", True), "y")
    ref, err, _, _ = lu.adapters(y, p["w_out"], p["a_out"], p["b_out"], index, p["scale"])
    lu.check(h, ref, err, "h")
    ref, err, lse_ref, lse_err, _, _ = lu.loss(h, p["head"], target)
    lu.check(loss, ref, err, "loss")
    lu.check(lse, lse_ref, lse_err, "lse")

    grads = step.backward(saved, grad)
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), 5)
    h_grad, _ = dg.gemm_loss_backward_tensors(grad, h, p["head"], target, lse, w_grad=False)
    ref, err = lu.loss_backward(grad, h, p["head"], target, lse)[0]
    lu.check(h_grad, ref, err, "h_grad")
    kept = bu.values(codes.data, codes.scale, 1)
    y2 = dg.gemm_activation_value_tensors(codes, "silu", True, dt)
    y_grad, a_out, b_out = dg.gemm_adapters_backward_tensors(h_grad, y2, u_out, p["w_out"], p["a_out"], p["b_out"],
                                                             index, plan, p["scale"])
    for name, have, (ref, err) in zip(("y_grad", "a_out", "b_out"), (y_grad, a_out, b_out), lu.adapters_backward(
            h_grad, y2, u_out, p["w_out"], p["a_out"], p["b_out"], index, p["scale"])):
        lu.check(have, ref, err, name)
    z_grad, y3 = dg.gemm_activation_backward_tensors(y_grad, codes, "silu", True)
    assert torch.equal(y2, y3)
    (ref, err), (y_ref, y_err) = lu.activation_backward(y_grad, kept, "silu", True)
    lu.check(z_grad, ref, err, "z_grad")
    lu.check(y2, y_ref, y_err, "y again")
    want = lu.adapters_backward(z_grad, x, u_in, p["w_in"], p["a_in"], p["b_in"], index, p["scale"])
    for name, (ref, err) in zip(("x", "a_in", "b_in"), want):
        lu.check(grads[name], ref, err, name)
    assert torch.equal(grads["a_out"], a_out) and torch.equal(grads["b_out"], b_out)


def test_example():
    """The example's step against full precision. A code is off by at most 2^-4 of its value, and so is the
    gate's value and slope by little more (|v s'| < 1.1 s at most): products of two of them by less than
    (1 + 1.1 2^-4)^2 - 1 = 0.15 of the terms' 2-norm. The loss does not meet the codes: its 16-bit
    roundings are 2^-8 each, three one after the other on the way to logits of about 1."""
    off = example().main(tokens=300, adapters=3, rank=8, width=128, inner=256, words=1000, repeat=1)
    assert off.pop("loss") < 3 * 2.0 ** -8 and all(v < 0.15 for v in off.values()), off


def on_graph(call, change, replays=3):
    """call captured once and replayed with changed inputs, eager calls between the replays."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call()
    for i in range(replays):
        change(i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, call()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [BF16, F16, F32])
@pytest.mark.parametrize("T", [3, 150, 700])
def test_step_on_a_graph(T, dt):
    x, p, index, target, grad = inputs(T, 128, 256, 1100, 4, 16, dt, seed=T)
    step = example()

    def call():
        loss, saved = step.forward(x, p, index, target)
        return [loss, *step.backward(saved, grad).values()]

    g = torch.Generator().manual_seed(1)

    def change(i):
        x.copy_(torch.randn(x.shape, generator=g))
        index.copy_(torch.randint(-1, 4, index.shape, generator=g))
        target.copy_(torch.randint(-3, 1100, target.shape, generator=g))

    on_graph(call, change)


def test_weight_gradient_on_a_graph():
    """Large enough for every kernel of the loss: wide and narrow tiles, copies of x, pieces."""
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(515, 256, generator=g).to(F16).cuda(), (torch.randn(9001, 256, generator=g) * 0.1).to(F16).cuda()
    target, grad = torch.randint(0, 9001, (515,), generator=g).cuda(), torch.rand(515, generator=g).cuda()

    def call():
        loss, lse = dg.gemm_loss_tensors(x, w, target)
        return [loss, lse, *dg.gemm_loss_backward_tensors(grad, x, w, target, lse, piece=4096)]

    on_graph(call, lambda i: x.copy_(torch.randn(x.shape, generator=g)))


def test_two_graphs_and_other_streams():
    """Two captured steps replayed at once on two streams do not share anything."""
    steps = []
    for seed in (3, 4):
        x, p, index, target, grad = inputs(200, 128, 256, 900, 4, 8, BF16, seed=seed)
        want = dg.gemm_loss_tensors(dg.gemm_adapters_tensors(x, p["w_in"], p["a_in"], p["b_in"], index, p["scale"])[:, :128],
                                    p["head"], target)

        def call(x=x, p=p, index=index, target=target):
            h = dg.gemm_adapters_tensors(x, p["w_in"], p["a_in"], p["b_in"], index, p["scale"])[:, :128]
            return dg.gemm_loss_tensors(h, p["head"], target)

        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            call()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                kept = call()
        steps.append((s, graph, kept, want))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph, _, _ in steps:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, kept, want in steps:
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_threads():
    """Calls of several threads, each on its own stream."""
    jobs, errors = [], []
    for seed in range(4):
        x, p, index, target, grad = inputs(90 + 70 * seed, 128, 256, 700, 3, 16, BF16, seed=seed)
        step = example()
        loss, saved = step.forward(x, p, index, target)
        jobs.append((x, p, index, target, grad, loss, step.backward(saved, grad)))
    torch.cuda.synchronize()

    def run(job):
        x, p, index, target, grad, loss, grads = job
        step = example()
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got, saved = step.forward(x, p, index, target)
                    have = step.backward(saved, grad)
                    torch.cuda.current_stream().synchronize()
                    assert torch.equal(got, loss) and all(torch.equal(have[n], grads[n]) for n in grads)
        except BaseException as e:  # noqa: BLE001  (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors, errors


def test_rows_behind_the_last_stay():
    """Outputs written through the C interface leave what lies around them alone."""
    T, N, K, R, rank = 70, 130, 72, 3, 12
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(T, K, generator=g).to(BF16).cuda(), torch.randn(N, K, generator=g).to(BF16).cuda()
    a, b = torch.randn(R, rank, K, generator=g).to(BF16).cuda(), torch.randn(R, N, rank, generator=g).to(BF16).cuda()
    index = torch.randint(-1, R, (T,), generator=g, dtype=torch.int32).cuda()
    want, u_want = dg.gemm_adapters_tensors(x, w, a, b, index, keep=True)
    lib = dg.library()
    y = torch.full((T + 2, N + 7), 7.0, dtype=BF16, device="cuda")
    u = torch.full((T + 2, rank), 7.0, device="cuda")
    s = dg.gemm_adapter_set(a.data_ptr(), b.data_ptr(), None, R, rank, K, rank * K, rank, N * rank)
    n = lib.gemm_adapters_workspace(T, N, K, rank, dg.GEMM_BF16)
    work = torch.full((n + 1024,), 165, dtype=torch.uint8, device="cuda")
    st = lib.gemm_adapters_product(x.data_ptr(), T, K, K, w.data_ptr(), N, K, dg.GEMM_BF16, s, index.data_ptr(),
                                   y[1:].data_ptr() + 2 * 3, N + 7, u[1:].data_ptr(), work.data_ptr(), n,
                                   torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(y[1:T + 1, 3:N + 3], want) and torch.equal(u[1:T + 1], u_want)
    assert (y[0] == 7).all() and (y[T + 1] == 7).all() and (y[1:T + 1, :3] == 7).all() and (y[1:T + 1, N + 3:] == 7).all()
    assert (u[0] == 7).all() and (u[T + 1] == 7).all() and (work[n:] == 165).all()

    V = 300
    w = torch.randn(V, K, generator=g).to(BF16).cuda()
    target, grad = torch.randint(0, V, (T,), generator=g).cuda(), torch.rand(T, generator=g).cuda()
    lse = dg.gemm_loss_tensors(x, w, target)[1]
    want = dg.gemm_loss_backward_tensors(grad, x, w, target, lse)
    xg = torch.full((T + 2, K + 5), 7.0, dtype=BF16, device="cuda")
    wg = torch.full((V + 2, K + 5), 7.0, dtype=BF16, device="cuda")
    n = lib.gemm_loss_backward_workspace(T, V, K, dg.GEMM_BF16, 1, 1, 0)
    work = torch.full((n + 1024,), 165, dtype=torch.uint8, device="cuda")
    st = lib.gemm_loss_backward(grad.data_ptr(), x.data_ptr(), T, K, K, w.data_ptr(), V, K, dg.GEMM_BF16,
                                target.data_ptr(), lse.data_ptr(), xg[1:].data_ptr(), K + 5, wg[1:].data_ptr(), K + 5, 0,
                                work.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    for have, ref in zip((xg, wg), want):
        assert torch.equal(have[1:-1, :K], ref)
        assert (have[0] == 7).all() and (have[-1] == 7).all() and (have[:, K:] == 7).all()
    assert (work[n:] == 165).all()


def test_broken_plans_stay_inside():
    """Plans whose arrays hold anything at all give some gradient, inside the arrays."""
    x, p, index, target, grad = inputs(100, 128, 64, 50, 4, 16, BF16, seed=6)
    y, u = dg.gemm_adapters_tensors(x, p["w_in"], p["a_in"], p["b_in"], index, p["scale"], keep=True)
    plan = dg.gemm_experts_dispatch_tensors(index[:, None].contiguous(), 4)
    g = torch.Generator().manual_seed(7)
    for low, high in ((-5, 300), (-2 ** 31, 2 ** 31 - 1)):
        broken = dg.ExpertPlan(*(torch.randint(low, high, t.shape, generator=g, dtype=torch.int32).cuda()
                                 for t in (plan.offsets, plan.counts, plan.rows, plan.position)))
        for dt in (BF16, F32):
            q = {n: t.to(dt) if n != "scale" else t for n, t in p.items()}
            xg, ag, bg = dg.gemm_adapters_backward_tensors(y.to(dt), x.to(dt), u, q["w_in"], q["a_in"], q["b_in"], index,
                                                           broken, q["scale"])
            torch.cuda.synchronize()
            assert xg.shape == x.shape and ag.shape == q["a_in"].shape and bg.shape == q["b_in"].shape

"""GPU tests of the block-scaled 8-bit operators: quantization and products, against their
definitions in 64 bits on the CPU."""
import pytest
import torch

import dense_gemm_06_amd as dg
from block_util import BLOCK, HALF, QMAX, blocks, check_product, codes, quantize, values

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(b):
    return dg.BlockTensor(b[0].cuda(), b[1].t().contiguous().t().cuda() if b[1].dim() == 2 else b[1].cuda(), b[2])


def same_codes(got, want):
    """Equal as bits, any NaN equal to any NaN."""
    g, w = got.cpu(), want
    nan = torch.isnan(w.float())
    assert torch.equal(torch.isnan(g.float()), nan)
    assert torch.equal(g.view(torch.uint8)[~nan], w.view(torch.uint8)[~nan])


def check_quantized(q, x, dtype, block_rows):
    want, scale = quantize(x, dtype, block_rows)
    same_codes(q.data, want)
    assert torch.equal(torch.nan_to_num(q.scale.cpu(), nan=-1.0), torch.nan_to_num(scale, nan=-1.0))
    assert q.scale.shape == scale.shape


# ----------------------------------------------------------------------------- quantize
@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (3, 130), (16, 4096), (127, 255), (129, 384), (200, 1000),
                                 (513, 129), (40, 7)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_quantize(M, K, dtype):
    g = gen(M * 1000 + K)
    x = (torch.randn(M, K, generator=g) * torch.exp(torch.randn(1, K, generator=g))).to(dtype)
    for qtype in (E4, E5):
        for block_rows in (1, BLOCK):
            q, t = dg.gemm_block_quantize_tensors(x.cuda(), qtype, block_rows, natural=True, transposed=True)
            check_quantized(q, x, qtype, block_rows)
            check_quantized(t, x.t().contiguous(), qtype, block_rows)
            q1, none = dg.gemm_block_quantize_tensors(x.cuda(), qtype, block_rows)
            assert none is None and torch.equal(q1.data.view(torch.uint8), q.data.view(torch.uint8))
            none, t1 = dg.gemm_block_quantize_tensors(x.cuda(), qtype, block_rows, natural=False, transposed=True)
            assert none is None and torch.equal(t1.data.view(torch.uint8), t.data.view(torch.uint8))


def test_quantize_half_a_step():
    """A code's number lies within half a step of its type of the value (2^-4, 2^-3 of it; the type's
    smallest step below its normal range), and two fp32 roundings."""
    x = torch.randn(300, 500, generator=gen(5))
    for qtype, half, least in ((E4, 2.0 ** -4, 2.0 ** -10), (E5, 2.0 ** -3, 2.0 ** -17)):
        q, _ = dg.gemm_block_quantize_tensors(x.cuda(), qtype)
        s = q.scale.cpu().double().repeat_interleave(BLOCK, 1)[:, :500]
        err = (values(q.data, q.scale, 1) - x.double()).abs()
        assert (err <= (x.double().abs() * half + s * least) * (1 + 2.0 ** -10) + x.double().abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("block_rows", [1, BLOCK])
def test_quantize_special_values(block_rows):
    """Zero blocks, tiny blocks below the floor, subnormals, infinities and NaNs."""
    x = torch.randn(300, 300, generator=gen(7))
    x[0] = 0
    x[1] = 1e-40
    x[2, :128] = 2.0 ** -101
    x[3, 5] = float("inf")
    x[4, 140] = float("nan")
    x[290, 290] = -float("inf")
    x[130:200, 130] = 0
    x[128:256, 256:] = 0
    for qtype in (E4, E5):
        q, t = dg.gemm_block_quantize_tensors(x.cuda(), qtype, block_rows, transposed=True)
        check_quantized(q, x, qtype, block_rows)
        check_quantized(t, x.t().contiguous(), qtype, block_rows)


@pytest.mark.parametrize("block_rows", [1, BLOCK])
def test_quantize_gather(block_rows):
    """Rows in any order, repeated, and out of range on both sides (zeros)."""
    g = gen(11)
    x = torch.randn(70, 200, generator=g).to(BF16)
    rows = torch.randint(-2, 72, (333,), generator=g).to(torch.int32)
    picked = torch.zeros(333, 200, dtype=BF16)
    ok = (rows >= 0) & (rows < 70)
    picked[ok] = x[rows[ok].long()]
    q, t = dg.gemm_block_quantize_tensors(x.cuda(), E4, block_rows, transposed=True, rows=rows.cuda())
    check_quantized(q, picked, E4, block_rows)
    check_quantized(t, picked.t().contiguous(), E4, block_rows)


def test_quantize_gather_from_no_rows():
    rows = torch.zeros(130, dtype=torch.int32, device="cuda")
    q, t = dg.gemm_block_quantize_tensors(torch.empty(0, 200, device="cuda"), E4, transposed=True, rows=rows)
    check_quantized(q, torch.zeros(130, 200), E4, 1)
    check_quantized(t, torch.zeros(200, 130), E4, 1)


def test_quantize_strided_input():
    x = torch.randn(100, 333, generator=gen(3)).to(BF16).cuda()
    view = x[5:77, 3:290]
    q, t = dg.gemm_block_quantize_tensors(view, E4, transposed=True)
    check_quantized(q, view.cpu(), E4, 1)
    check_quantized(t, view.cpu().t().contiguous(), E4, 1)


def test_quantize_empty():
    for shape in ((0, 64), (64, 0)):
        q, t = dg.gemm_block_quantize_tensors(torch.empty(shape, device="cuda"), E4, transposed=True)
        assert q.data.shape == shape and t.data.shape == shape[::-1]


# ----------------------------------------------------------------------------- products
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 512), (7, 33, 129), (16, 16, 2048), (17, 130, 300), (33, 64, 4096),
          (64, 256, 256), (65, 128, 128), (128, 128, 1024), (129, 257, 384), (100, 1000, 48), (300, 70, 1000),
          (512, 512, 640), (1000, 520, 272)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("b_rows", [1, BLOCK])
def test_product(M, N, K, b_rows):
    g = gen(M + 3 * N + 7 * K)
    outs = [BF16, F16, F32]
    for i, (ta, tb) in enumerate(((E4, E4), (E4, E5), (E5, E4), (E5, E5))):
        a, b = codes(g, M, K, ta, 1), codes(g, N, K, tb, b_rows)
        out = outs[(i + M) % 3]
        c = dg.gemm_block_product_tensors(dev((*a, 1)), dev((*b, b_rows)), out)
        check_product(c, values(*a, 1), values(*b, b_rows), out, (ta, tb, out))


@pytest.mark.parametrize("M,N,K", [(2048, 4096, 256), (4000, 3300, 400), (3000, 4100, 128), (2056, 4000, 1040)])
@pytest.mark.parametrize("b_rows", [1, BLOCK])
@pytest.mark.parametrize("out", [F32, BF16])
def test_product_many_tiles(M, N, K, b_rows, out):
    g = gen(M)
    a, b = codes(g, M, K, E4, 1), codes(g, N, K, E4, b_rows)
    c = dg.gemm_block_product_tensors(dev((*a, 1)), dev((*b, b_rows)), out)
    check_product(c, values(*a, 1), values(*b, b_rows), out)


def test_product_block_rows_of_a():
    g = gen(1)
    for M in (5, 200, 300):
        a, b = codes(g, M, 400, E4, BLOCK), codes(g, 260, 400, E4, BLOCK)
        c = dg.gemm_block_product_tensors(dev((*a, BLOCK)), dev((*b, BLOCK)), F32)
        check_product(c, values(*a, BLOCK), values(*b, BLOCK), F32)


@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (40, 96, 300), (256, 256, 512), (256, 8192, 128), (300, 200, 130)])
def test_product_exact_integers(M, N, K):
    """Small whole numbers with scales of powers of two: every partial sum is exact."""
    g = gen(9)
    a = torch.randint(-8, 9, (M, K), generator=g).float().to(E4)
    b = torch.randint(-8, 9, (N, K), generator=g).float().to(E4)
    sa = 2.0 ** torch.randint(-2, 3, (M, blocks(K)), generator=g).float()
    sb = 2.0 ** torch.randint(-2, 3, (N, blocks(K)), generator=g).float()
    c = dg.gemm_block_product_tensors(dev((a, sa, 1)), dev((b, sb, 1)), F32)
    assert torch.equal(c.cpu().double(), values(a, sa, 1) @ values(b, sb, 1).t())


def test_product_every_code():
    """Each code of each type times one, alone in its sum: its number comes back (NaN and infinity too)."""
    for t in (E4, E5):
        every = torch.arange(256, dtype=torch.uint8).view(t)
        for M in (256, 16):
            a = torch.zeros(256, 128).to(t)
            a[torch.arange(256), torch.arange(256) % 128] = every
            b = torch.zeros(128, 128).to(E4)
            for i in range(128):
                b[i, i] = 1.0
            a = a[:M]
            c = dg.gemm_block_product_tensors(dev((a, torch.ones(M, 1), 1)), dev((b, torch.ones(1, 1), BLOCK)), F32)
            got = c.cpu()[torch.arange(M), torch.arange(M) % 128]
            want = every[:M].float()
            fin = torch.isfinite(want)
            assert torch.equal(got[fin], want[fin])
            assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isinf(got), torch.isinf(want))


def test_product_nonfinite_scales_stay_in_their_block():
    g = gen(2)
    a, b = codes(g, 80, 300, E4, 1), codes(g, 140, 300, E4, 1)
    a[1][3, 1] = float("nan")
    b[1][7, 0] = float("inf")
    c = dg.gemm_block_product_tensors(dev((*a, 1)), dev((*b, 1)), F32).cpu()
    bad = torch.zeros(80, 140, dtype=torch.bool)
    bad[3] = True
    bad[:, 7] = True
    assert torch.equal(~torch.isfinite(c), bad)


def test_product_strides():
    """Views: odd leading dimensions and bases, scales with the blocks adjacent or broadcast."""
    g = gen(4)
    for M in (9, 90, 300):
        a, b = codes(g, M + 2, 520, E4, 1), codes(g, 203, 520, E5, 1)
        ad, bd = a[0].cuda()[2:, 3:403], b[0].cuda()[3:, 1:401]
        sa, sb = torch.rand(M, 4, generator=g) + 0.5, (torch.rand(1, 4, generator=g) + 0.5).expand(200, 4)
        c = dg.gemm_block_product_tensors(dg.BlockTensor(ad, sa.cuda(), 1), dg.BlockTensor(bd, sb.cuda(), 1), F32)
        check_product(c, values(ad, sa, 1), values(bd, sb, 1), F32)


@pytest.mark.parametrize("M,N,K", [(2, 2, 2), (16, 48, 300), (130, 200, 257), (256, 144, 512), (100, 333, 1000), (5, 400, 2048)])
def test_product_operands_with_adjacent_rows(M, N, K):
    """Codes stored transposed, for either operand and both, aligned and not; 128 x 128 blocks as their own transpose."""
    g = gen(M * N)
    for i, (ta, tb) in enumerate(((E4, E4), (E4, E5), (E5, E4), (E5, E5))):
        a, b = codes(g, M, K, ta, 1), codes(g, N, K, tb, BLOCK if i & 1 else 1)
        rb = BLOCK if i & 1 else 1
        flip = lambda x: x.cuda().t().contiguous().t()  # noqa: E731
        for fa, fb in ((False, True), (True, False), (True, True)):
            A = dg.BlockTensor(flip(a[0]) if fa else a[0].cuda(), a[1].cuda(), 1)
            B = dg.BlockTensor(flip(b[0]) if fb else b[0].cuda(), b[1].cuda(), rb)
            out = (F32, BF16)[(i + fa) % 2]
            check_product(dg.gemm_block_product_tensors(A, B, out), values(*a, 1), values(*b, rb), out, (ta, tb, fa, fb))
    w = codes(g, K, N, E4, BLOCK)
    W = dg.BlockTensor(w[0].cuda(), w[1].cuda(), BLOCK)
    a = codes(g, M, K, E4, 1)
    check_product(dg.gemm_block_product_tensors(dev((*a, 1)), W.t(), BF16), values(*a, 1), values(*w, BLOCK).t().contiguous(), BF16)


@pytest.mark.parametrize("M,ld", [(40, 1 << 27), (150, 1 << 25), (300, 1 << 24)])
def test_offsets_past_32_bits(M, ld):
    """Rows so far apart that byte offsets pass 2^32, for operands and for the quantizer's input."""
    g = gen(M)
    a, b = codes(g, M, 256, E4, 1), codes(g, 270, 256, E4, BLOCK)
    far = torch.empty(M * ld, dtype=torch.uint8, device="cuda").view(E4).view(M, ld)[:, :256]
    far.view(torch.uint8).copy_(a[0].view(torch.uint8))
    for out in (BF16, F32):
        c = dg.gemm_block_product_tensors(dg.BlockTensor(far, a[1].cuda(), 1), dev((*b, BLOCK)), out)
        check_product(c, values(*a, 1), values(*b, BLOCK), out)
        c = dg.gemm_block_product_tensors(dev((*b, BLOCK)), dg.BlockTensor(far, a[1].cuda(), 1), out)
        check_product(c, values(*b, BLOCK), values(*a, 1), out)
    del far
    x = torch.randn(M, 256, generator=g).to(BF16)
    far = torch.empty(M * ld // 2, dtype=BF16, device="cuda").view(M, ld // 2)[:, :256]
    far.copy_(x)
    q, t = dg.gemm_block_quantize_tensors(far, E4, transposed=True)
    check_quantized(q, x, E4, 1)
    check_quantized(t, x.t().contiguous(), E4, 1)


def test_product_empty():
    z = lambda r, k: dg.BlockTensor(torch.empty(r, k, dtype=E4, device="cuda"),  # noqa: E731
                                    torch.empty(r, blocks(k), device="cuda"), 1)
    assert dg.gemm_block_product_tensors(z(0, 128), z(5, 128)).shape == (0, 5)
    assert dg.gemm_block_product_tensors(z(5, 128), z(0, 128)).shape == (5, 0)
    for M in (5, 300):
        assert torch.equal(dg.gemm_block_product_tensors(z(M, 0), z(70, 0)), torch.zeros(M, 70, dtype=BF16, device="cuda"))


def test_product_side_stream_and_graph():
    """On a stream of its own, and captured: replays with new contents match eager calls."""
    g = gen(6)
    for M, N, K in ((8, 256, 4096), (256, 256, 1024)):
        a, b = dev((*codes(g, M, K, E4, 1), 1)), dev((*codes(g, N, K, E4, BLOCK), BLOCK))
        x = torch.randn(M, K, generator=g).to(BF16).cuda()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(2):
                q, _ = dg.gemm_block_quantize_tensors(x, E4)
                dg.gemm_block_product_tensors(q, b)
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q, _ = dg.gemm_block_quantize_tensors(x, E4)
            c = dg.gemm_block_product_tensors(q, b)
        for i in range(3):
            x.copy_(torch.randn(M, K, generator=g).to(BF16))
            graph.replay()
            torch.cuda.synchronize()
            q2, _ = dg.gemm_block_quantize_tensors(x, E4)
            assert torch.equal(c, dg.gemm_block_product_tensors(q2, b))


def test_repeated_calls_agree():
    g = gen(8)
    for M, N, K in ((4, 64, 8192), (100, 128, 4096), (512, 512, 1024)):
        a, b = dev((*codes(g, M, K, E4, 1), 1)), dev((*codes(g, N, K, E4, 1), 1))
        first = dg.gemm_block_product_tensors(a, b, F32)
        for _ in range(3):
            assert torch.equal(first, dg.gemm_block_product_tensors(a, b, F32))

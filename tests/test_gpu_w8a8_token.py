"""The W8A8 linear layer with a scale per token and per output channel:
codes and scales bit for bit, outputs within the rounding of the exact
product, over odd sizes, both types, strided rows, special rows, other
streams and captured graphs."""
import pytest
import torch

from tests import _layer_ref as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def sg():
    from sparse_bit_attention_smoothing_b200 import build
    build.build()
    import sparse_bit_attention_smoothing_b200 as s
    assert torch.cuda.is_available()
    return s


def inputs(M, N, K, dtype, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, K, generator=g) * torch.linspace(0.1, 4.0, K)).to(dtype).cuda()
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(dtype).cuda()
    b = torch.randn(N, generator=g).to(dtype).cuda() if bias else None
    return x, w, b


def check(y, xq, sx, wq, sw, b, dtype):
    r, tol = ref.token_linear(xq, sx, wq, sw, b, dtype)
    ref.inside(y, r, tol, "y")


@pytest.mark.parametrize("rows,cols,dtype", [(1, 16, BF), (1, 5120, BF), (77, 256, HF), (300, 1040, BF), (5, 13824, HF),
                                             (1000, 48, HF), (3, 131056, BF)])
def test_quant_bit_exact(sg, rows, cols, dtype):
    x, _, _ = inputs(rows, 1, cols, dtype, rows + cols)
    if rows > 2:
        x[1] = 0
        x[2, 0] = 2 * x[2].abs().max()  # halves fall on ties of the codes
        x[2, 1:] = x[2, 0] / 2
    codes, scales = sg.sagesla_w8a8_token_quant(x)
    q, s = ref.token_quant(x)
    assert torch.equal(codes.double().cpu(), q) and torch.equal(scales.double().cpu(), s)


def test_quant_special_rows(sg):
    x = torch.randn(9, 64).bfloat16()
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 6] = float("nan")
    x[3, 7] = float("-inf")
    x[4] = 2.0 ** -101
    x[5] = 2.0 ** -100
    x[6] = 2.0 ** -130
    x[7] = -3.0e38
    x[8, 1:] = 0
    q, s = ref.token_quant(x)
    codes, scales = sg.sagesla_w8a8_token_quant(x.cuda())
    assert torch.equal(codes.double().cpu(), q)
    assert torch.equal(torch.nan_to_num(scales.double().cpu(), nan=-1.0), torch.nan_to_num(s, nan=-1.0))
    w = torch.randn(40, 64).bfloat16().cuda()
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    y = sg.sagesla_w8a8_token_linear(x.cuda(), wq, sw).cpu()
    assert torch.isnan(y[1:4]).all() and not torch.isnan(y[[0, 4, 5, 6, 8]]).any() and not y[[0, 4, 6]].any()


SIZES = [  # M, N, K: both sides of every tile edge, one, odd, long
    (1, 1, 16), (1, 5120, 5120), (2, 33, 48), (3, 1001, 640), (4, 129, 2048), (7, 64, 13824), (8, 13, 1040), (9, 77, 80),
    (15, 256, 256), (16, 100, 5120), (17, 1280, 1280), (31, 95, 112), (32, 96, 96), (33, 257, 528), (63, 63, 64),
    (64, 65, 144), (65, 512, 1536), (100, 1001, 208), (127, 127, 128), (128, 128, 128), (129, 129, 144), (200, 333, 5120),
    (255, 256, 384), (256, 255, 256), (257, 513, 272), (333, 1001, 1280), (512, 384, 1024), (513, 2049, 160),
    (1000, 1536, 1536), (1025, 5120, 256), (4000, 129, 400), (2500, 4999, 64),
]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear(sg, M, N, K, dtype):
    x, w, b = inputs(M, N, K, dtype, M + N + K, bias=(M + N) % 2 == 0)
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    y = sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b)
    torch.cuda.synchronize()
    assert sg.sync_status() == 0
    qx, sx = ref.token_quant(x)
    check(y, qx, sx, wq, sw, b, dtype)
    xq, sx = sg.sagesla_w8a8_token_quant(x)
    y2 = sg.sagesla_w8a8_token_gemm(xq, sx, wq, sw, bias=b, dtype=dtype)
    check(y2, xq, sx, wq, sw, b, dtype)
    assert torch.equal(y, y2)  # the sums are exact: any order gives the same bits


@pytest.mark.parametrize("M", [1, 12, 40, 300])
def test_gemm_extreme_codes(sg, M):
    """All of int8 over the longest K: the sums reach 2^14 K and stay exact."""
    K, N = 131056, 40
    xq = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    wq = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    wq[1] = 127
    wq[2, ::2] = 127
    sx, sw = torch.full((M,), 0.5, device="cuda"), torch.full((N,), 2.0 ** -20, device="cuda")
    y = sg.sagesla_w8a8_token_gemm(xq, sx, wq, sw)
    check(y, xq, sx, wq, sw, None, BF)


@pytest.mark.parametrize("M", [1, 3, 37, 260])
def test_strided_rows_and_given_output(sg, M):
    x, w, b = inputs(M, 200, 320, BF, M)
    wide = torch.full((M, 3 * 320 + 8), float("nan"), dtype=BF, device="cuda")
    xs = wide[:, 320:640]
    xs.copy_(x)
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    y = torch.full((M, 200), float("nan"), dtype=BF, device="cuda")
    assert sg.sagesla_w8a8_token_linear(xs, wq, sw, bias=b, y=y) is y
    assert torch.equal(y, sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b))
    codes, scales = sg.sagesla_w8a8_token_quant(xs)
    want = sg.sagesla_w8a8_token_quant(x)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("M,N,K", [(1, 77, 256), (20, 33, 256), (200, 301, 256), (700, 129, 512)])
def test_nothing_past_the_output(sg, M, N, K):
    x, w, b = inputs(M, N, K, HF, 3)
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    buf = torch.full((M * N + 512,), 7.0, dtype=HF, device="cuda")
    y = buf[:M * N].view(M, N)
    sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b, y=y)
    assert (buf[M * N:] == 7).all()
    qx, sx = ref.token_quant(x)
    check(y, qx, sx, wq, sw, b, HF)


def test_many_tiles_sampled(sg):
    """More output tiles than SMs many times over; sampled rows in full."""
    M, N, K = 20011, 1536, 1536
    x, w, b = inputs(M, N, K, BF, 11)
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    y = sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b)
    rows = torch.cat([torch.arange(0, M, 97), torch.arange(M - 130, M)])
    qx, sx = ref.token_quant(x[rows.cuda()])
    check(y[rows.cuda()], qx, sx, wq, sw, b, BF)
    assert sg.sync_status() == 0


def test_output_offsets_past_32_bits(sg):
    """y of more than 2^31 elements; its last rows in full."""
    M, N, K = 270011, 8192, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    xq = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sx, sw = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    y = sg.sagesla_w8a8_token_gemm(xq, sx, wq, sw)
    for r in (slice(0, 3), slice(262140, 262150), slice(M - 150, M)):
        check(y[r], xq[r], sx[r], wq, sw, None, BF)


@pytest.mark.parametrize("M", [1, 24, 300])
def test_other_stream_and_captured(sg, M):
    x, w, b = inputs(M, 640, 1280, BF, 2)
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    want = sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    graphs, xs, outs = [], [x.clone(), x.clone()], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sg.sagesla_w8a8_token_linear(xs[i], wq, sw, bias=b))
        graphs.append(g)
    xs[1].neg_()
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):  # both at once: each graph has its own workspace
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want)
    assert torch.equal(outs[1], sg.sagesla_w8a8_token_linear(xs[1], wq, sw, bias=b))
    assert sg.sync_status() == 0


@pytest.mark.parametrize("N,K", [(5120, 5120), (77, 16), (129, 144), (1000, 1168), (300, 13824), (40000, 5120), (130, 131056)])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
def test_linear_is_quantiser_and_product(sg, M, N, K):
    # one call of the layer: the same bits as its two halves, special rows too
    x, w, b = inputs(M, N, K, HF if M % 2 else BF, M + K)
    if M > 2:
        x[1] = 0
        x[2, K - 1] = float("nan")
    if M > 4:
        x[3] = 2.0 ** -20 if x.dtype == HF else 2.0 ** -110
        x[4, 0] = float("inf")
    wq, sw = sg.sagesla_w8a8_token_quant(w)
    xq, sx = sg.sagesla_w8a8_token_quant(x)
    want = sg.sagesla_w8a8_token_gemm(xq, sx, wq, sw, bias=b, dtype=x.dtype)
    got = sg.sagesla_w8a8_token_linear(x, wq, sw, bias=b)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))

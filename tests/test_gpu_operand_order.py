"""Codes that one call writes and the next reads as its second operand, with no
synchronisation between: products of two activations, and weights written right
before they are used.  The products request that operand before the previous kernel
has ended, so no kernel that writes codes may let them start early."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROUNDS = 24     # calls in a row, each on other inputs, through the same buffers


@pytest.fixture(scope="module")
def w8():
    import w4a8_int8_quantized_gb300 as w8
    from w4a8_int8_quantized_gb300 import build
    build.build()
    yield w8
    assert w8.w8a8_check_status() == 0


def half(*shape, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=gen).half()


class Codes:
    """Buffers of [rows, cols] codes that every round writes again."""

    def __init__(self, rows, cols):
        self.q = torch.full((rows, cols), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        self.s = torch.full((rows, -(-cols // 128)), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)


def chains(w8, M, N, K):
    """name -> f(round, y), each a few calls in a row that end in y [M, N]."""
    x, k = [half(M, K, seed=i) for i in range(3)], [half(N, K, seed=10 + i) for i in range(3)]
    nw = half(1, K, seed=20)[0]
    a, b, c = Codes(M, K), Codes(N, K), Codes(N, K)
    g, d = Codes(N, 256), Codes(M, 256)
    values = torch.empty(M, K, dtype=torch.float16, device="cuda")
    wk = w8.quantize_weight_fp8(half(256, K, seed=30) / 16)
    wx = half(M, 256, seed=31)
    ws = torch.empty(w8.fp8_feed_forward_workspace_bytes(M, K, N) + 256, dtype=torch.uint8, device="cuda")
    down = w8.quantize_weight_fp8(half(N, N, seed=32) / 16) if N % 16 == 0 else None

    def two_norms(i, y):
        w8.rms_norm_quantize(k[i % 3], nw, codes="fp8", q=b.q, scale=b.s)
        w8.rms_norm_quantize(x[i % 3], nw, codes="fp8", q=a.q, scale=a.s)
        w8.fp8_gemm(a.q, a.s, b.q, b.s, y=y)

    def second_operand_last(i, y):
        w8.rms_norm_quantize(x[i % 3], nw, codes="fp8", q=a.q, scale=a.s)
        w8.rms_norm_quantize(k[i % 3], nw, codes="fp8", q=b.q, scale=b.s)
        w8.fp8_gemm(a.q, a.s, b.q, b.s, y=y)

    def two_quantizers(i, y):
        w8.quantize_act_fp8(x[i % 3], a.q, a.s)
        w8.quantize_act_fp8(k[i % 3], b.q, b.s)
        w8.fp8_gemm(a.q, a.s, b.q, b.s, y=y)

    def kernels_between(i, y):
        # the norm of values lets the layer start early, and waits after it has said so
        w8.quantize_act_fp8(k[i % 3], b.q, b.s)
        w8.rms_norm(x[i % 3], nw, y=values)
        w8.fp8_linear(values, b.q, b.s, workspace=ws, y=y)

    def weights_between(i, y):
        w8.quantize_weight_fp8(k[i % 3], b.q, b.s)
        w8.rms_norm_quantize(x[i % 3], nw, codes="fp8", q=a.q, scale=a.s)
        w8.fp8_gemm(a.q, a.s, b.q, b.s, y=y)

    def layer(i, y):
        w8.quantize_act_fp8(k[i % 3], b.q, b.s)
        w8.fp8_linear(x[i % 3], b.q, b.s, workspace=ws, y=y)

    def hidden(i, y):
        # the gated pair's codes as the second operand of a product
        w8.quantize_act_fp8(k[i % 3], b.q, b.s)
        w8.quantize_act_fp8(wx, d.q, d.s)
        w8.fp8_gated_gemm(b.q, b.s, *wk, *wk, codes=True, h=g.q, scale_h=g.s)
        w8.fp8_gemm(d.q, d.s, g.q, g.s, y=y)

    def gated(i, y):
        w8.quantize_act_fp8(x[i % 3], a.q, a.s)
        w8.rms_norm_quantize(k[i % 3], nw, codes="fp8", q=b.q, scale=b.s)
        w8.quantize_act_fp8(k[(i + 1) % 3], c.q, c.s)
        w8.fp8_gated_gemm(a.q, a.s, b.q, b.s, c.q, c.s, h=y)

    def block(i, y):
        w8.quantize_act_fp8(k[i % 3], b.q, b.s)
        w8.quantize_act_fp8(k[(i + 1) % 3], c.q, c.s)
        w8.fp8_feed_forward(x[i % 3], b.q, b.s, c.q, c.s, *down, workspace=ws, y=y)

    return {f.__name__: f for f in (two_norms, second_operand_last, two_quantizers, kernels_between, weights_between,
                                    layer, hidden, gated) + ((block,) if down else ())}


def check(f, shape):
    want = []
    for i in range(3):
        y = torch.empty(shape, dtype=torch.float16, device="cuda")
        f(i, y)           # whatever this read, the buffers now hold round i
        torch.cuda.synchronize()
        f(i, y)
        torch.cuda.synchronize()
        want.append(y)
    assert not torch.equal(want[0], want[1])
    got = [torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(ROUNDS)]
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        f(i, y)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3]), i
    graph = torch.cuda.CUDAGraph()
    for y in got:
        y.zero_()
    with torch.cuda.graph(graph):
        for i, y in enumerate(got):
            f(i, y)
    graph.replay()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 3]), i


NAMES = ["two_norms", "second_operand_last", "two_quantizers", "kernels_between", "weights_between", "layer", "hidden",
         "gated", "block"]


# grids small enough to run beside one another, and a second operand that takes long to write
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("M,N,K", [(1, 256, 256), (16, 256, 256), (40, 256, 2560), (100, 1024, 256), (200, 512, 272),
                                   (8, 8192, 512), (1500, 256, 256)])
def test_codes_just_written_as_the_second_operand(w8, name, M, N, K):
    check(chains(w8, M, N, K)[name], (M, N))


@pytest.mark.parametrize("N,K", [(256, 256), (4096, 512), (300, 2048)])
@pytest.mark.parametrize("call", ["mv", "layer", "rows"])
def test_int8_codes_just_written_as_the_second_operand(w8, call, N, K):
    """The same for the matrix-vector kernels, which read INT8 weights as early."""
    M = 4 if call == "rows" else 1
    x, k = [half(M, K, seed=i) for i in range(3)], [half(N, K, seed=10 + i) for i in range(3)]
    nw = half(1, K, seed=20)[0]
    q, s = torch.zeros(N, K, dtype=torch.int8, device="cuda"), torch.zeros(N, 1, device="cuda")
    xq, xs = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, 1, device="cuda")
    ws = torch.empty(w8.w8a8_linear_workspace_bytes(M, K, 0), dtype=torch.uint8, device="cuda")
    values = torch.empty(M, K, dtype=torch.float16, device="cuda")

    def f(i, y):
        if call == "mv":
            w8.rms_norm_quantize(x[i % 3], nw, q=xq, scale=xs)
            w8.rms_norm_quantize(k[i % 3], nw, q=q, scale=s)
            w8.w8a8_mv(xq, xs, q, s, y=y)
        else:
            w8.rms_norm_quantize(k[i % 3], nw, q=q, scale=s)
            if i % 2:
                w8.rms_norm(x[i % 3], nw, y=values)      # a kernel between that lets the next start early
            w8.linear(x[i % 3], q, s, workspace=ws, y=y)

    check(f, (M, N))

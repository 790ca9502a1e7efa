"""The products in 8-bit floats: the layer, the gated pair and the whole block."""
import pytest

torch = pytest.importorskip("torch")
import fp8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w8():
    import w4a8_int8_quantized_gb300 as w8
    from w4a8_int8_quantized_gb300 import build
    build.build()
    yield w8
    assert w8.w8a8_check_status() == 0


def rows(M, K, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=gen)
    x *= 1 + 30 * (torch.rand(K, device="cuda", generator=gen) > 0.98)
    x *= 0.1 + 3 * torch.rand(M, 1, device="cuda", generator=gen)
    return x.half()


def weights(w8, N, K, seed=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    w = torch.randn(N, K, device="cuda", generator=gen) * K ** -0.5
    w *= 0.05 + 2 * torch.rand(N, 1, device="cuda", generator=gen)
    return w8.quantize_weight_fp8(w.half())


def framed(shape, dtype):
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    pad = -n % 256 + 256
    raw = torch.full((256 + n + pad,), 0xA5, dtype=torch.uint8, device="cuda")
    return raw[256:256 + n].view(dtype).view(shape), lambda: bool((raw[:256] == 0xA5).all() and (raw[256 + n:] == 0xA5).all())


# rows around every change of kernel and tile, K with a short last group, with
# an odd number of groups, of one group and of many; N odd, small, one tile and more
PRODUCTS = [(1, 1, 16), (1, 77, 48), (2, 16, 128), (5, 640, 2560), (8, 130, 144), (9, 129, 400), (13, 1000, 4096),
            (16, 257, 1040), (17, 64, 128), (17, 1001, 1296), (32, 511, 640), (64, 256, 2560), (65, 120, 80),
            (100, 2560, 2560), (127, 333, 528), (128, 128, 512), (129, 8, 1536), (130, 700, 656), (200, 1, 272),
            (256, 256, 1024), (257, 515, 784), (300, 1032, 16), (511, 2056, 1168), (1000, 96, 2064), (513, 5003, 640),
            (2049, 776, 528), (3, 24, 32768), (140, 264, 32768), (5000, 520, 256)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(w8, M, N, K):
    x, wq = rows(M, K), weights(w8, N, K)
    xq = w8.quantize_act_fp8(x)
    y, fine = framed((M, N), torch.float16)
    w8.fp8_gemm(*xq, *wq, y=y)
    ref.check_product(y, *ref.product(ref.values(*xq), ref.values(*wq)))
    assert fine()
    assert torch.equal(w8.fp8_linear(x, *wq), y)


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("M,F,K", [(1, 16, 16), (1, 640, 2560), (3, 144, 144), (8, 1008, 4096), (11, 272, 656),
                                   (16, 128, 528), (17, 16, 128), (40, 400, 272), (128, 128, 1280), (129, 1296, 528),
                                   (255, 48, 2560), (300, 2064, 784), (777, 512, 400), (2100, 1168, 272)])
def test_gated(w8, M, F, K, gelu):
    x = w8.quantize_act_fp8(rows(M, K))
    wg, wu = weights(w8, F, K, 2), weights(w8, F, K, 3)
    h, err = ref.gated(ref.values(*x), ref.values(*wg), ref.values(*wu), gelu)
    kind = "gelu" if gelu else "silu"
    y, fine = framed((M, F), torch.float16)
    w8.fp8_gated_gemm(*x, *wg, *wu, activation=kind, h=y)
    assert fine()
    ref.check_product(y, h, err)
    q, fine = framed((M, F), torch.float8_e4m3fn)
    s, fine_too = framed((M, -(-F // 128)), torch.float8_e8m0fnu)
    w8.fp8_gated_gemm(*x, *wg, *wu, activation=kind, codes=True, h=q, scale_h=s)
    assert fine() and fine_too()
    ref.check_fp8(q, s, h, err)


@pytest.mark.parametrize("M", [1, 7, 16, 17, 150, 600])
def test_gated_values_of_any_width(w8, M):
    """fp16 out needs no group: odd widths."""
    for F in (1, 77, 131, 259):
        x = w8.quantize_act_fp8(rows(M, 272))
        wg, wu = weights(w8, F, 272, 2), weights(w8, F, 272, 3)
        y, fine = framed((M, F), torch.float16)
        w8.fp8_gated_gemm(*x, *wg, *wu, h=y)
        assert fine()
        ref.check_product(y, *ref.gated(ref.values(*x), ref.values(*wg), ref.values(*wu)))


@pytest.mark.parametrize("M,K,F,N", [(1, 256, 640, 256), (4, 2560, 10240, 2560), (16, 144, 400, 77), (17, 144, 400, 77),
                                     (200, 528, 1296, 528), (700, 1024, 2064, 1000)])
def test_block(w8, M, K, F, N):
    """The whole block is its parts, one after the other."""
    x = rows(M, K)
    wg, wu, wd = weights(w8, F, K, 2), weights(w8, F, K, 3), weights(w8, N, F, 4)
    for kind in ("silu", "gelu"):
        h = w8.fp8_gated_gemm(*w8.quantize_act_fp8(x), *wg, *wu, activation=kind, codes=True)
        y = w8.fp8_feed_forward(x, *wg, *wu, *wd, activation=kind)
        assert torch.equal(y, w8.fp8_gemm(*h, *wd))
    ref.check_product(y, *ref.product(ref.values(*h), ref.values(*wd)))


def test_scales_far_apart(w8):
    """Scale bytes over their whole useful range, on both operands."""
    gen = torch.Generator("cuda").manual_seed(0)
    for M in (1, 16, 200):
        for K in (272, 1536):
            G = -(-K // 128)
            x, w = (torch.randn(n, K, device="cuda", generator=gen).to(torch.float8_e4m3fn) for n in (M, 160))
            sx = torch.randint(97, 158, (M, G), device="cuda", generator=gen).to(torch.uint8).view(torch.float8_e8m0fnu)
            sw = torch.randint(80, 120, (160, G), device="cuda", generator=gen).to(torch.uint8).view(torch.float8_e8m0fnu)
            y = w8.fp8_gemm(x, sx, w, sw)
            want, err = ref.product(ref.values(x, sx), ref.values(w, sw))
            fits = want.abs() + err < 65000
            diff = (y.double() - want).abs()
            assert (diff <= want.abs() * 2.0 ** -11 + 2.0 ** -25 + 1.001 * err)[fits].all()
            assert y[want.abs() - err > 65520].isinf().all()


def test_every_code(w8):
    """Every e4m3 code but NaN, against ones and against itself: exact sums."""
    every = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn)
    every = every[every.float().isfinite()]
    one = torch.full((1, 2), 127, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    for M in (len(every), 16):
        x = torch.zeros(M, 144, device="cuda")
        x[torch.arange(M), torch.arange(M) % 144] = every[:M].float()
        w = torch.zeros(150, 144, device="cuda")
        w[:144, :144] = torch.eye(144, device="cuda")
        y = w8.fp8_gemm(x.to(torch.float8_e4m3fn), one.expand(M, 2).contiguous(), w.to(torch.float8_e4m3fn),
                        one.expand(150, 2).contiguous())
        assert torch.equal(y.float(), x @ w.T)


def test_each_scale_reaches_its_group(w8):
    """One nonzero group at a time, with a scale of its own on either side: exact."""
    for M in (3, 16, 140, 300):
        K, N = 128 * 13 + 16, 300
        G = 14
        x, w = torch.ones(M, K, device="cuda"), torch.ones(N, K, device="cuda")
        sx = (120 + (torch.arange(M)[:, None] * 3 + torch.arange(G)[None] * 5) % 11).to(torch.uint8).cuda()
        sw = (121 + (torch.arange(N)[:, None] * 7 + torch.arange(G)[None] * 3) % 9).to(torch.uint8).cuda()
        for g in (0, 1, 2, 3, 4, 7, 8, 12, 13):
            part = torch.zeros_like(x)
            part[:, 128 * g:128 * g + 128] = 1
            y = w8.fp8_gemm(part.to(torch.float8_e4m3fn), sx.view(torch.float8_e8m0fnu), w.to(torch.float8_e4m3fn),
                            sw.view(torch.float8_e8m0fnu))
            n = min(128, K - 128 * g)
            want = n * ref.bits(sx[:, g].long()[:, None] + sw[:, g].long()[None] - 254)
            assert (y.double() == want).all()


@pytest.mark.parametrize("M", [1, 12, 64, 300])
def test_slices_of_fused_weights(w8, M):
    """Row slices of one tensor, whose scale rows start at any address."""
    K, F = 272, 75
    wq, sw = weights(w8, 2 * F + 1, K)
    x = w8.quantize_act_fp8(rows(M, K))
    whole = w8.fp8_gemm(*x, wq, sw)
    assert torch.equal(w8.fp8_gemm(*x, wq[1:], sw[1:]), whole[:, 1:])
    h = w8.fp8_gated_gemm(*x, wq[:F], sw[:F], wq[F:2 * F], sw[F:2 * F])
    y = w8.fp8_gated_gemm(*x, wq[:F].clone(), sw[:F].clone(), wq[F:2 * F].clone(), sw[F:2 * F].clone())
    assert torch.equal(h, y)


def test_rows_do_not_depend_on_their_neighbours(w8):
    """A row's result is the same in every batch that runs on the same kernel."""
    K, N = 1296, 515
    wq = weights(w8, N, K)
    x = rows(600, K)
    whole = w8.fp8_linear(x, *wq)
    assert torch.equal(w8.fp8_linear(x[:400].contiguous(), *wq), whole[:400])
    assert torch.equal(w8.fp8_linear(x[:600].flip(0).contiguous(), *wq).flip(0), whole)
    few = w8.fp8_linear(x[:16].contiguous(), *wq)
    assert torch.equal(w8.fp8_linear(x[8:16].contiguous(), *wq), few[8:16])


@pytest.mark.parametrize("M", [1, 16, 90, 600])
def test_streams_graphs_and_stale_workspaces(w8, M):
    K, F = 528, 1296
    wg, wu, wd = weights(w8, F, K, 2), weights(w8, F, K, 3), weights(w8, K, F, 4)
    x = rows(M, K)
    want = w8.fp8_feed_forward(x, *wg, *wu, *wd)
    need = w8.fp8_feed_forward_workspace_bytes(M, K, F)
    spaces = [torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s, ws in zip(streams, spaces):           # two calls at once, each with its workspace
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(4):
                y = w8.fp8_feed_forward(x, *wg, *wu, *wd, workspace=ws)
            outs.append(y)
    for s, y in zip(streams, outs):
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    ws = spaces[0]
    with torch.cuda.graph(graph):
        y = w8.fp8_feed_forward(x, *wg, *wu, *wd, workspace=ws)
        z = w8.fp8_linear(y, *wg, workspace=ws)
    x2 = rows(M, K, 50)
    x.copy_(x2)
    ws.fill_(0xFF)
    graph.replay()
    assert torch.equal(y, w8.fp8_feed_forward(x2, *wg, *wu, *wd))
    assert torch.equal(z, w8.fp8_linear(y, *wg))
    with pytest.raises(w8.W8A8Error) as e:
        w8.fp8_feed_forward(x, *wg, *wu, *wd, workspace=ws[:need - 256])
    assert e.value.status == 6


def test_refusals(w8):
    x, wq = rows(4, 256), weights(w8, 48, 256)
    xq = w8.quantize_act_fp8(x)
    with pytest.raises(ValueError):
        w8.fp8_gemm(xq[0], xq[1][:, :1], *wq)
    with pytest.raises(ValueError):
        w8.fp8_gemm(xq[0][:, :128], xq[1], *wq)
    with pytest.raises(ValueError):
        w8.fp8_gemm(xq[0][:, :128].contiguous(), xq[1][:, :1].contiguous(), *wq)
    with pytest.raises(TypeError):
        w8.fp8_gemm(xq[0], xq[1].view(torch.uint8), *wq)
    with pytest.raises(TypeError):
        w8.fp8_linear(x, wq[0].view(torch.uint8), wq[1])
    with pytest.raises(ValueError):
        w8.fp8_linear(x, *wq, y=torch.empty(4, 47, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        w8.fp8_linear(x, *wq, workspace=torch.empty(4096, device="cuda"))
    with pytest.raises(ValueError):
        w8.fp8_gated_gemm(*xq, *wq, wq[0][:32], wq[1][:32])
    with pytest.raises(ValueError):
        w8.fp8_gated_gemm(*xq, *wq, *wq, scale_h=xq[1])
    with pytest.raises(w8.W8A8Error):
        w8.fp8_gated_gemm(*xq, wq[0][:40], wq[1][:40], wq[0][:40], wq[1][:40], codes=True)
    assert w8.fp8_linear(x[:0], *wq).shape == (0, 48)
    assert w8.fp8_gemm(*xq, wq[0][:0], wq[1][:0]).shape == (4, 0)

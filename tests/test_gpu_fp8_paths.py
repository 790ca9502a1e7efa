"""The 8-bit float products by the way they take: tiles, parts of K, fused
quantization, long offsets, waits that run out; and the norm, the projections and
the feed-forward block together, as a decoder layer calls them."""
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
    return w8.quantize_weight_fp8(w.half())


# classes of batches: the order of a sum is the same throughout
CLASSES = [(1, 3, 7, 16), (17, 33, 64), (65, 100, 128), (129, 257, 384), (385, 700, 1024), (1025, 1800, 2049)]


@pytest.mark.parametrize("N,K", [(64, 8192), (515, 1296), (4096, 4112), (2048, 14336)])
@pytest.mark.parametrize("sizes", CLASSES)
def test_rows_do_not_depend_on_the_batch(w8, sizes, N, K):
    wq = weights(w8, N, K)
    x = rows(sizes[-1], K)
    whole = w8.fp8_linear(x, *wq)
    for m in sizes[:-1]:
        assert torch.equal(w8.fp8_linear(x[:m].contiguous(), *wq), whole[:m])
        assert torch.equal(w8.fp8_linear(x[-m:].contiguous(), *wq), whole[-m:])


@pytest.mark.parametrize("sizes", CLASSES)
def test_gated_rows_do_not_depend_on_the_batch(w8, sizes):
    F, K = 1040, 2576
    wg, wu = weights(w8, F, K, 2), weights(w8, F, K, 3)
    x = w8.quantize_act_fp8(rows(sizes[-1], K))
    for codes in (False, True):
        whole = w8.fp8_gated_gemm(*x, *wg, *wu, codes=codes)
        for m in sizes[:-1]:
            part = w8.fp8_gated_gemm(x[0][:m], x[1][:m], *wg, *wu, codes=codes)
            if codes:
                assert torch.equal(part[0].view(torch.uint8), whole[0][:m].view(torch.uint8))
                assert torch.equal(part[1].view(torch.uint8), whole[1][:m].view(torch.uint8))
            else:
                assert torch.equal(part, whole[:m])


@pytest.mark.parametrize("M", [1, 2, 5, 8, 16, 31, 32])
@pytest.mark.parametrize("K", [16, 128, 144, 512, 656, 2048, 4096, 4112, 8192, 14336, 32768])
def test_few_rows_quantized_on_the_way(w8, M, K):
    """One kernel or two: the same bits, and right; workspaces that hold NaN codes."""
    x, wq = rows(M, K), weights(w8, 80, K)
    ws = torch.full((w8.fp8_linear_workspace_bytes(M, K),), 0xFF, dtype=torch.uint8, device="cuda")
    y = w8.fp8_linear(x, *wq, workspace=ws)
    xq = w8.quantize_act_fp8(x)
    assert torch.equal(y, w8.fp8_gemm(*xq, *wq))
    ref.check_product(y, *ref.product(ref.values(*xq), ref.values(*wq)))


def test_few_rows_of_zeros_and_extremes(w8):
    K = 656
    wq = weights(w8, 80, K)
    x = torch.zeros(6, K, device="cuda").half()
    x[1, 130] = 6e-8       # the smallest half
    x[2, :] = 65504
    x[3, 650] = -65504
    x[4] = rows(1, K)[0]
    y = w8.fp8_linear(x, *wq)
    xq = w8.quantize_act_fp8(x)
    assert torch.equal(y, w8.fp8_gemm(*xq, *wq))
    assert (y[0] == 0).all() and (y[5] == 0).all()
    want, err = ref.product(ref.values(*xq), ref.values(*wq))
    fits = want.abs() + err < 65000
    assert ((y.double() - want).abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -25 + 1.001 * err)[fits].all()


# scales read by 16 bytes, by 4 and one by one, in parts that start within a
# group of four
@pytest.mark.parametrize("M", [3, 100, 200, 1500])
@pytest.mark.parametrize("K", [8192, 10240, 2560, 8208, 1920, 4224])
def test_scales_at_every_address(w8, M, K):
    N = 96
    wq, sw = weights(w8, N + 3, K)
    x = w8.quantize_act_fp8(rows(M + 3, K))
    for i in range(4):
        a, b = (x[0][i:i + M], x[1][i:i + M]), (wq[i:i + N], sw[i:i + N])
        y = w8.fp8_gemm(*a, *b)
        assert torch.equal(y, w8.fp8_gemm(*(t.clone() for t in a), *(t.clone() for t in b)))
        ref.check_product(y, *ref.product(ref.values(*a), ref.values(*b)))


@pytest.mark.parametrize("M", [2, 100, 600])
def test_weights_past_32_bits(w8, M):
    """2.3 GB of codes: the last columns against those rows on their own."""
    N, K = 140016, 16384
    gen = torch.Generator("cuda").manual_seed(0)
    wq = torch.randint(0, 256, (N, K), dtype=torch.uint8, device="cuda", generator=gen)
    wq &= 0xBF             # below 2: no NaN
    wq = wq.view(torch.float8_e4m3fn)
    sw = torch.randint(100, 110, (N, K // 128), dtype=torch.uint8, device="cuda", generator=gen).view(torch.float8_e8m0fnu)
    x = w8.quantize_act_fp8(rows(M, K))
    y = w8.fp8_gemm(*x, wq, sw)
    for n in (0, 131056, N - 48):
        part = slice(n, n + 48)
        ref.check_product(y[:, part], *ref.product(ref.values(*x), ref.values(wq[part], sw[part])))


def test_norm_past_32_bits(w8):
    M, K = 140001, 16384
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.empty(M, K, dtype=torch.float16, device="cuda").normal_(generator=gen)
    w = rows(1, K)[0]
    q, s, h = w8.rms_norm_quantize(x, w, residual=x, codes="fp8")
    y = w8.rms_norm(x, w)
    for at in (0, 131071, M - 9):
        part = x[at:at + 9]
        want = w8.rms_norm_quantize(part, w, residual=part, codes="fp8")
        for a, b in zip((q, s, h), want):
            assert torch.equal(a[at:at + 9].view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(y[at:at + 9], w8.rms_norm(part, w))


@pytest.mark.parametrize("M", [1, 40, 300, 2500])
def test_wait_that_gives_up(w8, M):
    """A copy that never comes: the kernels return, the status says so, and the
    next call is right."""
    K, F = 2560, 1040
    wg, wu, wd = weights(w8, F, K, 2), weights(w8, F, K, 3), weights(w8, K, F, 4)
    x = rows(M, K)
    xq = w8.quantize_act_fp8(x)
    want = w8.fp8_feed_forward(x, *wg, *wu, *wd), w8.fp8_gemm(*xq, *wg), w8.fp8_gated_gemm(*xq, *wg, *wu)
    assert w8.w8a8_check_status() == 0
    calls = (lambda: w8.fp8_feed_forward(x, *wg, *wu, *wd), lambda: w8.fp8_gemm(*xq, *wg),
             lambda: w8.fp8_gated_gemm(*xq, *wg, *wu))
    for call, right in zip(calls, want):
        w8.w8a8_test_set_fault(2_000_000, True)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            w8.w8a8_test_set_fault(0, False)
        assert w8.w8a8_check_status() == 5
        assert torch.equal(call(), right)
        assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("M", [1, 7, 33, 130, 700])
def test_a_decoder_layers_projections(w8, M):
    """Norm to codes, projection, residual, norm to codes, gated block, residual:
    each step against the definition on what the step before gave."""
    K, F = 1040, 2064
    x, r = rows(M, K), rows(M, K, 7)
    n1, n2 = rows(1, K, 8)[0], rows(1, K, 9)[0]
    wo = weights(w8, K, K, 1)
    wg, wu, wd = weights(w8, F, K, 2), weights(w8, F, K, 3), weights(w8, K, F, 4)
    q, s, h = w8.rms_norm_quantize(x, n1, residual=r, codes="fp8")
    v, want_h = ref.norm(x, n1, r)
    assert torch.equal(h, want_h.half())
    ref.check_fp8(q, s, v, v.abs() * ref.NORM)
    o = w8.fp8_gemm(q, s, *wo)
    ref.check_product(o, *ref.product(ref.values(q, s), ref.values(*wo)))
    q2, s2, h2 = w8.rms_norm_quantize(o, n2, residual=h, codes="fp8", residual_out=h)
    assert h2 is h and torch.equal(h2, (o.double() + want_h).half())
    g, gs = w8.fp8_gated_gemm(q2, s2, *wg, *wu, codes=True)
    want, err = ref.gated(ref.values(q2, s2), ref.values(*wg), ref.values(*wu))
    ref.check_fp8(g, gs, want, err)
    y = w8.fp8_gemm(g, gs, *wd)
    ref.check_product(y, *ref.product(ref.values(g, gs), ref.values(*wd)))
    # the block called as one, on the norm's values
    z = w8.rms_norm(o, n2, residual=want_h.half())[0]
    whole = w8.fp8_feed_forward(z, *wg, *wu, *wd)
    parts = w8.fp8_gemm(*w8.fp8_gated_gemm(*w8.quantize_act_fp8(z), *wg, *wu, codes=True), *wd)
    assert torch.equal(whole, parts)


@pytest.mark.parametrize("group", [0, 64, 128])
def test_int8_codes_go_on_to_the_int8_products(w8, group):
    """The norm's INT8 codes are what w8a8_gemm and w8a8_gemm_h read."""
    M, K, N = 70, 1024, 200
    x, w = rows(M, K), rows(1, K, 3)[0]
    gen = torch.Generator("cuda").manual_seed(2)
    wq, sw = w8.quantize_weight_int8((0.02 * torch.randn(N, K, device="cuda", generator=gen)).half(), group)
    a, sa = w8.rms_norm_quantize(x, w, codes="int8", group_size=group)
    b, sb = w8.rms_norm_quantize(x, w, codes="half", group_size=group)
    assert torch.equal(a.half(), b) and torch.equal(sa, sb)
    y = w8.w8a8_gemm(a, sa, wq, sw, group)
    z = w8.w8a8_gemm_h(b, sb, wq, sw, group)
    size = group or K
    part = (a.double().view(M, -1, size) * sa.double().view(M, -1, 1)).flatten(1)
    back = (wq.double().view(N, -1, size) * sw.double().view(N, -1, 1)).flatten(1)
    want = part @ back.T
    # integer sums, then a scale product, a product (an addition) for each group, one rounding
    err = (K // size + 2) * 2.0 ** -23 * (part.abs() @ back.abs().T)
    for got in (y, z):
        assert ((got.double() - want).abs() <= want.abs() * 2.0 ** -11 + 2.0 ** -25 + 1.001 * err).all()


def test_two_graphs_share_a_workspace(w8):
    M, K, F = 40, 528, 1296
    wg, wu, wd = weights(w8, F, K, 2), weights(w8, F, K, 3), weights(w8, K, F, 4)
    ws = torch.empty(w8.fp8_feed_forward_workspace_bytes(M, K, F), dtype=torch.uint8, device="cuda")
    xs = [rows(m, K, m) for m in (M, 1)]
    want = [w8.fp8_feed_forward(x, *wg, *wu, *wd) for x in xs]
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w8.fp8_feed_forward(x, *wg, *wu, *wd, workspace=ws))
        graphs.append(g)
    for _ in range(3):
        for g, y, right in zip(graphs, outs, want):
            y.zero_()
            g.replay()
            assert torch.equal(y, right)

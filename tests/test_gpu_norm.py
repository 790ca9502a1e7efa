"""The root-mean-square norm, as values and as codes, and the 8-bit float quantizer."""
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


def rows(M, K, seed=0, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(M, K, device="cuda", generator=gen) * scale
    x *= 1 + 30 * (torch.rand(K, device="cuda", generator=gen) > 0.98)
    x *= 0.1 + 3 * torch.rand(M, 1, device="cuda", generator=gen)
    return x.half()


def weight(K, seed=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (1 + 0.5 * torch.randn(K, device="cuda", generator=gen)).half()


def framed(shape, dtype):
    """A tensor inside a larger one of a known pattern, and what tells whether that is intact."""
    n = torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()
    pad = -n % 256 + 256
    raw = torch.full((256 + n + pad,), 0xA5, dtype=torch.uint8, device="cuda")
    return raw[256:256 + n].view(dtype).view(shape), lambda: bool((raw[:256] == 0xA5).all() and (raw[256 + n:] == 0xA5).all())


# one vector, a warp, part of a warp, odd group counts, the ends of each count
# of vectors a thread (1024, 8192, 16384), the longest row
SIZES = [(1, 16), (3, 48), (5, 256), (2, 272), (7, 1024), (2, 1040), (301, 2560), (1, 4096), (9, 4112),
         (3, 8192), (2, 8208), (2, 14336), (3, 16400), (2, 32768), (2500, 128), (1, 12816)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_values(w8, M, K, residual):
    x, w = rows(M, K), weight(K)
    r = rows(M, K, 5, 4.0) if residual else None
    y, fine = framed((M, K), torch.float16)
    got = w8.rms_norm(x, w, residual=r, eps=1e-6, y=y)
    v, h = ref.norm(x, w, r, 1e-6)
    if residual:
        assert got[0] is y and torch.equal(got[1], h.half())
    ref.check_values(y, v, ref.NORM)
    assert fine()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,K", SIZES)
def test_codes(w8, M, K, residual):
    x, w = rows(M, K), weight(K)
    r = rows(M, K, 5, 4.0) if residual else None
    v, h = ref.norm(x, w, r, 1e-6)
    for group in (0, 64, 128):
        if group and K % group:
            continue
        got = {}
        for form, dtype in (("int8", torch.int8), ("half", torch.float16)):
            q, fine = framed((M, K), dtype)
            scale, fine_too = framed((M, K // group if group else 1), torch.float32)
            out = w8.rms_norm_quantize(x, w, residual=r, eps=1e-6, codes=form, group_size=group, q=q, scale=scale)
            assert fine() and fine_too() and (not residual or torch.equal(out[2], h.half()))
            ref.check_int8(q, scale, v, group, ref.NORM)
            got[form] = q, scale
        assert torch.equal(got["int8"][0].half(), got["half"][0]) and torch.equal(got["int8"][1], got["half"][1])
    q, fine = framed((M, K), torch.float8_e4m3fn)
    scale, fine_too = framed((M, -(-K // 128)), torch.float8_e8m0fnu)
    w8.rms_norm_quantize(x, w, residual=r, eps=1e-6, codes="fp8", q=q, scale=scale)
    ref.check_fp8(q, scale, v, 2 * ref.NORM * v.abs())
    assert fine() and fine_too()


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("name", ["quantize_act_fp8", "quantize_weight_fp8"])
def test_quantizer_is_exact(w8, name, M, K):
    x = rows(M, K)
    x[0, :8] = torch.tensor([65504.0, -65504, 6e-8, -6e-8, 0, 448, 1.0625, 17.0])
    if M > 1:
        x[1] = 0
    q, fine = framed((M, K), torch.float8_e4m3fn)
    scale, fine_too = framed((M, -(-K // 128)), torch.float8_e8m0fnu)
    getattr(w8, name)(x, q, scale)
    codes, s = ref.quantize(x.double())
    assert torch.equal(q.double(), codes) and torch.equal(scale.double(), s)
    assert fine() and fine_too()


def test_every_half(w8):
    """Every finite fp16 value beside each of several group maxima."""
    every = torch.arange(1 << 16, device="cuda").to(torch.int32).to(torch.uint16).view(torch.float16)
    every = every[every.isfinite()]
    for top in (65504.0, 448.0, 449.0, 1.0, 2.0 ** -14, 2.0 ** -24):
        part = every[every.abs() <= top]
        part = torch.nn.functional.pad(part, (0, -len(part) % 127)).view(-1, 127)
        x = torch.cat([torch.full_like(part[:, :1], top), part], 1)
        q, scale = w8.quantize_act_fp8(x)
        codes, s = ref.quantize(x.double())
        assert torch.equal(q.double(), codes) and torch.equal(scale.double(), s)


def test_zero_rows_and_extremes(w8):
    K = 640
    w = weight(K)
    x = torch.zeros(5, K, dtype=torch.float16, device="cuda")
    x[1] = 65504
    x[2] = 6e-8
    x[3, 5] = -65504
    for eps in (0.0, 1e-6):
        v, _ = ref.norm(x, w, None, eps)
        y = w8.rms_norm(x, w, eps=eps)
        ref.check_values(y, v, ref.NORM)
        assert (y[0] == 0).all() and (y[4] == 0).all()
        q, scale = w8.rms_norm_quantize(x, w, eps=eps, codes="int8")
        ref.check_int8(q, scale, v, 0, ref.NORM)
        assert scale[0].item() == 0 and (q[0] == 0).all()
        q, scale = w8.rms_norm_quantize(x, w, eps=eps, codes="fp8")
        ref.check_fp8(q, scale, v, 2 * ref.NORM * v.abs())
        assert (scale[0].float() == 1).all() and (q[0].float() == 0).all()
    # a weight of zeros
    q, scale = w8.rms_norm_quantize(x, torch.zeros_like(w), codes="int8", group_size=64)
    assert (q == 0).all() and (scale == 0).all()


def test_residual_in_place(w8):
    x, w, r = rows(33, 2560), weight(2560), rows(33, 2560, 7)
    want = w8.rms_norm(x, w, residual=r)
    keep = x.clone()
    y, h = w8.rms_norm(x, w, residual=r, residual_out=r)
    assert h is r and torch.equal(y, want[0]) and torch.equal(r, want[1]) and torch.equal(x, keep)
    r2 = rows(33, 2560, 7)
    y, h = w8.rms_norm(x, w, residual=r2, residual_out=x)
    assert h is x and torch.equal(y, want[0]) and torch.equal(x, want[1])


def test_rounding_of_the_residual(w8):
    """h is x + r rounded once to fp16, overflow included in neither direction."""
    x = torch.tensor([[2048.0, 1.0, 2049.0, 6e-8] * 4], device="cuda").half()
    r = torch.tensor([[1.0, 2.0 ** -11, 2.0 ** -24, 6e-8] * 4], device="cuda").half()
    _, h = w8.rms_norm(x, torch.ones(16, device="cuda").half(), residual=r)
    assert torch.equal(h, (x.double() + r.double()).half())


def test_refusals(w8):
    x, w = rows(4, 256), weight(256)
    for bad in (x[:, ::2], x[0], x.t()):
        with pytest.raises(ValueError):
            w8.rms_norm(bad, w)
    for kw in (dict(residual=x[:2]), dict(residual=x[:, :128]), dict(residual_out=x), dict(y=x[:2])):
        with pytest.raises(ValueError):
            w8.rms_norm(x, w, **kw)
    with pytest.raises(ValueError):
        w8.rms_norm(x, w[:128])
    with pytest.raises(ValueError):
        w8.rms_norm(x, w.cpu())
    with pytest.raises(TypeError):
        w8.rms_norm(x, w.float())
    with pytest.raises(TypeError):
        w8.rms_norm_quantize(x, w, q=torch.empty_like(x))
    with pytest.raises(w8.W8A8Error):
        w8.rms_norm(x, w, eps=-1.0)
    with pytest.raises(w8.W8A8Error):
        w8.rms_norm(x[:, :40].contiguous(), w[:40].contiguous())
    assert w8.rms_norm(x[:0], w).shape == (0, 256)


def test_streams_and_graph(w8):
    """On another stream, and captured: chains of the norm and its readers."""
    M, K, N = 65, 2560, 640
    x, r, w = rows(M, K), rows(M, K, 3), weight(K)
    wq, sw = w8.quantize_weight_int8(rows(N, K, 9, 0.02))
    q, s, h = w8.rms_norm_quantize(x, w, residual=r, codes="half")
    want = w8.w8a8_gemm_h(q, s, wq, sw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            a, b, c = w8.rms_norm_quantize(x, w, residual=r, codes="half")
            y = w8.w8a8_gemm_h(a, b, wq, sw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want) and torch.equal(c, h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b, c = w8.rms_norm_quantize(x, w, residual=r, codes="half")
        y = w8.w8a8_gemm_h(a, b, wq, sw)
    x2, r2 = rows(M, K, 20), rows(M, K, 21)
    x.copy_(x2)
    r.copy_(r2)
    graph.replay()
    q, s, h = w8.rms_norm_quantize(x2, w, residual=r2, codes="half")
    assert torch.equal(y, w8.w8a8_gemm_h(q, s, wq, sw)) and torch.equal(c, h)
    y0 = w8.linear(w8.rms_norm(x2, w), wq, sw)            # values into a layer that quantizes its own rows
    assert torch.equal(y0, w8.linear(w8.rms_norm(x2, w).clone(), wq, sw))

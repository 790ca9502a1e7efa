"""The 8-bit float products in the classes of large batches: a row's result is the
same in every batch of a class, whichever kernel its size takes, and right on both
sides of each class's border; outputs of more than 2^31 values."""
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


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# the smallest and the largest of a class, and two between
CLASSES = [(1025, 1300, 2000, 2560), (2561, 4000, 6000, 8192), (8193, 9001, 16390)]


# narrow outputs with K divided (64), undivided ones whose kernel changes within a
# class (1060), odd widths, and rows of scales at any address (1296, 4112)
@pytest.mark.parametrize("N,K", [(64, 8192), (64, 14336), (1060, 2048), (515, 1296), (2048, 272), (333, 4112)])
@pytest.mark.parametrize("sizes", CLASSES)
def test_rows_do_not_depend_on_the_batch(w8, sizes, N, K):
    wq = weights(w8, N, K)
    x = w8.quantize_act_fp8(rows(sizes[-1], K))
    whole = w8.fp8_gemm(*x, *wq)
    for m in sizes[:-1]:
        assert torch.equal(w8.fp8_gemm(x[0][:m], x[1][:m], *wq), whole[:m])
        end = [t[-m:].clone() for t in x]      # codes have to start at 16 bytes, scales anywhere
        assert torch.equal(w8.fp8_gemm(*end, *wq), whole[-m:])


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("F,K", [(64, 8192), (528, 2048), (1040, 656)])
@pytest.mark.parametrize("sizes", CLASSES)
def test_gated_rows_do_not_depend_on_the_batch(w8, sizes, F, K, codes):
    wg, wu = weights(w8, F, K, 2), weights(w8, F, K, 3)
    x = w8.quantize_act_fp8(rows(sizes[-1], K))
    whole = w8.fp8_gated_gemm(*x, *wg, *wu, codes=codes)
    for m in sizes[:-1]:
        part = w8.fp8_gated_gemm(x[0][:m], x[1][:m], *wg, *wu, codes=codes)
        if codes:
            assert same(part[0], whole[0][:m]) and same(part[1], whole[1][:m])
        else:
            assert torch.equal(part, whole[:m])


@pytest.mark.parametrize("M", [2560, 2561, 8192, 8193, 9001])
@pytest.mark.parametrize("N,K", [(77, 8192), (1061, 2048), (259, 144), (520, 656)])
def test_product_beside_a_border(w8, M, N, K):
    x, wq = rows(M, K), weights(w8, N, K)
    xq = w8.quantize_act_fp8(x)
    y = w8.fp8_gemm(*xq, *wq)
    ref.check_product(y, *ref.product(ref.values(*xq), ref.values(*wq)))
    assert torch.equal(w8.fp8_linear(x, *wq), y)


@pytest.mark.parametrize("gelu", [False, True])
@pytest.mark.parametrize("M", [2560, 2561, 8192, 8193])
@pytest.mark.parametrize("F,K", [(144, 2048), (1040, 272)])
def test_gated_beside_a_border(w8, M, F, K, gelu):
    x = w8.quantize_act_fp8(rows(M, K))
    wg, wu = weights(w8, F, K, 2), weights(w8, F, K, 3)
    h, err = ref.gated(ref.values(*x), ref.values(*wg), ref.values(*wu), gelu)
    kind = "gelu" if gelu else "silu"
    ref.check_product(w8.fp8_gated_gemm(*x, *wg, *wu, activation=kind), h, err)
    ref.check_fp8(*w8.fp8_gated_gemm(*x, *wg, *wu, activation=kind, codes=True), h, err)


# y's last element is past 2^31: few rows of very many columns, many rows, and rows
# that do not start at 16 bytes
@pytest.mark.parametrize("M,N,K", [(120, 17_900_005, 16), (9000, 240_000, 144), (9001, 239_001, 144), (1_200_003, 2000, 128)])
def test_outputs_past_32_bits(w8, M, N, K):
    assert M * N > 2 ** 31
    x, wq = w8.quantize_act_fp8(rows(M, K)), w8.quantize_weight_fp8(rows(N, K, 1))
    y = w8.fp8_gemm(*x, *wq)
    for m in (0, M // 2, M - min(M, 40)):
        for n in (0, N // 2, N - 48):
            a, b = (t[m:m + 40] for t in x), (t[n:n + 48] for t in wq)
            ref.check_product(y[m:m + 40, n:n + 48], *ref.product(ref.values(*a), ref.values(*b)))


def test_codes_past_32_bits(w8):
    M, F, K = 66_001, 32768, 128
    assert M * F > 2 ** 31
    x = w8.quantize_act_fp8(rows(M, K))
    wg, wu = weights(w8, F, K, 2), weights(w8, F, K, 3)
    q, s = w8.fp8_gated_gemm(*x, *wg, *wu, codes=True)
    for m in (0, 65_536, M - 40):
        a = ref.values(*(t[m:m + 40] for t in x))
        ref.check_fp8(q[m:m + 40], s[m:m + 40], *ref.gated(a, ref.values(*wg), ref.values(*wu)))

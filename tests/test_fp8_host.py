"""Refusals of the norm and of the 8-bit float layers, checked on the host (no
GPU needed), and the plain reference that the GPU tests compare with."""
import ctypes

import pytest

import fp8_reference as ref
from w4a8_int8_quantized_gb300 import binding, build

P = ctypes.c_void_p
A, B, C, D, E, F, G = (P(i << 20) for i in range(1, 8))   # aligned, never dereferenced
ODD8 = P((9 << 20) + 8)
ODD2 = P((9 << 20) + 2)
NUL = P(0)
S0 = P(0)
OK, INV, MIS, UNSUP, WS = 0, 1, 2, 3, 6
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def norm(lib, x=A, r=B, w=C, M=4, K=64, eps=1e-5, h=D, y=E):
    return lib.rms_norm(x, r, w, M, K, eps, h, y, S0)


def quant(lib, x=A, r=B, w=C, M=4, K=256, eps=1e-5, form=0, gs=0, h=D, q=E, scale=F):
    return lib.rms_norm_quantize(x, r, w, M, K, eps, form, gs, h, q, scale, S0)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INV), (dict(K=0), INV), (dict(K=-16), INV), (dict(K=40), MIS), (dict(K=32784), INV),
    (dict(eps=-1e-6), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(x=NUL), INV), (dict(w=NUL), INV), (dict(x=ODD8), MIS), (dict(w=ODD8), MIS),
    (dict(r=NUL), INV), (dict(h=NUL), INV), (dict(r=ODD8), MIS), (dict(h=ODD8), MIS)])
def test_norm_arguments(lib, kw, want):
    assert norm(lib, **kw) == want
    assert quant(lib, **kw) == want


def test_norm_outputs(lib):
    assert norm(lib, y=NUL) == INV and norm(lib, y=ODD8) == MIS
    assert norm(lib, M=0, x=NUL, w=NUL, r=NUL, h=NUL, y=NUL) == OK
    assert quant(lib, q=NUL) == INV and quant(lib, q=ODD8) == MIS
    assert quant(lib, scale=NUL) == INV and quant(lib, scale=ODD2) == MIS
    assert quant(lib, form=3) == INV and quant(lib, form=-1) == INV
    assert quant(lib, gs=32) == INV and quant(lib, K=192, gs=128) == INV
    assert quant(lib, form=2, gs=0) == INV and quant(lib, form=2, gs=64) == INV
    assert quant(lib, M=0, x=NUL, w=NUL, r=NUL, h=NUL, q=NUL, scale=NUL) == OK


@pytest.mark.parametrize("name", ["quantize_act_fp8", "quantize_weight_fp8"])
def test_quantizer_arguments(lib, name):
    q = getattr(lib, name)
    assert q(A, -1, 64, B, C, S0) == INV
    assert q(A, 4, 0, B, C, S0) == INV
    assert q(A, 4, 72, B, C, S0) == MIS
    assert q(A, 4, 40000, B, C, S0) == INV
    assert q(NUL, 4, 64, B, C, S0) == INV
    assert q(A, 4, 64, NUL, C, S0) == INV
    assert q(A, 4, 64, B, NUL, S0) == INV
    assert q(ODD8, 4, 64, B, C, S0) == MIS
    assert q(A, 4, 64, ODD8, C, S0) == MIS
    assert q(NUL, 0, 64, NUL, NUL, S0) == OK


def test_product_arguments(lib):
    g = lib.fp8_gemm
    assert g(A, B, C, D, -1, 8, 64, E, S0) == INV
    assert g(A, B, C, D, 8, -1, 64, E, S0) == INV
    assert g(A, B, C, D, 8, 8, 0, E, S0) == INV
    assert g(A, B, C, D, 8, 8, 56, E, S0) == MIS
    assert g(A, B, C, D, 8, 8, 32784, E, S0) == INV
    for i in range(4):
        args = [A, B, C, D]
        args[i] = NUL
        assert g(*args, 8, 8, 64, E, S0) == INV
    assert g(A, B, C, D, 8, 8, 64, NUL, S0) == INV
    assert g(ODD8, B, C, D, 8, 8, 64, E, S0) == MIS
    assert g(A, B, ODD8, D, 8, 8, 64, E, S0) == MIS
    assert g(A, B, C, D, 8, 8, 64, ODD8, S0) == MIS
    assert g(NUL, NUL, NUL, NUL, 0, 8, 64, NUL, S0) == OK
    assert g(NUL, NUL, NUL, NUL, 8, 0, 64, NUL, S0) == OK


def gate(lib, ptrs=(A, B, C, D, E, F), M=8, n=64, K=64, kind=0, h=NUL, hq=G, sh=P(8 << 20)):
    return lib.fp8_gated_gemm(*ptrs, M, n, K, kind, h, hq, sh, S0)


def test_gated_arguments(lib):
    assert gate(lib, M=-1) == INV and gate(lib, n=-16) == INV and gate(lib, K=0) == INV
    assert gate(lib, K=56) == MIS
    assert gate(lib, kind=2) == INV and gate(lib, kind=-1) == INV
    assert gate(lib, n=72) == MIS and gate(lib, n=40000) == INV      # codes: a row of a product
    assert gate(lib, h=G) == INV                                     # two forms of output
    assert gate(lib, h=G, hq=NUL) == INV
    assert gate(lib, hq=NUL, sh=NUL) == INV                          # none
    assert gate(lib, sh=NUL) == INV and gate(lib, hq=ODD8) == MIS
    assert gate(lib, h=ODD8, hq=NUL, sh=NUL) == MIS
    for i in range(6):
        ptrs = [A, B, C, D, E, F]
        ptrs[i] = NUL
        assert gate(lib, ptrs) == INV
    for i in (0, 2, 4):
        ptrs = [A, B, C, D, E, F]
        ptrs[i] = ODD8
        assert gate(lib, ptrs) == MIS
    assert gate(lib, [NUL] * 6, M=0, hq=NUL, sh=NUL) == OK
    assert gate(lib, [NUL] * 6, n=0, hq=NUL, sh=NUL) == OK


def test_layer_arguments(lib):
    f = lib.fp8_linear_workspace_bytes
    assert f(3, 272) == 1024 + 256 and f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 72) == 0
    assert f(1 << 20, 32768) == (1 << 35) + (1 << 28)
    ln = lib.fp8_linear
    need = f(8, 64)
    assert ln(A, B, C, -1, 8, 64, D, need, E, S0) == INV
    assert ln(A, B, C, 8, 8, 56, D, need, E, S0) == MIS
    assert ln(NUL, B, C, 8, 8, 64, D, need, E, S0) == INV
    assert ln(A, ODD8, C, 8, 8, 64, D, need, E, S0) == MIS
    assert ln(A, B, NUL, 8, 8, 64, D, need, E, S0) == INV
    assert ln(A, B, C, 8, 8, 64, NUL, need, E, S0) == WS
    assert ln(A, B, C, 8, 8, 64, P((1 << 20) + 16), need, E, S0) == WS
    assert ln(A, B, C, 8, 8, 64, D, need - 1, E, S0) == WS
    assert ln(NUL, NUL, NUL, 0, 8, 64, NUL, 0, NUL, S0) == OK
    w = lib.fp8_feed_forward_workspace_bytes
    assert w(3, 272, 144) == f(3, 272) + f(3, 144)
    assert w(3, 272, 100) == 0 and w(3, 100, 144) == 0 and w(-1, 64, 64) == 0

    def ff(x=A, wg=B, sg=C, wu=D, su=E, wd=F, sd=G, M=8, K=64, n=128, N=32, kind=0, ws=A,
           size=w(8, 64, 128), y=B):
        return lib.fp8_feed_forward(x, wg, sg, wu, su, wd, sd, M, K, n, N, kind, ws, size, y, S0)

    assert ff(M=-1) == INV and ff(N=-1) == INV and ff(K=0) == INV and ff(n=0) == INV
    assert ff(K=72) == MIS and ff(n=72) == MIS and ff(kind=5) == INV
    for name in ("x", "wg", "sg", "wu", "su", "wd", "sd", "y"):
        assert ff(**{name: NUL}) == INV
    for name in ("x", "wg", "wu", "wd", "y"):
        assert ff(**{name: ODD8}) == MIS
    assert ff(ws=NUL) == WS and ff(size=w(8, 64, 128) - 1) == WS
    assert ff(M=0, x=NUL, y=NUL, ws=NUL) == OK and ff(N=0, wd=NUL, ws=NUL) == OK


def test_no_launch_without_the_gpu(lib):
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert norm(lib) == UNSUP and quant(lib) == UNSUP
    assert quant(lib, form=2, gs=128) == UNSUP
    assert lib.quantize_act_fp8(A, 4, 64, B, C, S0) == UNSUP
    assert lib.fp8_gemm(A, B, C, D, 8, 8, 64, E, S0) == UNSUP
    assert gate(lib) == UNSUP and gate(lib, h=G, hq=NUL, sh=NUL, n=7) == UNSUP
    assert lib.fp8_linear(A, B, C, 8, 8, 64, D, 1 << 20, E, S0) == UNSUP


def test_binding_refusals():
    half = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.rms_norm(half, half[0])                    # CPU tensors
    with pytest.raises(TypeError):
        binding.rms_norm(half.float(), half[0])
    with pytest.raises(ValueError):
        binding.rms_norm_quantize(half, half[0], codes="int4")
    with pytest.raises(ValueError):
        binding.rms_norm_quantize(half, half[0], codes="fp8", group_size=64)
    with pytest.raises(ValueError):
        binding.rms_norm_quantize(half, half[0], codes="half", group_size=32)
    with pytest.raises(TypeError):
        binding.quantize_act_fp8(half.float())
    with pytest.raises(TypeError):
        binding.fp8_gemm(half, half, half, half)
    codes, scale = half.to(torch.float8_e4m3fn), torch.full((4, 1), 127, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(ValueError):
        binding.fp8_gemm(codes, scale, codes, scale)       # CPU tensors
    with pytest.raises(ValueError):
        binding.fp8_gated_gemm(codes, scale, codes, scale, codes, scale, activation="relu")
    with pytest.raises(ValueError):
        binding.fp8_feed_forward(half, codes, scale, codes, scale, codes, scale, activation="relu")


def test_reference_rule():
    """The reference against torch's own type and values whose codes are known."""
    x = torch.cat([torch.linspace(-448, 448, 4001), torch.logspace(-12, 9, 999, base=2)]).double().clamp(max=448)
    assert (ref.e4m3(x) == x.float().to(torch.float8_e4m3fn).double()).all()
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    every = every[every.isfinite()]
    assert (ref.e4m3(every) == every).all()
    top = torch.tensor([448.0, 448.0001, 449.0, 447.9, 224.0, 224.5, 1.0, 0.0, 2.0 ** -140, 65504.0])
    assert ref.scale_of(top.double()).tolist() == [1, 2, 2, 1, 0.5, 1, 2.0 ** -8, 1, 2.0 ** -126, 256]
    codes, scale = ref.quantize(torch.tensor([[448.0, 1.0, -3.3] + [0.0] * 125 + [7.0]], dtype=torch.float64))
    assert scale.tolist() == [[1, 2.0 ** -6]] and codes[0, [0, 1, 2, 128]].tolist() == [448, 1, -3.25, 448]


def test_reference_norm():
    x = torch.tensor([[3.0, 4.0] * 8, [0.0] * 16])
    w = torch.full((16,), 2.0)
    v, h = ref.norm(x, w, eps=0.0)
    assert torch.allclose(v[0], 2 * x[0].double() / 12.5 ** 0.5) and (v[1] == 0).all()
    assert (ref.norm(x, w, -x, eps=0.0)[0] == 0).all()
    assert torch.allclose(ref.act(torch.tensor([-1.0, 0.0, 2.0]).double(), False),
                          torch.nn.functional.silu(torch.tensor([-1.0, 0.0, 2.0]).double()))
    assert torch.allclose(ref.act(torch.tensor([-1.0, 0.0, 2.0]).double(), True),
                          torch.nn.functional.gelu(torch.tensor([-1.0, 0.0, 2.0]).double(), approximate="tanh"))

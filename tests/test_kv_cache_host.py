"""Refusals of the key/value cache calls, checked on the host (no GPU needed),
and the plain reference that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import kv_reference as ref
from w4a8_int8_quantized_gb300 import binding, build

P = ctypes.c_void_p
A, B, C, D = (P(i << 20) for i in (1, 2, 3, 4))   # aligned, never dereferenced
ODD8 = P((5 << 20) + 8)
NUL = P(0)
OK, INV, MIS, UNSUP, WS = 0, 1, 2, 3, 6


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def cache(**kw):
    f = dict(k_codes=1 << 20, v_codes=2 << 20, k_scale=3 << 20, v_scale=4 << 20, num_pages=10,
             kv_heads=4, page_size=16, head_dim=128, bits=4)
    f.update(kw)
    return ctypes.byref(binding._CacheStruct(**f))


BAD_CACHES = [(dict(bits=5), INV), (dict(head_dim=96), INV), (dict(kv_heads=0), INV),
              (dict(page_size=8), INV), (dict(page_size=48), INV), (dict(page_size=2048), INV),
              (dict(num_pages=-1), INV), (dict(num_pages=1 << 31), INV), (dict(k_codes=0), INV),
              (dict(v_scale=0), INV), (dict(k_codes=(1 << 20) + 8), MIS),
              (dict(v_scale=(4 << 20) + 4), MIS)]


def attend(lib, c, q=A, ts=2048, hs=128, T=8, heads=8, off=B, nb=2, max_q=8, table=C, width=4,
           lens=D, scale=0.1, causal=1, window=0, ws=A, wsb=1 << 40, out=B, lse=NUL):
    return lib.kv_cache_attention(q, ts, hs, T, heads, off, nb, max_q, table, width, lens, c, scale,
                                  causal, window, ws, wsb, out, lse, P(0))


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches(lib, kw, want):
    c = cache(**kw)
    assert lib.kv_cache_write(A, 512, 128, B, 512, 128, C, 4, c, P(0)) == want
    assert lib.kv_cache_read(C, 4, c, A, B, P(0)) == want
    assert attend(lib, c) == want


def test_write_and_read_arguments(lib):
    c = cache()
    w = lib.kv_cache_write
    assert w(A, 512, 128, B, 512, 128, C, 4, None, P(0)) == INV
    assert w(A, 512, 128, B, 512, 128, C, -1, c, P(0)) == INV
    assert w(NUL, 512, 128, B, 512, 128, C, 4, c, P(0)) == INV
    assert w(A, 512, 128, B, 512, 128, NUL, 4, c, P(0)) == INV
    assert w(A, -512, 128, B, 512, 128, C, 4, c, P(0)) == INV
    assert w(A, 516, 128, B, 512, 128, C, 4, c, P(0)) == MIS
    assert w(A, 512, 128, B, 512, 132, C, 4, c, P(0)) == MIS
    assert w(ODD8, 512, 128, B, 512, 128, C, 4, c, P(0)) == MIS
    assert w(A, 512, 128, B, 512, 128, P((3 << 20) + 4), 4, c, P(0)) == MIS
    assert w(NUL, 512, 128, NUL, 512, 128, NUL, 0, c, P(0)) == OK      # nothing to do
    r = lib.kv_cache_read
    assert r(C, -1, c, A, B, P(0)) == INV
    assert r(NUL, 4, c, A, B, P(0)) == INV
    assert r(C, 4, c, NUL, B, P(0)) == INV
    assert r(C, 4, c, A, ODD8, P(0)) == MIS
    assert r(NUL, 0, c, NUL, NUL, P(0)) == OK


def test_attention_arguments(lib):
    c = cache()
    assert attend(lib, c, T=-1) == INV
    assert attend(lib, c, nb=-1) == INV
    assert attend(lib, c, heads=0) == INV
    assert attend(lib, c, heads=6) == INV                  # not a multiple of kv_heads
    assert attend(lib, c, max_q=0) == INV
    assert attend(lib, c, width=-1) == INV
    assert attend(lib, c, width=1 << 28) == INV            # more tokens than an int32 length
    assert attend(lib, c, window=-1) == INV
    assert attend(lib, c, causal=0, window=4) == INV
    assert attend(lib, c, causal=2) == INV
    assert attend(lib, c, scale=float("nan")) == INV
    assert attend(lib, c, scale=float("inf")) == INV
    assert attend(lib, c, off=NUL) == INV                  # one query a sequence, but T != B
    assert attend(lib, c, q=NUL) == INV
    assert attend(lib, c, out=NUL) == INV
    assert attend(lib, c, lens=NUL) == INV
    assert attend(lib, c, table=NUL) == INV
    assert attend(lib, c, q=ODD8) == MIS
    assert attend(lib, c, ts=2052) == MIS
    assert attend(lib, c, out=ODD8) == MIS
    assert attend(lib, c, lens=P((4 << 20) + 2)) == MIS
    assert attend(lib, c, T=0, q=NUL, out=NUL) == OK
    need = lib.kv_cache_attention_workspace_bytes(8, 8, 2, 8, 4, c)
    if need:
        assert attend(lib, c, ws=NUL) == WS
        assert attend(lib, c, ws=P((1 << 20) + 16)) == WS
        assert attend(lib, c, wsb=need - 1) == WS
    assert lib.kv_cache_attention_workspace_bytes(8, 6, 2, 8, 4, c) == 0
    assert lib.kv_cache_attention_workspace_bytes(8, 8, 2, 8, 4, cache(bits=3)) == 0


def test_no_launch_without_the_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    assert lib.kv_cache_write(A, 512, 128, B, 512, 128, C, 4, cache(), P(0)) == UNSUP
    assert lib.kv_cache_read(C, 4, cache(), A, B, P(0)) == UNSUP
    assert attend(lib, cache()) == UNSUP
    assert lib.w8a8_status_string(7) not in (b"ok", b"unknown status")


def test_handle_refusals():
    import torch
    codes, scale = torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16)
    with pytest.raises(ValueError):
        binding.KVCache(codes, codes, scale, scale)        # CPU tensors
    with pytest.raises(TypeError):
        binding.KVCache(codes.float(), codes, scale, scale)
    with pytest.raises(TypeError):
        binding.KVCache(None, codes, scale, scale)
    with pytest.raises(ValueError):
        binding.KVCache(codes[0], codes[0], scale, scale)
    with pytest.raises(ValueError):
        binding.KVCache.empty(4, 2, 16, 64, bits=3, device="cpu")


@pytest.mark.parametrize("bits", [4, 8])
def test_reference_rule(bits):
    """The reference against the definition on values whose codes are known."""
    qmax = 2 ** (bits - 1) - 1
    x = np.zeros((3, 64), np.float16)
    x[0, :4] = [qmax, -qmax, 1, 0.5]        # scale 1, the tie goes to even
    x[2, 5] = np.inf
    x[2, 6] = np.nan
    q, s = ref.quantize(x, bits)
    assert s.tolist() == [1.0, 0.0, float(np.float32(65504.0 / qmax))]
    assert q[0, :4].tolist() == [qmax, -qmax, 1, 0] and not q[1].any()
    assert q[2, 5] == qmax and q[2, 6] == 0
    assert (ref.unpack(ref.pack(q, bits), bits) == q).all()


def test_reference_attention():
    """Two equal keys average their values; a query before every key sees nothing."""
    kc = np.ones((2, 1, 64), np.int64)
    vc = np.stack([np.full((1, 64), 2), np.full((1, 64), 4)])
    s = np.ones((2, 1))
    out, lse, _, _ = ref.attend(np.ones((3, 1, 64), np.float16), kc, s, vc, s, 1 / 64)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf      # position -1
    assert np.allclose(out[1], 2) and np.allclose(lse[1], 1)
    assert np.allclose(out[2], 3) and np.allclose(lse[2], 1 + np.log(2))

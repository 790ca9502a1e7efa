"""The quantized cache's attention where it is easy to get wrong: items that end
inside a warp, waits that give up, weights far apart, rows that nobody owns.
References and tolerances are those of kv_reference."""
import numpy as np
import pytest

import kv_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_kv_cache import Cache, attend, check, cuda, rows  # noqa: E402

if torch.cuda.is_available():
    import w4a8_int8_quantized_gb300 as w8


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64)])
@pytest.mark.parametrize("new", [[33, 65, 95], [127, 129, 1], [161, 255, 257]])
@pytest.mark.parametrize("behind", [0, 2500])
def test_rows_that_do_not_fill_a_warp(bits, D, new, behind):
    """Lanes without a row leave the warp's stores early and have to be back for its
    next tensor-memory load; whole items, and items cut between blocks."""
    rng = np.random.default_rng(bits + D + sum(new) + behind)
    c = Cache(rng, [n + behind for n in new], 1, D, 64, bits)
    q = rows(rng, sum(new), 1, D)
    check(c, q, new, *attend(c, q, new, max_q=max(new)))
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("lens,new,group", [([3000], [1], 4), ([300, 40], [4, 2], 4), ([90] * 1200, [1] * 1200, 1),
                                            ([900, 300], [200, 40], 4)])
def test_wait_that_gives_up(lens, new, group):
    """A copy (few rows) or a hand-over (many rows) left out with the waits cut to about
    1 ms: the kernel returns, the status says so, and the next call is right."""
    rng = np.random.default_rng(len(lens))
    c = Cache(rng, lens, 1, 128, 16, 4)
    q = rows(rng, sum(new), group, 128)
    call = lambda: attend(c, q, new, max_q=max(new))  # noqa: E731
    assert w8.w8a8_check_status() == 0
    try:
        w8.w8a8_test_set_fault(2_000_000, True)
        call()
        status = w8.w8a8_check_status()
    finally:
        w8.w8a8_test_set_fault(0, False)
    assert status == 5, w8.w8a8_status_string(status)
    assert w8.w8a8_check_status() == 0
    check(c, q, new, *call())
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("size", [1.0, 0.05, 0.001])
@pytest.mark.parametrize("at", [0, 200, 451])
def test_leading_key_without_a_value(bits, new, size, at):
    """A key far above the others whose value is zero (scale 0): the tokens that make up
    the output keep their weights' bits."""
    rng = np.random.default_rng(bits + new + at)
    c = Cache(rng, [512], 1, 128, 16, bits)
    q = rows(rng, new, 4, 128)
    q[..., 0] = 4
    c.k[0][..., 0] = 0
    c.k[0][at] = 0
    c.k[0][at, :, 0] = 28                                    # about 10 nats above the rest
    c.v[0] = (c.v[0] * size).astype(np.float16)
    c.v[0][at] = 0
    w8.kv_cache_write(cuda(c.k[0]), cuda(c.v[0]), cuda(c.slots(0, np.arange(512))), c.handle)
    check(c, q, [new], *attend(c, q, [new], max_q=new))


def test_timeout_is_reported_before_an_index():
    """An index out of range does not hide a wait that gave up after it."""
    cache = w8.KVCache.empty(2, 1, 16, 64)
    x = torch.ones(1, 1, 64, dtype=torch.float16, device="cuda")
    a = torch.ones(130, 512, dtype=torch.int8, device="cuda")
    w = torch.ones(257, 512, dtype=torch.int8, device="cuda")
    assert w8.w8a8_check_status() == 0
    w8.kv_cache_write(x, x, torch.tensor([99], device="cuda"), cache)
    try:
        w8.w8a8_test_set_fault(2_000_000, True)
        w8.w8a8_gemm_i32(a, w)
        status = w8.w8a8_check_status()
    finally:
        w8.w8a8_test_set_fault(0, False)
    assert status == 5, w8.w8a8_status_string(status)
    assert w8.w8a8_check_status() == 0
    w8.kv_cache_write(x, x, torch.tensor([99], device="cuda"), cache)
    assert w8.w8a8_check_status() == 7
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64)])
@pytest.mark.parametrize("new", [1, 5, 30, 100])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 1e-40, -1.0])
def test_slots_before_the_window_may_hold_anything(bits, D, new, scale):
    """Also those that share a page and a group of 16 with the window's first key."""
    rng = np.random.default_rng(bits + new)
    n, window = 999, 300
    c = Cache(rng, [n], 2, D, 64, bits)
    q = rows(rng, new, 8, D)
    first = n - new + 1 - window
    assert first % 16
    slots = c.slots(0, np.arange(first))
    c.handle.k_scale[slots // 64, :, slots % 64] = scale
    c.handle.v_scale[slots // 64, :, slots % 64] = scale
    check(c, q, [new], *attend(c, q, [new], max_q=new, window=window), window=window)
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("new", [[1, 0, 3], [70, 0, 90], [2, 8, 1]])
@pytest.mark.parametrize("before,after", [(0, 5), (4, 0), (3, 700)])
def test_rows_that_no_sequence_owns(new, before, after):
    """Padding before the first and after the last sequence: out 0, lse -inf, no report."""
    rng = np.random.default_rng(sum(new) + before + after)
    c = Cache(rng, [90, 20, 333], 2, 128, 16, 4)
    q = rows(rng, before + sum(new) + after, 8, 128)
    off = cuda((before + np.concatenate([[0], np.cumsum(new)])).astype(np.int32))
    out = torch.full(q.shape, 7, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], 7, dtype=torch.float32, device="cuda")
    w8.kv_cache_attention(cuda(q), c.handle, cuda(c.table), cuda(np.array(c.lens, np.int32)), q_offsets=off,
                          max_q=max(new), return_lse=True, out=out, lse=lse)
    assert w8.w8a8_check_status() == 0
    end = before + sum(new)
    check(c, q[before:end], new, out[before:end], lse[before:end])
    for rest in (slice(0, before), slice(end, None)):
        assert not out[rest].any() and (lse[rest] == -np.inf).all()


@pytest.mark.parametrize("max_q", [3, 40])
def test_queries_beyond_max_q(max_q):
    """Reported, and their rows hold 0 and -inf; the other sequences are right."""
    rng = np.random.default_rng(max_q)
    new = [max_q - 1, max_q + 7, max_q]
    c = Cache(rng, [100, 200, 60], 2, 128, 16, 8)
    q = rows(rng, sum(new), 8, 128)
    out = torch.full(q.shape, 7, dtype=torch.float16, device="cuda")
    lse = torch.full(q.shape[:2], 7, dtype=torch.float32, device="cuda")
    attend(c, q, new, max_q=max_q, out=out, lse=lse)
    assert w8.w8a8_check_status() == 7
    over = slice(new[0] + max_q, new[0] + new[1])
    assert not out[over].any() and (lse[over] == -np.inf).all()
    for b, r in ((0, slice(0, new[0])), (2, slice(new[0] + new[1], None))):
        one = Cache.__new__(Cache)
        one.__dict__.update(c.__dict__, lens=[c.lens[b]], k=[c.k[b]], v=[c.v[b]])
        check(one, q[r], [new[b]], out[r], lse[r])


@pytest.mark.parametrize("T", [1, 700])
def test_no_sequences(T):
    """Query rows and no sequence: every row is padding."""
    c = w8.KVCache.empty(4, 2, 16, 64)
    out = torch.full((T, 4, 64), 7, dtype=torch.float16, device="cuda")
    lse = torch.full((T, 4), 7, dtype=torch.float32, device="cuda")
    w8.kv_cache_attention(torch.ones_like(out), c, torch.zeros(0, 3, dtype=torch.int32, device="cuda"),
                          torch.zeros(0, dtype=torch.int32, device="cuda"),
                          q_offsets=torch.zeros(1, dtype=torch.int32, device="cuda"), return_lse=True, out=out, lse=lse)
    assert not out.any() and (lse == -np.inf).all()
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("new", [[45, 1], [300, 20]])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
def test_window_without_bound_and_queries_before_every_key(new, window):
    """The largest window with more queries than tokens: positions far below zero."""
    rng = np.random.default_rng(sum(new))
    c = Cache(rng, [37, 40], 2, 128, 16, 4)
    q = rows(rng, sum(new), 8, 128)
    check(c, q, new, *attend(c, q, new, max_q=max(new), window=window), window=window)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,n", [(1, 40), (2, 5000), (60, 60), (60, 5000)])
def test_outputs_at_the_largest_half(bits, new, n):
    """Values of +-65504 (infinite ones are stored so) average to themselves, not to infinity."""
    rng = np.random.default_rng(bits + new + n)
    c = Cache(rng, [n], 2, 128, 16, bits)
    q = rows(rng, new, 8, 128)
    c.v[0][..., 5], c.v[0][..., 70] = np.inf, -65504
    w8.kv_cache_write(cuda(c.k[0]), cuda(c.v[0]), cuda(c.slots(0, np.arange(n))), c.handle)
    out, lse = attend(c, q, [new], max_q=new)
    assert torch.isfinite(out).all()
    check(c, q, [new], out, lse)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_far_from_zero(new, sign):
    """A score of 1e33 in either direction, the only one of its row: its value."""
    rng = np.random.default_rng(new)
    c = Cache(rng, [new], 2, 128, 16, 8)
    q = rows(rng, new, 2, 128)
    out, lse = attend(c, q, [new], max_q=new, softmax_scale=sign * 1e32, window=1)
    _, _, vc, vs = c.quantized(0)
    want = vc * vs[..., None]
    np.testing.assert_allclose(out.double().cpu().numpy(), want, rtol=2.0 ** -10, atol=2.0 ** -24)
    assert torch.isfinite(lse).all()


def test_more_sequences_times_heads_than_32_bits_hold():
    B, heads = 1 << 21, 1024
    cache = w8.KVCache.empty(1, heads, 16, 64)
    x = torch.randn(16, heads, 64, device="cuda").half()
    w8.kv_cache_write(x, x, torch.arange(16, device="cuda"), cache)
    new = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new[[5, B // 2, B - 1]] = 1
    lens[[5, B // 2, B - 1]] = torch.tensor([3, 16, 7], dtype=torch.int32, device="cuda")
    off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    off[1:] = new.cumsum(0).int()
    q = torch.randn(3, heads, 64, device="cuda").half()
    out = w8.kv_cache_attention(q, cache, torch.zeros(B, 1, dtype=torch.int32, device="cuda"), lens, q_offsets=off, max_q=1)
    want = w8.kv_cache_attention(q, cache, torch.zeros(3, 1, dtype=torch.int32, device="cuda"),
                                 torch.tensor([3, 16, 7], dtype=torch.int32, device="cuda"))
    assert torch.equal(out, want)
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_every_magnitude(bits):
    """Every finite fp16 value as a row's largest: its scale and the codes of the row, half of
    them within a few units in the last place of a tie."""
    rng = np.random.default_rng(bits)
    most = np.arange(0, 0x7c00, dtype=np.uint16).view(np.float16)
    T, qmax, page = len(most), 2 ** (bits - 1) - 1, 1024
    x = rng.uniform(-1, 1, (T, 1, 64)) * most[:, None, None].astype(np.float64)
    ties = (rng.integers(-qmax, qmax, (T, 1, 32)) + 0.5) / qmax * most[:, None, None].astype(np.float64)
    x[..., :32] = ties
    x = x.astype(np.float16)
    x[..., 40] = most[:, None]
    cache = w8.KVCache.empty(-(-T // page), 1, page, 64, bits)
    slots = np.arange(T)
    w8.kv_cache_write(cuda(x), cuda(-x), cuda(slots), cache)
    q, s = ref.quantize(x, bits)
    for codes, scale, sign in ((cache.k_codes, cache.k_scale, 1), (cache.v_codes, cache.v_scale, -1)):
        np.testing.assert_array_equal(scale.cpu().numpy()[slots // page, :, slots % page], s.astype(np.float32))
        np.testing.assert_array_equal(codes.cpu().numpy()[slots // page, :, slots % page], ref.pack(sign * q, bits))

"""The quantized key/value cache and its attention on the GPU, through the
binding, against plain 64-bit arithmetic (kv_reference: the tolerances and what
they follow from are there).  Codes, scales and read-back values are exact."""
import numpy as np
import pytest

import kv_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import w4a8_int8_quantized_gb300 as w8


def rows(rng, *shape):
    """Activations with a few strong channels and tokens of unlike size."""
    x = rng.standard_normal(shape) * (1 + 6 * (rng.random(shape[-1]) > 0.97))
    return (x * (0.5 + rng.random(shape[:-1]))[..., None]).astype(np.float16)


class Cache:
    """A cache on the GPU whose tokens are also held here; unwritten rows hold garbage."""

    def __init__(self, rng, lens, heads, D, page, bits, spare=3):
        self.rng, self.page, self.bits, self.heads, self.D = rng, page, bits, heads, D
        counts = [-(-n // page) for n in lens]
        self.pages = sum(counts) + spare
        ids = rng.permutation(self.pages)
        width = max(counts + [1]) + 1
        self.table = rng.integers(0, self.pages, (len(lens), width)).astype(np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = ids[at:at + c]
            at += c
        self.handle = w8.KVCache.empty(self.pages, heads, page, D, bits)
        self.handle.k_codes.view(torch.uint8).fill_(0x88)
        self.handle.v_codes.view(torch.uint8).fill_(0x88)
        self.handle.k_scale.fill_(float("nan"))
        self.handle.v_scale.fill_(float("inf"))
        self.lens = list(lens)
        self.k = [rows(rng, n, heads, D) for n in lens]
        self.v = [rows(rng, n, heads, D) for n in lens]
        if sum(lens):
            slots = np.concatenate([self.slots(b, np.arange(n)) for b, n in enumerate(lens)])
            w8.kv_cache_write(cuda(np.concatenate(self.k)), cuda(np.concatenate(self.v)),
                              cuda(slots), self.handle)

    def slots(self, b, t):
        return self.table[b, t // self.page].astype(np.int64) * self.page + t % self.page

    def quantized(self, b):
        kc, ks = ref.quantize(self.k[b], self.bits)
        vc, vs = ref.quantize(self.v[b], self.bits)
        return kc, ks, vc, vs


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def offsets(new):
    return cuda(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))


def check(c, q, new, out, lse, scale=None, causal=True, window=0):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    scale = c.D ** -0.5 if scale is None else scale
    at = 0
    for b, n in enumerate(new):
        o, s, tol, tol_lse = ref.attend(q[at:at + n], *c.quantized(b), scale, causal, window)
        empty = ~np.isfinite(s)
        assert (out[at:at + n][empty] == 0).all()
        assert (lse[at:at + n][empty] == -np.inf).all()
        err = np.abs(out[at:at + n] - o)
        assert (err <= tol).all(), f"sequence {b}: {err.max()} at {np.unravel_index((err - tol).argmax(), err.shape)}"
        err = np.abs(np.where(empty, 0, lse[at:at + n] - np.where(empty, 0, s)))
        assert (err <= tol_lse).all(), f"lse of sequence {b}: {err.max()}"
        at += n


def attend(c, q, new=None, **kw):
    return w8.kv_cache_attention(cuda(q) if isinstance(q, np.ndarray) else q, c.handle, cuda(c.table),
                                 cuda(np.array(c.lens, np.int32)),
                                 q_offsets=None if new is None else offsets(new), return_lse=True, **kw)


# ------------------------------------------------------------ write, read ----

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,heads,page", [(1, 1, 16), (1, 8, 64), (7, 3, 16), (33, 2, 32), (130, 5, 1024), (257, 16, 128)])
def test_write_and_read(bits, D, T, heads, page):
    rng = np.random.default_rng(T * heads + D + bits)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.1] = -1 - rng.integers(0, 5)
    qkv = rows(rng, T, 3 * heads, D)                        # k and v as strided slices
    qkv[rng.random(T) < 0.1] = 0                            # rows of zeros: scale 0
    tiny = rng.random(T) < 0.1
    qkv[tiny] = (rng.integers(-3, 4, qkv[tiny].shape) * 2.0 ** -24).astype(np.float16)
    qkv[0, -1, :5] = [np.nan, np.inf, -np.inf, 65504, -1]
    x = cuda(qkv)
    cache = w8.KVCache.empty(pages, heads, page, D, bits)
    for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale):
        t.fill_(77)
    w8.kv_cache_write(x[:, heads:2 * heads], x[:, 2 * heads:], cuda(slots), cache)
    got = w8.kv_cache_read(cuda(slots), cache)
    keep = slots >= 0
    for i, (codes, scale, back) in enumerate(((cache.k_codes, cache.k_scale, got[0]),
                                              (cache.v_codes, cache.v_scale, got[1]))):
        q, s = ref.quantize(qkv[:, (i + 1) * heads:(i + 2) * heads], bits)
        want_c = np.full(codes.shape, 77, np.int8 if bits == 8 else np.uint8)
        want_s = np.full(scale.shape, 77, np.float32)
        want_c[slots[keep] // page, :, slots[keep] % page] = ref.pack(q, bits)[keep]
        want_s[slots[keep] // page, :, slots[keep] % page] = s[keep]
        np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
        np.testing.assert_array_equal(scale.cpu().numpy(), want_s)
        value = (q.astype(np.float32) * s[..., None].astype(np.float32)).astype(np.float16)
        value[~keep] = 0
        np.testing.assert_array_equal(back.cpu().numpy(), value)
    assert w8.w8a8_check_status() == 0


def test_slots_outside_the_cache():
    cache = w8.KVCache.empty(2, 1, 16, 64)
    for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale):
        t.fill_(3)
    x = torch.ones(3, 1, 64, dtype=torch.float16, device="cuda")
    slots = torch.tensor([32, 5, 1 << 40], device="cuda")
    w8.kv_cache_write(x, x, slots, cache)
    assert w8.w8a8_check_status() == 7
    assert w8.w8a8_check_status() == 0
    assert (cache.k_scale != 3).sum().item() == 1 and cache.k_scale[0, 0, 5].item() != 3
    k, v = w8.kv_cache_read(slots, cache)
    assert w8.w8a8_check_status() == 7
    assert not k[0].any() and not v[2].any() and k[1].all()


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 4 GB into the buffer."""
    pages = (1 << 32) // (8 * 16 * 64) + 50
    cache = w8.KVCache.empty(pages, 8, 16, 128)
    rng = np.random.default_rng(5)
    n = 100
    c = Cache.__new__(Cache)
    c.rng, c.page, c.bits, c.heads, c.D, c.lens, c.handle = rng, 16, 4, 8, 128, [n], cache
    c.table = np.concatenate([pages - 1 - np.arange(4), [1, 0, pages - 9]]).astype(np.int32)[None]
    c.k, c.v = [rows(rng, n, 8, 128)], [rows(rng, n, 8, 128)]
    slots = cuda(c.slots(0, np.arange(n)))
    w8.kv_cache_write(cuda(c.k[0]), cuda(c.v[0]), slots, cache)
    k, _ = w8.kv_cache_read(slots, cache)
    kc, ks, _, _ = c.quantized(0)
    np.testing.assert_array_equal(k.cpu().numpy(), (kc.astype(np.float32) * ks[..., None].astype(np.float32)).astype(np.float16))
    for new in ([1], [40]):
        q = rows(rng, new[0], 16, 128)
        check(c, q, new, *attend(c, q, new))
    del cache, c
    torch.cuda.empty_cache()


# -------------------------------------------------------- single tokens ----

LENS = [0, 1, 15, 16, 17, 31, 33, 64, 65, 127, 129, 300, 1000]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,group,page", [(1, 1, 16), (2, 4, 16), (3, 8, 64), (2, 3, 32), (1, 16, 128), (2, 7, 1024), (1, 40, 16)])
def test_decode(bits, D, heads, group, page):
    rng = np.random.default_rng(heads + group + D + bits)
    c = Cache(rng, LENS, heads, D, page, bits)
    q = rows(rng, len(LENS), heads * group, D)
    new = [1] * len(LENS)
    check(c, q, new, *attend(c, q))
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("window", [1, 2, 16, 100, 5000])
def test_decode_window(window):
    rng = np.random.default_rng(window)
    c = Cache(rng, LENS, 2, 128, 16, 4)
    q = rows(rng, len(LENS), 8, 128)
    check(c, q, [1] * len(LENS), *attend(c, q, window=window), window=window)


@pytest.mark.parametrize("bits,D", [(4, 128), (8, 64)])
def test_decode_long(bits, D):
    """Long enough for the keys of one sequence to be split many times."""
    rng = np.random.default_rng(bits)
    lens = [20011, 3]
    c = Cache(rng, lens, 2, D, 64, bits)
    q = rows(rng, 2, 8, D)
    check(c, q, [1, 1], *attend(c, q))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("new,group", [([2, 5, 0, 8, 3], 1), ([4, 1, 4, 2, 4], 4), ([3, 3, 3, 3, 3], 5)])
def test_few_queries(bits, new, group):
    """Draft verification: a few queries a sequence, some of them before every key."""
    rng = np.random.default_rng(bits + group)
    c = Cache(rng, [1, 70, 33, 5, 700], 2, 128, 16, bits)
    q = rows(rng, sum(new), 2 * group, 128)
    check(c, q, new, *attend(c, q, new, max_q=max(new)))


# --------------------------------------------------------------- prompts ----

@pytest.mark.parametrize("bits,D", [(4, 128), (4, 64), (8, 128), (8, 64)])
@pytest.mark.parametrize("heads,group,page", [(2, 4, 16), (1, 1, 64), (2, 3, 128), (1, 16, 32)])
def test_prefill(bits, D, heads, group, page):
    rng = np.random.default_rng(bits + D + group)
    lens, new = [200, 64, 131, 1, 40, 0, 513], [200, 64, 17, 1, 55, 6, 100]
    c = Cache(rng, lens, heads, D, page, bits)
    q = rows(rng, sum(new), heads * group, D)
    check(c, q, new, *attend(c, q, new, max_q=max(new)))
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("window", [1, 7, 128, 200])
def test_prefill_window(window):
    rng = np.random.default_rng(window)
    lens, new = [300, 517], [300, 129]
    c = Cache(rng, lens, 2, 128, 16, 4)
    q = rows(rng, sum(new), 4, 128)
    check(c, q, new, *attend(c, q, new, max_q=300, window=window), window=window)


@pytest.mark.parametrize("new", [[1, 1], [3, 90]])
def test_every_key_visible(new):
    rng = np.random.default_rng(3)
    c = Cache(rng, [45, 260], 2, 64, 32, 8)
    q = rows(rng, sum(new), 6, 64)
    check(c, q, new, *attend(c, q, new, causal=False), causal=False)


def test_chunk_behind_a_long_prefix():
    rng = np.random.default_rng(11)
    c = Cache(rng, [3500], 2, 128, 64, 4)
    q = rows(rng, 70, 8, 128)
    check(c, q, [70], *attend(c, q, [70]))


# --------------------------------------------------------- values, layouts ----

@pytest.mark.parametrize("new", [[1, 1, 1], [20, 50, 40]])
@pytest.mark.parametrize("kind", ["zero v", "unlike v", "large scores", "negative scale", "tiny"])
def test_value_ranges(new, kind):
    """Values of zero (scale 0), token sizes over many powers of two, scores far apart."""
    rng = np.random.default_rng(len(kind))
    lens = [60, 200, 333]
    c = Cache(rng, lens, 2, 128, 16, 4)
    scale = 128 ** -0.5
    q = rows(rng, sum(new), 8, 128)
    for b, n in enumerate(lens):
        if kind == "zero v":
            c.v[b][rng.random(n) < 0.5] = 0
            c.v[b][:17] = 0
        elif kind == "unlike v":
            c.v[b] = (c.v[b] * 2.0 ** rng.integers(-12, 8, (n, 1, 1))).astype(np.float16)
        elif kind == "tiny":
            c.v[b] = (c.v[b] * 2.0 ** -18).astype(np.float16)
            c.k[b] = (c.k[b] * 2.0 ** -12).astype(np.float16)
    if kind == "large scores":
        q = (q * 12).astype(np.float16)
    if kind == "negative scale":
        scale = -0.2
    slots = np.concatenate([c.slots(b, np.arange(n)) for b, n in enumerate(lens)])
    w8.kv_cache_write(cuda(np.concatenate(c.k)), cuda(np.concatenate(c.v)), cuda(slots), c.handle)
    check(c, q, new, *attend(c, q, new, softmax_scale=scale), scale=scale)


@pytest.mark.parametrize("new", [[1, 1], [70, 9]])
def test_query_with_nan_keeps_to_itself(new):
    rng = np.random.default_rng(2)
    c = Cache(rng, [100, 40], 2, 128, 16, 4)
    q = rows(rng, sum(new), 8, 128)
    bad = q.copy()
    bad[0, 3, 7] = np.nan
    good, lse = attend(c, q, new)
    out, lse2 = attend(c, bad, new)
    assert torch.isnan(lse2[0, 3]) or torch.isnan(out[0, 3]).any()
    mask = torch.ones(good.shape[:2], dtype=torch.bool, device="cuda")
    mask[0, 3] = False
    assert torch.equal(good[mask], out[mask]) and torch.equal(lse[mask], lse2[mask])


@pytest.mark.parametrize("new", [[1, 1, 1], [30, 80, 7]])
def test_strides_streams_and_repeats(new):
    """q as a slice of a fused projection, on another stream, twice: the same bits."""
    rng = np.random.default_rng(9)
    c = Cache(rng, [90, 150, 2100], 2, 128, 16, 4)
    q = rows(rng, sum(new), 8, 128)
    fused = torch.full((sum(new), 13, 128), float("nan"), dtype=torch.float16, device="cuda")
    fused[:, 3:11] = cuda(q)
    first = attend(c, q, new)
    check(c, q, new, *first)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        again = attend(c, fused[:, 3:11], new)
        third = attend(c, fused[:, 3:11], new)
    stream.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    for a, b in zip(first, third):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new", [[1, 1], [64, 40]])
def test_graph_replay(new):
    """Captured once, replayed after the lengths and the cache have moved on."""
    rng = np.random.default_rng(4)
    c = Cache(rng, [400, 640], 2, 128, 64, 4)
    q, table, off = cuda(rows(rng, sum(new), 8, 128)), cuda(c.table), offsets(new)
    lens = cuda(np.array([100, 90], np.int32))
    run = lambda: w8.kv_cache_attention(q, c.handle, table, lens, q_offsets=off, max_q=max(new), return_lse=True)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run()
    lens.copy_(cuda(np.array(c.lens, np.int32)))
    graph.replay()
    check(c, q.cpu().numpy(), new, out, lse)


def test_indices_outside_their_range():
    """Left out and reported; what is inside stays right."""
    rng = np.random.default_rng(8)
    for new in ([1, 1], [50, 40]):
        c = Cache(rng, [100, 60], 2, 128, 16, 4)
        q = rows(rng, sum(new), 8, 128)
        want = attend(c, q, new)
        good = c.table.copy()
        rest = slice(0, new[0])                                 # the other sequence's rows
        for bad in (c.pages, -1, 2 ** 31 - 1):
            c.table = good.copy()
            c.table[1, 2] = bad
            out = attend(c, q, new)
            assert w8.w8a8_check_status() == 7
            assert torch.equal(out[0][rest], want[0][rest]) and torch.isfinite(out[0]).all()
        c.table = good
        c.lens = [100, 16 * good.shape[1] + 1]                  # beyond the table
        c.table[1] = good[0, 0]
        out = attend(c, q, new)
        assert w8.w8a8_check_status() == 7
        assert torch.equal(out[0][rest], want[0][rest])
        c.lens = [100, -5]
        out = attend(c, q, new)
        assert w8.w8a8_check_status() == 7
        assert not out[0][new[0]:].any() and (out[1][new[0]:] == -np.inf).all()
        c.lens = [100, 60]
        c.table = good
        for off in ([0, new[0], sum(new) + 3], [0, new[0], new[0] - 1], [-2, new[0], sum(new)]):
            w8.kv_cache_attention(cuda(q), c.handle, cuda(c.table), cuda(np.array(c.lens, np.int32)),
                                  q_offsets=cuda(np.array(off, np.int32)))
            assert w8.w8a8_check_status() == 7
        assert w8.w8a8_check_status() == 0


# ------------------------------------------------- how the work is divided ----

@pytest.mark.parametrize("B", [32, 33, 100, 700, 1300])
def test_decode_of_many_sequences(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 60, B).tolist()
    c = Cache(rng, lens, 1, 64, 16, 4)
    q = rows(rng, B, 4, 64)
    check(c, q, [1] * B, *attend(c, q))
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("B", [140, 530, 1100])
def test_prompts_of_many_sequences(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 50, B)
    new = np.minimum(rng.integers(0, 10, B), lens)
    new[7], lens[7] = 90, 90                                 # rows for two blocks of 256
    c = Cache(rng, lens.tolist(), 1, 64, 16, 8)
    q = rows(rng, int(new.sum()), 4, 64)
    check(c, q, new.tolist(), *attend(c, q, new.tolist(), max_q=90))
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("new,group", [([17], 1), ([31, 2], 1), ([32, 32], 1), ([33, 1], 1), ([8, 3], 4),
                                       ([6, 5], 5), ([4], 8), ([5], 8), ([2, 1], 16), ([3, 2], 16)])
def test_rows_around_the_change_of_kernel(new, group):
    rng = np.random.default_rng(sum(new) + group)
    c = Cache(rng, [500, 45][:len(new)], 2, 128, 32, 4)
    q = rows(rng, sum(new), 2 * group, 128)
    check(c, q, new, *attend(c, q, new, max_q=max(new)))
    loose = attend(c, q, new)                                # max_q left to the number of rows
    check(c, q, new, *loose)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [[16], [17], [32], [33]])
def test_rows_around_the_change_of_kernel_by_type(bits, D, new):
    rng = np.random.default_rng(bits + D + new[0])
    c = Cache(rng, [333], 2, D, 16, bits)
    q = rows(rng, new[0], 2, D)
    check(c, q, new, *attend(c, q, new, max_q=new[0]))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,window,causal", [([40], 0, True), ([70], 0, False), ([33, 12], 4000, True), ([300], 700, True)])
def test_long_keys_cut_between_blocks(bits, D, new, window, causal):
    """Items whose keys many blocks share; the joined result is the same each time."""
    rng = np.random.default_rng(bits + D + sum(new))
    c = Cache(rng, [9003, 5000][:len(new)], 1, D, 64, bits)
    q = rows(rng, sum(new), 4, D)
    kw = dict(causal=causal, window=window)
    first = attend(c, q, new, max_q=max(new), **kw)
    check(c, q, new, *first, **kw)
    for _ in range(3):
        for a, b in zip(first, attend(c, q, new, max_q=max(new), **kw)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("new", [[1], [8], [100]])
@pytest.mark.parametrize("page", [16, 1024])
def test_windows_over_released_pages(new, page):
    """Pages wholly before every window may be anyone's: neither read nor reported."""
    rng = np.random.default_rng(page + new[0])
    c = Cache(rng, [6000], 2, 128, page, 4)
    first = (6000 - new[0] + 1 - 300) // page                # page of the first key any row sees
    c.table[0, :first] = -1
    q = rows(rng, new[0], 8, 128)
    check(c, q, new, *attend(c, q, new, window=300), window=300)
    assert w8.w8a8_check_status() == 0


@pytest.mark.parametrize("new", [[1, 1], [40, 3]])
def test_table_much_wider_than_the_lengths(new):
    rng = np.random.default_rng(6)
    c = Cache(rng, [77, 300], 2, 128, 16, 4)
    wide = np.full((2, 20000), 2 ** 31 - 1, np.int32)
    wide[:, :c.table.shape[1] - 1] = c.table[:, :-1]
    c.table = wide
    q = rows(rng, sum(new), 8, 128)
    check(c, q, new, *attend(c, q, new))
    assert w8.w8a8_check_status() == 0


def test_pages_in_order_and_out_of_order():
    """Runs of neighbouring pages, and none: the same bits."""
    rng = np.random.default_rng(12)
    n = 3000
    for bits, D in ((4, 128), (8, 64)):
        c = Cache(rng, [n], 2, D, 16, bits)
        q = rows(rng, 1, 8, D)
        apart = attend(c, q)
        count = -(-n // 16)
        c.table = np.arange(c.pages - count, c.pages, dtype=np.int32)[None]
        w8.kv_cache_write(cuda(c.k[0]), cuda(c.v[0]), cuda(c.slots(0, np.arange(n))), c.handle)
        together = attend(c, q)
        check(c, q, [1], *together)
        for a, b in zip(apart, together):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bits,D", [(4, 128), (4, 64), (8, 128), (8, 64)])
@pytest.mark.parametrize("new,group", [([32], 1), ([9, 32, 19], 1), ([8], 4), ([16], 2), ([60], 1)])
def test_scales_left_by_an_earlier_call(bits, D, new, group):
    """On-chip memory full of another call's NaN scales: keys that no row of a block
    sees are not fetched, and what is there instead must not count."""
    rng = np.random.default_rng(bits + D + sum(new))
    dirt = w8.KVCache.empty(2000, 2, 16, D, bits)
    dirt.k_codes.zero_()
    dirt.v_codes.zero_()
    dirt.k_scale.fill_(float("nan"))
    dirt.v_scale.fill_(float("nan"))
    table = torch.arange(2000, dtype=torch.int32, device="cuda")[None].repeat(4, 1)
    c = Cache(rng, [39, 41, 300][:len(new)], 2, D, 32, bits)
    q = rows(rng, sum(new), 2 * group, D)
    for _ in range(3):
        x = torch.zeros(4 * new[0], 2 * group, D, dtype=torch.float16, device="cuda")
        w8.kv_cache_attention(x, dirt, table, torch.full((4,), 32000, dtype=torch.int32, device="cuda"),
                              q_offsets=torch.arange(5, dtype=torch.int32, device="cuda") * new[0], max_q=max(new))
        check(c, q, new, *attend(c, q, new, max_q=max(new)))


def test_refusals():
    c = w8.KVCache.empty(4, 2, 16, 64)
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    for err, f in ((TypeError, lambda: w8.kv_cache_attention(q.float(), c, table, lens)),
                   (TypeError, lambda: w8.kv_cache_attention(q, c, table.long(), lens)),
                   (ValueError, lambda: w8.kv_cache_attention(q, c, table, lens.cpu())),
                   (ValueError, lambda: w8.kv_cache_attention(q, c, table, lens.repeat(2))),
                   (ValueError, lambda: w8.kv_cache_attention(q[..., :32], c, table, lens)),
                   (ValueError, lambda: w8.kv_cache_attention(q.transpose(1, 2).contiguous().transpose(1, 2), c, table, lens)),
                   (w8.W8A8Error, lambda: w8.kv_cache_attention(q[:, :3].contiguous(), c, table, lens)),
                   (w8.W8A8Error, lambda: w8.kv_cache_attention(q, c, table, lens, causal=False, window=3)),
                   (ValueError, lambda: w8.kv_cache_write(q, q, slots, c)),
                   (TypeError, lambda: w8.kv_cache_write(q[:, :2], q[:, :2], slots.int(), c)),
                   (ValueError, lambda: w8.kv_cache_write(q[:, :2], q[:, :2], slots.repeat(2), c)),
                   (TypeError, lambda: w8.kv_cache_read(slots.int(), c))):
        with pytest.raises(err):
            f()
    if w8.kv_cache_attention_workspace_bytes(1, 4, c, table, 1):
        with pytest.raises(w8.W8A8Error):
            w8.kv_cache_attention(q, c, table, lens, workspace=ws)


def test_nothing_to_do():
    c = w8.KVCache.empty(4, 2, 16, 64)
    none = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    slots = torch.zeros(0, dtype=torch.int64, device="cuda")
    w8.kv_cache_write(none, none, slots, c)
    k, v = w8.kv_cache_read(slots, c)
    assert k.shape == v.shape == (0, 2, 64)
    out = w8.kv_cache_attention(none, c, torch.zeros(2, 4, dtype=torch.int32, device="cuda"),
                                torch.zeros(2, dtype=torch.int32, device="cuda"),
                                q_offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 2, 64)
    # no table at all: every sequence is empty
    q = torch.ones(2, 2, 64, dtype=torch.float16, device="cuda")
    out, lse = w8.kv_cache_attention(q, c, torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                                     torch.zeros(2, dtype=torch.int32, device="cuda"), return_lse=True)
    assert not out.any() and (lse == -np.inf).all()
    assert w8.w8a8_check_status() == 0

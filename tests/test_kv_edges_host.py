"""Limits of the key/value cache calls that are decided on the host (no GPU needed)."""
import pytest

from test_kv_cache_host import INV, WS, attend, cache, lib  # noqa: F401  (lib: a fixture)


@pytest.mark.parametrize("page", [16, 1024])
def test_tokens_of_a_table(lib, page):  # noqa: F811
    """Positions a little past a sequence's end have to fit 32 bits too: a table of up to
    2^31 - 65536 tokens passes (and is refused for its workspace only), a wider one does not."""
    c, most = cache(page_size=page), (2 ** 31 - 65536) // page
    for max_q in (1, 8, 100):
        assert attend(lib, c, T=200, width=most + 1, max_q=max_q) == INV
        assert attend(lib, c, T=200, width=2 ** 31 // page - 1, max_q=max_q) == INV
        assert attend(lib, c, T=200, width=most, max_q=max_q, wsb=0) == WS

"""Sizes at which a paged call's 32-bit indexes would wrap are refused on the host: nothing is launched, no GPU is needed."""
import pytest

from test_paged_host import CALLS, lib  # noqa: F401


@pytest.mark.parametrize("n", [(1 << 30) + 1, 2 ** 31 - 255, 2 ** 31 - 1])
def test_longest_list_of_pages(lib, n):  # noqa: F811
    """Blocks step through a list by 256 or 512 entries: an index near 2^31 would wrap to a negative one."""
    a = dict(CALLS["g3attn_page_select"], n=n)
    assert lib.g3attn_page_select(*a.values()) == 2
    assert lib.g3attn_last_error().startswith(b"page_select")

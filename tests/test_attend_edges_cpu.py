"""The paged cache's entry points at the edge of what they accept, and the division of an attention call with the
constants that its kernels run with, on a host-only build."""
import pytest

from test_attend_host_cpu import L, OK, EUNSUP, append, attend, launches, reset  # noqa: F401


# ---------------------------------------------------------------- large pages
@pytest.mark.timeout(20, method="thread")
@pytest.mark.parametrize("page", [(1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 1])
def test_pages_of_any_size(L, page):  # noqa: F811
    """Such a page holds more keys than a request may have, but a table without columns reads none of them."""
    assert L.stub_page_of(page, (1 << 24) - 1) == 0 and L.stub_page_of(page, 0) == 0
    assert attend(L, pages=1, page=page, cols=0, ldt=0, table=0) == OK
    assert len(launches(L)) == 1
    assert attend(L, pages=1, page=page) == EUNSUP
    assert append(L, pages=1, page=page) == OK

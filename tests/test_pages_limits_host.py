"""Limits that the calls on selected pages share (no GPU needed)."""

import pytest

from tests.helpers import ensure_built
from tests.test_block_host import UNSUPPORTED, _cache, _call
from tests.test_pages_host import BOUNDS, PAGES, SCORES, SELECT


@pytest.fixture(scope="module")
def B():
    return ensure_built()


@pytest.mark.parametrize("fn,args", [("moe_page_bounds", BOUNDS), ("moe_page_scores", SCORES), ("moe_page_select", SELECT),
                                     ("moe_attn_pages", PAGES)])
def test_pages_of_a_table(B, fn, args):
    """Every call on pages takes 2^30 of them to a table, and no more."""
    over = dict(pages=2**30 + 1)
    if "ld" in args:
        over["ld"] = 2**31
    if "cache" in args:
        over["cache"] = _cache(B)
    assert _call(getattr(B.lib(), fn), args, over) == UNSUPPORTED
    assert "max_pages" in B.lib().moe_last_error().decode()

"""Host-side checks of the calls on selected pages (no GPU needed)."""

import pytest
import torch

from tests.helpers import ensure_built
from tests.test_block_host import ATTN, BAD_CACHES, BF16, FP8, INVALID, P, UNSUPPORTED, WORKSPACE, _cache, _call

BOUNDS = dict(cache=None, bounds=P, table=P, ld=4, pages=4, B=2, lens=P, first=None, status=None, stream=None)
SCORES = dict(q=P, dt=BF16, qb=512, qh=64, B=2, hq=8, cache=None, bounds=P, table=P, ld=4, pages=4, lens=P, scores=P,
              status=None, stream=None)
SELECT = dict(scores=P, B=2, heads=4, table=P, ld=4, pages=4, lens=P, page=16, keep=8, sinks=1, recent=1, tables=P, kept=P,
              stream=None)
PAGES = {n: ATTN[n] for n in ATTN if n not in ("ld", "window")}


@pytest.fixture(scope="module")
def B():
    return ensure_built()


@pytest.mark.parametrize("fn,args", [("moe_page_bounds", BOUNDS), ("moe_page_scores", SCORES), ("moe_attn_pages", PAGES)])
@pytest.mark.parametrize("over,code,text", BAD_CACHES)
def test_bad_caches(B, fn, args, over, code, text):
    assert _call(getattr(B.lib(), fn), args, dict(cache=_cache(B, **over))) == code
    assert text in B.lib().moe_last_error().decode()
    assert _call(getattr(B.lib(), fn), args, {}) == INVALID       # no cache at all


REQUESTS = [(dict(B=-1), INVALID, "B"), (dict(pages=-1), INVALID, "max_pages"), (dict(ld=3), INVALID, "table_ld"),
            (dict(table=None), INVALID, "null"), (dict(lens=None), INVALID, "null")]


@pytest.mark.parametrize("over,code,text", REQUESTS + [
    (dict(bounds=None), INVALID, "bounds"),
    (dict(bounds=P + 8), INVALID, "bounds"),
])
def test_bounds_refusals(B, over, code, text):
    assert _call(B.lib().moe_page_bounds, dict(BOUNDS, cache=_cache(B)), over) == code
    assert text in B.lib().moe_last_error().decode()


@pytest.mark.parametrize("over,code,text", REQUESTS + [
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(hq=6), INVALID, "q_heads"),
    (dict(hq=0), INVALID, "q_heads"),
    (dict(q=None), INVALID, "q null"),
    (dict(q=P + 2), INVALID, "unaligned"),
    (dict(qh=60), INVALID, "stride"),
    (dict(bounds=None), INVALID, "bounds"),
    (dict(bounds=P + 8), INVALID, "bounds"),
    (dict(scores=None), INVALID, "null"),
])
def test_scores_refusals(B, over, code, text):
    assert _call(B.lib().moe_page_scores, dict(SCORES, cache=_cache(B)), over) == code
    assert text in B.lib().moe_last_error().decode()


@pytest.mark.parametrize("over,code,text", REQUESTS + [
    (dict(heads=0), INVALID, "heads"),
    (dict(page=0), INVALID, "page_size"),
    (dict(keep=0), INVALID, "keep"),
    (dict(sinks=-1), INVALID, "sinks"),
    (dict(recent=-1), INVALID, "recent"),
    (dict(sinks=4, recent=5), INVALID, "keep"),
    (dict(sinks=2**31 - 1, recent=2**31 - 1), INVALID, "keep"),
    (dict(B=1 << 20, heads=1 << 12), UNSUPPORTED, "2^31"),
    (dict(scores=None), INVALID, "null"),
    (dict(tables=None), INVALID, "null"),
    (dict(kept=None), INVALID, "null"),
])
def test_select_refusals(B, over, code, text):
    assert _call(B.lib().moe_page_select, SELECT, over) == code
    assert text in B.lib().moe_last_error().decode()


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=FP8), UNSUPPORTED, "dtypes"),
    (dict(odt=FP8), UNSUPPORTED, "dtypes"),
    (dict(B=-1), INVALID, "B"),
    (dict(hq=6), INVALID, "q_heads"),
    (dict(pages=-1), INVALID, "max_pages"),
    (dict(cap=-1.0), INVALID, "softcap"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(q=None), INVALID, "q or out"),
    (dict(oh=60), INVALID, "stride"),
    (dict(table=None), INVALID, "null"),
    (dict(lens=None), INVALID, "null"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws_bytes=64), WORKSPACE, "required"),
    (dict(B=1 << 30), UNSUPPORTED, "2^31"),
])
def test_attn_pages_refusals(B, over, code, text):
    over = dict(over)
    if over.get("B", 0) > 2:
        over["ws_bytes"] = 1 << 60
    assert _call(B.lib().moe_attn_pages, dict(PAGES, cache=_cache(B)), over) == code
    assert text in B.lib().moe_last_error().decode()


@pytest.mark.parametrize("over", [dict(B=2**30 + 1, heads=1), dict(pages=2**30 + 1, ld=2**31), dict(keep=2**30 + 1),
                                  dict(B=2**28 + 1)])
def test_select_more_than_an_index_steps_over(B, over):
    assert _call(B.lib().moe_page_select, SELECT, over) == UNSUPPORTED
    assert "2^30" in B.lib().moe_last_error().decode()


@pytest.mark.parametrize("over", [dict(B=2**30 + 1), dict(pages=2**30 + 1, ld=2**31)])
def test_bounds_and_scores_of_more_than_an_index_steps_over(B, over):
    for fn, args in (("moe_page_bounds", BOUNDS), ("moe_page_scores", SCORES)):
        assert _call(getattr(B.lib(), fn), dict(args, cache=_cache(B)), over) == UNSUPPORTED
        assert "2^30" in B.lib().moe_last_error().decode()


def test_attn_pages_of_more_tables_than_an_index_steps_over(B):
    over = dict(B=2**28 + 1, ws_bytes=1 << 60)       # of 4 heads each
    assert _call(B.lib().moe_attn_pages, dict(PAGES, cache=_cache(B)), over) == UNSUPPORTED
    assert "2^30" in B.lib().moe_last_error().decode()


def test_no_requests(B):
    """Nothing is launched, and pointers of an empty batch are not asked for."""
    L, none = B.lib(), dict(B=0, table=None, lens=None)
    assert _call(L.moe_page_bounds, dict(BOUNDS, cache=_cache(B)), dict(none, bounds=None)) == 0
    assert _call(L.moe_page_scores, dict(SCORES, cache=_cache(B)), dict(none, q=None, bounds=None, scores=None)) == 0
    assert _call(L.moe_page_select, SELECT, dict(none, scores=None, tables=None, kept=None)) == 0
    assert _call(L.moe_attn_pages, dict(PAGES, cache=_cache(B)), dict(none, q=None, out=None, ws=None)) == 0


def test_binding_refuses_what_is_no_cache_or_no_tensor(B):
    x, i = torch.zeros(1, 2, 64), torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: B.moe_page_bounds(None, x, i, i[0]), lambda: B.moe_page_scores(x, 3, x, i, i[0], x),
                 lambda: B.moe_attn_pages(x, x, i, i, 1.0, x, i)):
        with pytest.raises(ValueError, match="KvCache"):
            call()
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.moe_page_select(x, i, i[0], 16, i, i)

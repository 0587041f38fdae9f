"""moe_page_select where its blocks differ: every width of a block (256, 512 and 1024 threads, by pages and heads), all pages
in one turn or in several, and scores without a first or last one among them.

Selections are exact.  The outputs lie between guard words, which stay as they were.
"""

import math

import pytest
import torch

from tests.helpers import ensure_built
from tests.test_gpu_block import gen, normal

pytestmark = pytest.mark.gpu

INT = dict(dtype=torch.int32, device="cuda")
GUARD, KEYS = 4096, 8           # words; keys of a thread in one turn


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def best_columns(scores, pages, keep, sinks, recent):
    """[heads, keep] columns kept of the first ``pages`` of scores [heads, width] (more than ``keep``), in order."""
    s = scores[:, :pages].double().cpu()
    rank = torch.where(torch.isnan(s), 1e200, s.clamp(-1e100, 1e100))
    rank[:, :sinks] = 1e300
    rank[:, pages - recent:] = 1e300
    return torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :keep].sort(dim=1).values


def guarded(*shape):
    """(tensor of 99, all words around it included) contiguous, between guard words."""
    n = math.prod(shape)
    room = torch.full((n + 2 * GUARD,), 99, **INT)
    return room[GUARD:GUARD + n].view(*shape), room


def check(B, scores, lens, page, keep, sinks, recent, runs=1, seed=0):
    """scores [requests, heads, width]; every request has more than ``keep`` pages."""
    nb, heads, width = scores.shape
    table = torch.randint(0, 1 << 30, (nb, width), generator=gen(seed), **INT)
    seq = torch.tensor(lens, **INT)
    want = torch.empty(nb, heads, keep, dtype=torch.int32)
    n_want = torch.empty(nb, heads, dtype=torch.int32)
    host = table.cpu()
    for b, n in enumerate(lens):
        pages = -(-n // page)
        assert keep < pages <= width
        cols = best_columns(scores[b], pages, keep, sinks, recent)
        want[b] = host[b][cols]
        n_want[b] = keep * page - (cols[:, -1] == pages - 1).int() * (pages * page - n)
    for i in range(runs):
        (tables, t_room), (kept, k_room) = guarded(nb, heads, keep), guarded(nb, heads)
        B.moe_page_select(scores, table, seq, page, tables, kept, sinks=sinks, recent=recent)
        torch.cuda.synchronize()
        for name, got, room, w in (("tables", tables, t_room, want), ("lens", kept, k_room, n_want)):
            assert (room[:GUARD] == 99).all() and (room[-GUARD:] == 99).all(), f"words beside {name}, run {i}"
            assert torch.equal(got.cpu(), w), f"{name}, run {i}"


def blocks_of(threads):
    """(requests, heads) that get blocks of so many threads for more pages than the next narrower ones have in a turn."""
    return {256: (128, 9), 512: (sms() // 2, 4), 1024: (sms() // 4, 4)}[threads]


# pages of one turn of the narrower blocks, and one more; a full turn; some of both
WIDTHS = {256: [40, 255, 1000, 2048], 512: [2049, 3000, 4096], 1024: [4097, 5001, 8192]}


@pytest.mark.parametrize("threads,pages", [(t, p) for t in WIDTHS for p in WIDTHS[t]])
@pytest.mark.parametrize("kind", ["equal", "lowest", "nan", "zeros", "forced"])
def test_select_of_scores_that_are_all_alike(B, threads, pages, kind):
    """No key is above another, so that nothing is looked for: the first pages, and those that are forced."""
    nb, heads = blocks_of(threads)
    value = {"equal": 3.0, "lowest": -math.inf, "nan": math.nan, "zeros": 0.0, "forced": 3.0}[kind]
    scores = torch.full((nb, heads, pages), value, device="cuda")
    if kind == "zeros":
        scores[:, :, ::3] = -0.0
    if kind == "forced":              # all that are kept, whatever the scores
        check(B, normal(gen(1), nb, heads, pages), [pages] * nb, 1, 24, 20, 4, runs=4)
    for keep, sinks, recent in ((24, 4, 8), (1, 0, 0), (33, 0, 0)):
        check(B, scores, [pages] * nb, 1, keep, sinks, recent, runs=4)


@pytest.mark.parametrize("threads", [256, 512, 1024])
def test_select_of_two_pages_alike(B, threads):
    """Two pages beside the forced ones, of one score."""
    nb, heads = blocks_of(threads)
    pages = WIDTHS[threads][0]
    scores = normal(gen(2), nb, heads, pages)
    scores[:, :, 30:32] = 1.5
    check(B, scores, [pages * 2 - 1] * nb, 2, pages - 1, 30, pages - 32, runs=8)


# turns of 8 keys a thread: one of them, one and a page, several
ARMS = [(256, "many", 2048), (256, "many", 2049), (256, "many", 5000), (512, "few", 2049), (512, "few", 3000), (512, "few", 4096),
        (512, "some", 4097), (512, "some", 9000), (1024, "few", 4097), (1024, "few", 8193), (1024, "few", 20000)]


@pytest.mark.parametrize("threads,heads,pages", ARMS)
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 8)])
def test_select_widths_of_blocks_and_turns(B, threads, heads, pages, sinks, recent):
    """``heads``: more than two to an SM, up to two, or up to one.  Ties lie across the turns' borders, and the last page, a
    partial one, is kept by some heads and not by others."""
    nb, hkv = {"few": (3, 2), "some": (sms() // 4 + 1, 5), "many": (sms() // 2 + 1, 5)}[heads]
    g = gen(pages)
    scores = normal(g, nb, hkv, pages)
    for border in range(threads * KEYS, pages, threads * KEYS):
        scores[:, 0, border - 3:border + 3] = 2.5
        scores[:, 1, border - 1:border + 1] = 5.0
    other = torch.randint(0, pages, scores.shape, generator=g, device="cuda")
    scores = torch.where(torch.rand(scores.shape, generator=g, device="cuda") < 0.2, scores.gather(2, other), scores)
    scores[:, 0, pages - 1] = -9.0
    scores[:, 1, pages - 1] = 9.0
    lens = [3 * pages - 1 - i % 2 for i in range(nb)]
    for keep in (13, 200):
        check(B, scores.contiguous(), lens, 3, keep, sinks, recent, seed=keep)


@pytest.mark.parametrize("threads,heads,pages", [a for a in ARMS if a[2] > a[0] * KEYS])
def test_select_of_scores_alike_in_turns(B, threads, heads, pages):
    nb, hkv = {"few": (3, 2), "some": (sms() // 4 + 1, 5), "many": (sms() // 2 + 1, 5)}[heads]
    for value in (1.0, math.nan, -math.inf):
        scores = torch.full((nb, hkv, pages), value, device="cuda")
        check(B, scores, [pages] * nb, 1, 100, 1, 2, runs=2)
    turn = threads * KEYS             # and the first ones of a score end at a border, or one beyond
    for keep in (turn, turn + 1):
        if keep < pages:
            check(B, scores, [pages] * nb, 1, keep, 0, 0, runs=2)

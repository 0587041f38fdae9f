"""Attention over selected pages against the fp64 oracle: bounds, scores, selection, attention.

Bounds and selections are exact.  A score is, with u = 2^-24, a sum of G queries per channel (G - 1
roundings), a chain of 16 multiply-adds at most, 5 levels over the lanes and the scale of the keys: within
(G + 22) u of the sum of its terms' absolute values.  All of a channel's summed queries have one sign per
side, so that those absolute values are the terms' own (where lo <= 0 <= hi; elsewhere the two sides are
taken apart).  Attention: see test_gpu_block.py.
"""

import importlib.util
import math
import os
import subprocess
import sys

import pytest
import torch

from moe_decode_layer_fp32_gb300 import synth
from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import BF, DT, U, assert_within, cos_sin_table, gen, make_cache, normal, raw

pytestmark = pytest.mark.gpu

INT = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def make_table(g, lens, page, pad=0, spare=2):
    """(table [B, most + pad] with nonsense behind each request's pages, number of pages)"""
    need = [-(-max(n, 0) // page) for n in lens]
    pages = sum(need) + spare
    ids = torch.randperm(pages, generator=g, device="cuda").tolist()
    table = torch.full((len(lens), max(max(need), 1) + pad), -12345, dtype=torch.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
        at += c
    return table.cuda(), pages


def poison_unseen(k, table, lens, page, dtype):
    """NaN in every slot that no request has."""
    seen = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(-(-max(n, 0) // page)):
            seen[int(table[b, j]), :min(page, n - j * page)] = True
    raw(k)[~seen.cuda()] = 0x7F if dtype == "e4m3" else 0x7FC0


# ------------------------------------------------------------------------ bounds


def bounds_case(B, lens, first=None, hkv=3, D=128, page=16, dtype="bf16", heads_first=False, seed=0, pad=0):
    g = gen(seed)
    table, pages = make_table(g, lens, page, pad)
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype, heads_first)
    poison_unseen(k, table, lens, page, dtype)
    bounds = B.new_page_bounds(cache)
    raw(bounds).fill_(0x55)
    seq = torch.tensor(lens, **INT)
    f = torch.tensor(first, **INT) if first is not None else None
    status = torch.zeros(1, **INT)
    B.moe_page_bounds(cache, bounds, table, seq, first=f, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    written = torch.zeros(pages, dtype=torch.bool)
    got = O.f64(bounds)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        rows = O.cached_rows(k, None, table[b], 0, n)      # codes as they are: bounds hold codes
        for col, (lo, hi) in O.page_bounds(rows, page, first[b] if first is not None else 0, n).items():
            p = int(table[b, col])
            written[p] = True
            assert torch.equal(got[p, :, 0], lo) and torch.equal(got[p, :, 1], hi), f"page {col} of request {b}"
    assert (raw(bounds).cpu()[~written] == 0x55).all()


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("D", [16, 64, 80, 128, 256])
def test_bounds(B, dtype, heads_first, D):
    bounds_case(B, LENGTHS, D=D, dtype=dtype, heads_first=heads_first, seed=D)


@pytest.mark.parametrize("D", [8, 24, 72, 136, 248])
def test_bounds_head_dims_of_eight(B, D):
    bounds_case(B, LENGTHS, D=D, seed=D)


@pytest.mark.parametrize("page", [1, 2, 3, 7, 24, 64, 100, 128, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_bounds_page_sizes(B, page, dtype):
    bounds_case(B, [5, 0, 1000, 2049, 1], page=page, hkv=2, D=64, dtype=dtype, seed=page)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_bounds_from_the_first_new_token(B, dtype):
    lens = [0, 1, 16, 17, 40, 64, 300, 5, 9]
    bounds_case(B, lens, first=[max(n - 1, 0) for n in lens], dtype=dtype, seed=1)
    bounds_case(B, lens, first=[0, -7, 16, 16, 20, 63, 100, 9, 9], dtype=dtype, seed=2)
    bounds_case(B, [4000] * 3, first=[3990, 0, 17], hkv=8, dtype=dtype, seed=3)


@pytest.mark.parametrize("lens", [[1] * 300, [0] * 700 + [3], [20] * 1500, [30000], [9000, 0, 1] * 3])
def test_bounds_many_requests_and_long_ones(B, lens):
    bounds_case(B, lens, hkv=2, D=64, seed=len(lens), pad=3)


def test_bounds_of_special_keys(B):
    """Infinities count, zeros of either sign are alike, NaN shows, and the other channels are as they were."""
    for dtype in ("bf16", "e4m3"):
        g = gen(4)
        k, v, ks, vs, cache = make_cache(B, g, 2, 8, 2, 16, dtype)
        w = k.float()
        w[0, 3, 0, 1] = math.nan
        w[0, 2, 1, 2] = -448.0
        w[0, 4, 1, 2] = 448.0
        if dtype == "bf16":
            w[0, 5, 1, 3], w[0, 6, 1, 4] = math.inf, -math.inf
        w[0, :, 1, 5] = torch.tensor([0.0, -0.0] * 4)
        w[0, :, 1, 6] = torch.tensor([2.0 ** -9, -2.0 ** -9, 3 * 2.0 ** -9, 0.0] * 2)
        k.copy_(w.to(k.dtype))
        bounds = B.new_page_bounds(cache)
        B.moe_page_bounds(cache, bounds, torch.zeros(1, 1, **INT), torch.tensor([8], **INT))
        got, rows = O.f64(bounds[0]), O.f64(k[0])
        assert torch.isnan(got[0, :, 1]).any()
        rows[:, 0, 1] = 0.0
        got[0, :, 1] = 0.0
        assert torch.equal(got[:, 0], rows.min(0).values) and torch.equal(got[:, 1], rows.max(0).values)


def test_bounds_reports_what_it_cannot_read(B):
    g = gen(5)
    k, v, _, _, cache = make_cache(B, g, 4, 8, 2, 64, "bf16")
    for bad in ("length", "page_high", "page_negative"):
        table, seq = torch.arange(4, **INT).view(2, 2), torch.tensor([16, 16], **INT)
        if bad == "length":
            seq[1] = 2**31 - 1
        else:
            table[1, 1] = 4 if bad == "page_high" else -1
        bounds, status = B.new_page_bounds(cache).fill_(7.0), torch.zeros(1, **INT)
        B.moe_page_bounds(cache, bounds, table, seq, status=status)
        assert status.item() == -6
        for p in range(4):
            if bad != "length" and p == 3:
                assert (bounds[p] == 7.0).all()
            else:
                assert torch.equal(bounds[p, :, 0], k[p].amin(0)) and torch.equal(bounds[p, :, 1], k[p].amax(0))
        B.moe_page_bounds(cache, bounds, table, seq)                 # without a status word


# ------------------------------------------------------------------------ scores


def scores_case(B, lens, hq=6, hkv=3, D=128, page=16, q="bf16", dtype="bf16", seed=0, pad=0, strided=False):
    g = gen(seed)
    table, pages = make_table(g, lens, page, pad)
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype)
    mid, wide = normal(g, pages, hkv, D), normal(g, pages, hkv, D).abs()
    edge = torch.stack([mid - wide, mid + wide], 2)
    bounds = (edge if ks is None else (edge / ks[:, None, None]).clamp(-448, 448)).to(k.dtype)
    room = normal(g, len(lens), hq + 2, D + 8, dtype=DT[q])
    qt = room[:, 1:-1, 8:] if strided else room[:, 1:-1, 8:].contiguous()
    scores = torch.full((len(lens), hkv, table.shape[1]), 77.0, device="cuda")
    status = torch.zeros(1, **INT)
    B.moe_page_scores(qt, cache, bounds, table, torch.tensor(lens, **INT), scores, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for b, n in enumerate(lens):
        j = -(-max(n, 0) // page)
        assert (scores[b, :, j:] == 77.0).all()
        if not j:
            continue
        at = table[b, :j].long().cpu()
        lo, hi = (O.f64(bounds)[at][:, :, i] * (O.f64(ks)[:, None] if ks is not None else 1.0) for i in (0, 1))
        want, _ = O.page_scores(qt[b], lo, hi)
        # the two sides apart
        qd = O.f64(qt[b]).view(hkv, hq // hkv, D)
        size = (qd.clamp(max=0).sum(1).abs()[None] * lo.abs() + qd.clamp(min=0).sum(1)[None] * hi.abs()).sum(2).T
        assert_within(scores[b, :, :j], want, (hq // hkv + 22) * U * size, f"request {b}")


@pytest.mark.parametrize("D", [8, 16, 24, 32, 48, 64, 80, 96, 128, 144, 192, 248, 256])
@pytest.mark.parametrize("q", ["f32", "bf16"])
def test_scores_head_dims(B, D, q):
    scores_case(B, [0, 1, 40, 700], D=D, q=q, seed=D)
    if D % 16 == 0:
        scores_case(B, [0, 1, 40, 700], D=D, q=q, dtype="e4m3", seed=D)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (7, 1), (16, 1), (24, 2), (8, 8), (56, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_scores_head_groups(B, hq, hkv, dtype):
    scores_case(B, [100, 0, 33], hq=hq, hkv=hkv, dtype=dtype, seed=hq)


@pytest.mark.parametrize("lens", [LENGTHS, [1] * 300, [0] * 700 + [3], [40000], [9000, 0, 1] * 3, [500] * 100])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
def test_scores_lengths(B, lens, page):
    scores_case(B, lens, hq=4, hkv=2, D=64, page=page, seed=page, pad=2)


def test_scores_strided_q(B):
    scores_case(B, [100, 3, 257], strided=True, seed=1)
    scores_case(B, [100, 3, 257], strided=True, q="f32", dtype="e4m3", seed=2)


def test_scores_are_bounds(B):
    """No key of a page scores more, and a page of one key scores what that does."""
    g = gen(6)
    lens, page = [200, 33], 16
    table, pages = make_table(g, lens, page)
    k, v, ks, vs, cache = make_cache(B, g, pages, page, 2, 64, "bf16")
    bounds, q = B.new_page_bounds(cache), normal(g, 2, 4, 64)
    seq, scores = torch.tensor(lens, **INT), torch.zeros(2, 2, table.shape[1], device="cuda")
    B.moe_page_bounds(cache, bounds, table, seq)
    B.moe_page_scores(q, cache, bounds, table, seq, scores)
    for b, n in enumerate(lens):
        s = torch.einsum("ghd,lgd->gl", O.f64(q[b]).view(2, 2, 64), O.cached_rows(k, None, table[b], 0, n))
        for j in range(-(-n // page)):
            top = s[:, j * page:(j + 1) * page].max(1).values
            assert (O.f64(scores[b, :, j]) >= top - 1e-4).all()
            if j * page == n - 1:
                assert_within(scores[b, :, j], top, 1e-4, "one key")


def test_scores_of_special_values(B):
    """A NaN query or bound spoils its own head and page; a page outside the cache scores -inf."""
    g = gen(7)
    k, v, _, _, cache = make_cache(B, g, 6, 16, 2, 64, "bf16")
    bounds = torch.stack([k.amin(1), k.amax(1)], 2).contiguous()
    bounds[2, 1, 0, 3] = math.nan
    q = normal(g, 2, 4, 64)
    q[1, 3, 9] = math.nan
    table, seq = torch.tensor([[0, 1, 2], [3, 6, -2**31]], **INT), torch.tensor([48, 40], **INT)
    scores, status = torch.zeros(2, 2, 3, device="cuda"), torch.zeros(1, **INT)
    B.moe_page_scores(q, cache, bounds, table, seq, scores, status=status)
    assert status.item() == -6
    nan = torch.isnan(scores).cpu()
    assert nan.tolist() == [[[False, False, False], [False, False, True]], [[False, False, False], [True, False, False]]]
    assert (scores[1, :, 1:] == -math.inf).all()
    seq[1], table[1] = 2**31 - 1, torch.tensor([3, 4, 5], **INT)
    status.zero_()
    B.moe_page_scores(q, cache, bounds, table, seq, scores, status=status)
    assert status.item() == -6 and torch.isfinite(scores[1, 0]).all()
    B.moe_page_scores(q, cache, bounds, table, seq, scores)


# ------------------------------------------------------------------------ select


def select_case(B, lens, hkv=2, page=16, keep=8, sinks=1, recent=2, scores=None, seed=0, pad=0):
    g = gen(seed)
    width = max(max(-(-max(n, 0) // page) for n in lens), 1) + pad
    table = torch.randint(0, 1 << 30, (len(lens), width + 3), generator=g, device="cuda", dtype=torch.int32)[:, :width]
    if scores is None:
        scores = 40 + 10 * normal(g, len(lens), hkv, width)
        # ties: some scores are those of another page
        other = torch.randint(0, width, scores.shape, generator=g, device="cuda")
        scores = torch.where(torch.rand(scores.shape, generator=g, device="cuda") < 0.3, scores.gather(2, other), scores)
    scores = scores.contiguous()
    tables, kept = torch.full((len(lens), hkv, keep), 99, **INT), torch.full((len(lens), hkv), 99, **INT)
    B.moe_page_select(scores, table, torch.tensor(lens, **INT), page, tables, kept, sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    ids, sc = table.cpu().tolist(), scores.cpu().tolist()
    got, n_got = tables.cpu().tolist(), kept.cpu().tolist()
    for b, n in enumerate(lens):
        pages = -(-max(n, 0) // page)
        for h in range(hkv):
            cols = O.page_select(sc[b][h], pages, keep, sinks, recent)
            assert got[b][h] == [ids[b][j] for j in cols] + [-1] * (keep - len(cols)), f"request {b}, head {h}"
            assert n_got[b][h] == sum(min(page, n - j * page) for j in cols)


@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (8, 1, 2), (8, 8, 0), (8, 0, 8), (8, 3, 5),
                                               (64, 4, 8), (200, 1, 1)])
def test_select_lengths(B, keep, sinks, recent):
    select_case(B, LENGTHS + [1000, 1600, 4096], keep=keep, sinks=sinks, recent=recent, seed=keep)


@pytest.mark.parametrize("page", [1, 3, 64, 1000])
def test_select_page_sizes(B, page):
    select_case(B, [0, 1, page, page + 1, 40 * page, 40 * page + 1, 41 * page - 1], page=page, seed=page, pad=5)


@pytest.mark.parametrize("pages", [255, 256, 257, 511, 513, 2048, 8191, 8192, 8193, 20000])
def test_select_many_pages(B, pages):
    select_case(B, [pages * 2 - 1, pages], page=2, hkv=3, keep=100, seed=pages)


def test_select_many_requests(B):
    select_case(B, [(37 * i) % 600 for i in range(300)], hkv=4, keep=5, seed=1)


def test_select_equal_and_special_scores(B):
    """Equal scores, zeros of both signs, infinities, NaN, neighbours in the last bit, a wide range."""
    n, page = 600, 1
    same = torch.full((1, 1, n), 3.0, device="cuda")
    for keep in (1, 7, 599):
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=0, scores=same)
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=0, scores=same * -math.inf)
        zeros = torch.where(torch.arange(n, device="cuda") % 3 == 0, 0.0, -0.0).view(1, 1, n)
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=1 if keep > 1 else 0, scores=zeros)
        last = (torch.arange(n, device="cuda", dtype=torch.int32) * 7919 % n + 0x41200000).view(torch.float32).view(1, 1, n)
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=0, scores=last)
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=0, scores=-last)
        wide = torch.randint(-2**31, 2**31 - 1, (1, 1, n), generator=gen(keep), device="cuda", dtype=torch.int32).view(torch.float32)
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=0, scores=wide)
        mixed = wide.clone()
        mixed[0, 0, ::5], mixed[0, 0, 1::5], mixed[0, 0, 2::5] = math.inf, math.nan, -math.inf
        select_case(B, [n], hkv=1, page=page, keep=keep, sinks=0, recent=0, scores=mixed)


def test_no_pages_in_the_table(B):
    """Tables without a column: no pages, and lengths that pass them."""
    tables, lens = torch.zeros(2, 3, 4, **INT), torch.ones(2, 3, **INT)
    B.moe_page_select(torch.empty(2, 3, 0, device="cuda"), torch.empty(2, 0, **INT), torch.tensor([5, 0], **INT), 16, tables, lens)
    assert (tables == -1).all() and (lens == 0).all()
    k, v, _, _, cache = make_cache(B, gen(0), 2, 16, 3, 64, "bf16")
    q, seq, status = normal(gen(1), 2, 3, 64), torch.tensor([5, 0], **INT), torch.zeros(1, **INT)
    bounds = B.new_page_bounds(cache).fill_(3.0)
    B.moe_page_bounds(cache, bounds, torch.empty(2, 0, **INT), seq, status=status)
    assert (bounds == 3.0).all() and status.item() == -6
    status.zero_()
    B.moe_page_scores(q, cache, bounds, torch.empty(2, 0, **INT), seq, torch.empty(2, 3, 0, device="cuda"), status=status)
    assert status.item() == -6
    out, ws = torch.ones_like(q), B.new_attn_workspace(2, 3, 3, 64)
    B.moe_attn_pages(q, cache, torch.empty(2, 3, 0, **INT), lens, 0.125, out, ws)
    assert (out == 0).all() and B.moe_read_status(ws)[0] == 0


def test_select_lengths_near_the_limit_of_int(B):
    """Pages of 2^30 slots: two of them hold 2^31 - 1 tokens, and nothing overflows."""
    select_case(B, [2**31 - 1, 2**30 + 1, 2**30], page=2**30, keep=1, sinks=0, recent=1)
    select_case(B, [2**31 - 1], page=2**30, keep=2, sinks=0, recent=0)


# --------------------------------------------------------------------- attention


def pages_case(B, counts, hq, hkv, D=128, page=16, q="bf16", dtype="bf16", out=None, heads_first=False, softcap=0.0, seed=0,
               lse=True, pad=0, pages=40):
    """counts[b][g]: slots that the heads of g attend to, in pages drawn for that head."""
    g = gen(seed)
    nb = len(counts)
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype, heads_first)
    width = max(max(-(-n // page) for row in counts for n in row), 1) + pad
    tables = torch.full((nb, hkv, width), -12345, dtype=torch.int32)
    for b in range(nb):
        for h in range(hkv):
            need = -(-max(counts[b][h], 0) // page)
            tables[b, h, :need] = torch.randint(0, pages, (need,), generator=g, device="cuda", dtype=torch.int32).cpu()
    tables = tables.cuda()
    lens = torch.tensor(counts, **INT)
    qt = normal(g, nb, hq, D, std=1.5, dtype=DT[q])
    ot = torch.full((nb, hq, D), 7.0, dtype=DT[out or q], device="cuda")
    lt = torch.empty(nb, hq, device="cuda") if lse else None
    ws = B.new_attn_workspace(nb, hq, hkv, D)
    scale, group = D ** -0.5, hq // hkv

    def go():
        B.moe_attn_pages(qt, cache, tables, lens, scale, ot, ws, softcap=softcap, lse=lt)

    go()
    torch.cuda.synchronize()
    assert B.moe_read_status(ws)[0] == 0
    for b in range(nb):
        for h in range(hkv):
            n, own = max(counts[b][h], 0), slice(h * group, (h + 1) * group)
            rk, rv = (O.cached_rows(c, s, tables[b, h], 0, n)[:, h:h + 1] for c, s in ((k, ks), (v, vs)))
            want, wl = O.decode_attention(qt[b, own], (rk, rv), scale, softcap)
            top = rv.abs().max().item() if n else 0.0
            bound = 1e-4 * top + (1.01 * BF * want.abs() if ot.dtype == torch.bfloat16 else 0.0)
            assert_within(ot[b, own], want, bound, f"request {b}, head {h}, {n} keys")
            if lse and n == 0:
                assert lt[b, own].eq(-math.inf).all()
            elif lse:
                assert_within(lt[b, own], wl, 1e-4 + 4 * U * wl.abs(), f"lse of request {b}, head {h}")
    return go, ot, lt


RAGGED = [[0, 1], [2, 15], [16, 17], [31, 100], [129, 0], [640, 33], [0, 0], [1, 1]]


@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads_first", [False, True])
def test_attn_pages_lengths(B, q, dtype, heads_first):
    pages_case(B, RAGGED, 8, 2, q=q, dtype=dtype, heads_first=heads_first, seed=1)
    pages_case(B, [[0, 0]], 8, 2, q=q, dtype=dtype, seed=2)
    pages_case(B, [[5]], 1, 1, D=64, q=q, dtype=dtype, seed=2)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_pages_head_dims(B, D, dtype):
    pages_case(B, RAGGED, 8, 2, D=D, dtype=dtype, seed=D)
    pages_case(B, RAGGED, 8, 2, D=D, dtype=dtype, q="f32", seed=D)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (7, 1), (9, 1), (16, 1), (17, 1), (40, 2), (6, 6), (56, 8)])
@pytest.mark.parametrize("q", ["f32", "bf16"])
def test_attn_pages_head_groups(B, hq, hkv, q):
    pages_case(B, [[(83 * h + 17 * b) % 300 for h in range(hkv)] for b in range(3)], hq, hkv, q=q, seed=hq)


@pytest.mark.parametrize("page", [1, 3, 24, 64, 100])
def test_attn_pages_page_sizes(B, page):
    pages_case(B, [[20 * page, page], [page - 1, 3 * page + 1]], 8, 2, page=page, seed=page, pad=2)


@pytest.mark.parametrize("softcap", [1.0, 30.0, 300.0])
def test_attn_pages_softcap(B, softcap):
    pages_case(B, RAGGED, 8, 2, softcap=softcap, dtype="e4m3", seed=3)
    pages_case(B, RAGGED, 8, 2, softcap=softcap, q="f32", seed=3, lse=False)


@pytest.mark.parametrize("counts,hq,hkv", [([[20000, 1]], 8, 2), ([[300] * 8] * 60, 16, 8), ([[0, 9000, 5]] * 4, 6, 3),
                                           ([[64] * 2] * 300, 4, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_pages_long_and_many(B, counts, hq, hkv, dtype):
    pages_case(B, counts, hq, hkv, D=64, dtype=dtype, pages=200, seed=4)


@pytest.mark.parametrize("dtype,q", [("bf16", "bf16"), ("e4m3", "bf16"), ("bf16", "f32")])
def test_attn_pages_mixes_of_short_and_long(B, dtype, q):
    """Lists that a CTA takes whole next to lists that several share, cut at many places: 30 mixes, each twice over one
    workspace (the counters are zero again)."""
    host = torch.Generator()
    host.manual_seed(30)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=host))

    g = gen(30)
    D, page, pages, hkv = 64, 16, 300, 2
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype)
    kd, vd = ((O.f64(c) * (O.f64(s)[:, None] if s is not None else 1.0)).cuda() for c, s in ((k, ks), (v, vs)))
    ws = B.new_attn_workspace(64, 8, hkv, D)
    for i in range(30):
        nb = pick(1, 60)
        lens = torch.zeros(nb, hkv, dtype=torch.int32)
        for b in range(nb):
            for h in range(hkv):
                kind = pick(0, 5)
                lens[b, h] = 0 if kind == 0 else pick(1, 700) if kind < 4 else pick(700, 4000)
        width = max(1, -(-int(lens.max()) // page))
        tables = torch.randint(0, pages, (nb, hkv, width), generator=g, device="cuda", dtype=torch.int32)
        lens = lens.cuda()
        qt = normal(g, nb, 8, D, std=1.5, dtype=DT[q])
        out = torch.full((nb, 8, D), 9.0, dtype=DT[q], device="cuda")
        at = torch.arange(width * page, device="cuda")
        want = torch.zeros(nb, hkv, 4, D, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            rows = tables[:, h].long()[:, at // page]
            s = torch.einsum("bgd,bld->bgl", qt.double().view(nb, hkv, 4, D)[:, h], kd[rows, at % page, h]) * 0.125
            seen = (at < lens[:, h, None])[:, None]
            s = torch.where(seen, s, -math.inf)
            p = torch.nan_to_num(torch.softmax(s, -1))
            want[:, h] = torch.einsum("bgl,bld->bgd", p, vd[rows, at % page, h])
        for _ in range(2):
            B.moe_attn_pages(qt, cache, tables, lens, 0.125, out, ws)
            bound = 1e-4 * vd.abs().max().item() + (1.01 * BF * want.abs() if q == "bf16" else 0.0)
            assert ((out.double().view_as(want) - want).abs() <= bound).all(), f"mix {i}"
    assert B.moe_read_status(ws)[0] == 0


def test_attn_pages_equal_calls_give_equal_bits(B):
    go, ot, lt = pages_case(B, [[5000, 700], [0, 3], [999, 4000]], 8, 2, q="f32", seed=5)
    first = ot.clone(), lt.clone()
    for _ in range(3):
        ot.zero_()
        go()
        assert torch.equal(ot, first[0]) and torch.equal(lt, first[1])


def test_attn_pages_output_types_and_strides(B):
    pages_case(B, RAGGED, 8, 2, q="bf16", out="f32", seed=6)
    pages_case(B, RAGGED, 8, 2, q="f32", out="bf16", seed=6)
    g = gen(7)
    k, v, _, _, cache = make_cache(B, g, 8, 16, 2, 64, "bf16")
    q = normal(g, 2, 9, 72, dtype=torch.bfloat16)[:, 1:5, 8:]
    out = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    tables, lens = torch.arange(8, **INT).view(2, 2, 2), torch.tensor([[32, 17], [1, 30]], **INT)
    B.moe_attn_pages(q, cache, tables, lens, 0.125, out, B.new_attn_workspace(5, 4, 2, 64))
    for b in range(2):
        for h in range(2):
            rk, rv = (O.cached_rows(c, None, tables[b, h], 0, int(lens[b, h]))[:, h:h + 1] for c in (k, v))
            want, _ = O.decode_attention(q[b, 2 * h:2 * h + 2], (rk, rv), 0.125)
            assert_within(out[b, 2 * h:2 * h + 2], want, 4e-4 + 1.01 * BF * want.abs(), f"{b}, {h}")


def test_attn_pages_as_attn_decode(B):
    """With every head's table the request's, and one workspace for both calls: the same up to the order of joins."""
    g = gen(8)
    lens = [700, 0, 33]
    table, pages = make_table(g, lens, 16)
    k, v, _, _, cache = make_cache(B, g, pages, 16, 4, 64, "bf16")
    q, ws = normal(g, 3, 8, 64), B.new_attn_workspace(3, 8, 4, 64)
    seq, a, b = torch.tensor(lens, **INT), torch.empty(3, 8, 64, device="cuda"), torch.empty(3, 8, 64, device="cuda")
    tables, each = table[:, None].expand(3, 4, -1).contiguous(), seq[:, None].expand(3, 4).contiguous()
    for _ in range(2):
        B.moe_attn_decode(q, cache, table, seq, 0.125, a, ws)
        B.moe_attn_pages(q, cache, tables, each, 0.125, b, ws)
        assert (a - b).abs().max() < 1e-5
    assert B.moe_read_status(ws)[0] == 0


def test_attn_pages_reports_what_it_cannot_read(B):
    g = gen(10)
    k, v, _, _, cache = make_cache(B, g, 8, 16, 2, 64, "bf16")
    q = normal(g, 1, 2, 64)
    for bad in ("length", "page_high", "page_negative"):
        tables, lens = torch.arange(8, **INT).view(1, 2, 4), torch.tensor([[64, 64]], **INT)
        left = list(range(64))
        if bad == "length":
            lens[0, 1] = 2_000_000_000
        else:
            tables[0, 1, 2] = 8 if bad == "page_high" else -3
            left = [i for i in left if i // 16 != 2]
        ws, o = B.new_attn_workspace(1, 2, 2, 64), torch.empty_like(q)
        B.moe_attn_pages(q, cache, tables, lens, 0.125, o, ws)
        torch.cuda.synchronize()
        assert B.moe_read_status(ws)[0] == -6
        for h, rows in ((0, list(range(64))), (1, left)):
            fk, fv = (torch.cat([O.f64(c[p, :, h:h + 1]) for p in range(4 * h, 4 * h + 4)])[rows] for c in (k, v))
            want, _ = O.decode_attention(q[0, h:h + 1], (fk, fv), 0.125)
            assert_within(o[0, h:h + 1], want, 4e-4, f"{bad}, head {h}")


# ----------------------------------------------------------------------- together


def chain(B, dtype="bf16", T=5, seed=0, prompt=180):
    """Buffers, and one decode step's calls: append, bounds, scores, selection, attention."""
    g = gen(seed)
    hq, hkv, D, page, keep = 8, 2, 64, 16, 4
    lens = [(prompt - 41 * i) % prompt + 1 for i in range(T)]
    table, pages = make_table(g, [n + 1 for n in lens], page)
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype)
    qkv = normal(g, T, hq + 2 * hkv, D, dtype=torch.bfloat16)
    pos, seq = torch.tensor(lens, **INT), torch.tensor(lens, **INT) + 1
    bounds, ws = B.new_page_bounds(cache), B.new_attn_workspace(T, hq, hkv, D)
    B.moe_page_bounds(cache, bounds, table, pos)                    # of the prompt
    w = [(1 + 0.2 * normal(g, D)).to(torch.bfloat16) for _ in range(2)]
    q, out = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    scores = torch.full((T, hkv, table.shape[1]), -math.inf, device="cuda")
    tables, kept = torch.empty(T, hkv, keep, **INT), torch.empty(T, hkv, **INT)
    cs = cos_sin_table(prompt + 2, D)

    def step():
        B.moe_qk_norm_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], w[0], w[1], 1e-6, cache, table, pos, q,
                             cos_sin=cs)
        B.moe_page_bounds(cache, bounds, table, seq, first=pos)
        B.moe_page_scores(q, cache, bounds, table, seq, scores)
        B.moe_page_select(scores, table, seq, page, tables, kept, sinks=1, recent=1)
        B.moe_attn_pages(q, cache, tables, kept, D ** -0.5, out, ws)

    return dict(step=step, q=q, out=out, scores=scores, tables=tables, kept=kept, bounds=bounds, k=k, v=v, ks=ks, vs=vs,
                table=table, seq=seq, page=page, keep=keep, hq=hq, hkv=hkv, D=D, qkv=qkv, w=w, cs=cs, pos=pos, ws=ws, cache=cache)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_step_of_all_calls(B, dtype):
    """The calls one after another, each against the oracle on what the one before it left."""
    c = chain(B, dtype)
    c["step"]()
    torch.cuda.synchronize()
    qr = O.rotate(O.qk_norm(c["qkv"][:, :c["hq"]], c["w"][0], 1e-6), c["pos"], c["cs"])
    assert_within(c["q"], qr, 1e-4 + 1.01 * BF * qr.abs(), "q")
    group = c["hq"] // c["hkv"]
    for b, n in enumerate(c["seq"].tolist()):
        rows = O.cached_rows(c["k"], None, c["table"][b], 0, n)
        edges = O.page_bounds(rows, c["page"], 0, n)
        at = c["table"][b, :len(edges)].long()
        got = O.f64(c["bounds"])[at.cpu()]
        lo, hi = torch.stack([edges[j][0] for j in edges]), torch.stack([edges[j][1] for j in edges])
        assert torch.equal(got[:, :, 0], lo) and torch.equal(got[:, :, 1], hi)
        if c["ks"] is not None:
            lo, hi = lo * O.f64(c["ks"])[:, None], hi * O.f64(c["ks"])[:, None]
        want, size = O.page_scores(c["q"][b], lo, hi)
        assert_within(c["scores"][b, :, :len(edges)], want, 30 * U * size + 1e-4, "scores")
        for h in range(c["hkv"]):
            cols = O.page_select(c["scores"][b, h].tolist(), len(edges), c["keep"], 1, 1)
            assert c["tables"][b, h].tolist() == [int(c["table"][b, j]) for j in cols] + [-1] * (c["keep"] - len(cols))
            m = int(c["kept"][b, h])
            own = slice(h * group, (h + 1) * group)
            rk, rv = (O.cached_rows(x, s, c["tables"][b, h], 0, m)[:, h:h + 1] for x, s in ((c["k"], c["ks"]), (c["v"], c["vs"])))
            o, _ = O.decode_attention(c["q"][b, own], (rk, rv), c["D"] ** -0.5)
            assert_within(c["out"][b, own], o, 1e-4 * rv.abs().max().item() + 1.01 * BF * o.abs(), f"{b}, {h}")


def test_a_step_on_another_stream_and_in_graphs(B):
    """On a side stream, captured and replayed, and two captured steps in turn: the bits of the eager run."""
    c, d = chain(B, seed=1), chain(B, "e4m3", T=9, seed=2)
    names = ("q", "out", "scores", "tables", "kept", "bounds", "k")
    want = []
    for x in (c, d):
        x["step"]()
        torch.cuda.synchronize()
        want.append([raw(x[n]).clone() if x[n].dtype.itemsize < 4 else x[n].clone() for n in names])

    def check():
        torch.cuda.synchronize()
        for x, w in ((c, want[0]), (d, want[1])):
            for n, t in zip(names, w):
                assert torch.equal(raw(x[n]) if x[n].dtype.itemsize < 4 else x[n], t), n
                if n in ("q", "out", "tables", "kept"):
                    x[n].zero_()

    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c["step"]()
        d["step"]()
    check()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, x in zip(graphs, (c, d)):
        with torch.cuda.graph(graph):
            x["step"]()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        check()


def test_padding_in_a_step(B):
    """A slot of the batch without a request: position -1, length 0; the others are as without it."""
    c = chain(B, T=4, seed=7)
    c["step"]()
    torch.cuda.synchronize()
    want = {n: c[n].clone() for n in ("out", "tables", "kept")}
    c["pos"][1], c["seq"][1] = -1, 0
    for n in want:
        c[n].fill_(5)
    c["step"]()
    torch.cuda.synchronize()
    assert (c["out"][1] == 0).all() and (c["tables"][1] == -1).all() and (c["kept"][1] == 0).all()
    for n, t in want.items():
        for b in (0, 2, 3):
            assert torch.equal(c[n][b], t[b])
    c["seq"][2], c["pos"][2] = -3, -1             # a negative length is none
    c["step"]()
    torch.cuda.synchronize()
    assert (c["out"][2] == 0).all() and torch.equal(c["out"][3], want["out"][3])


def test_steps_on_two_streams_at_once(B):
    cs = [chain(B, seed=8), chain(B, "e4m3", T=9, seed=9, prompt=700)]
    want = []
    for c in cs:
        c["step"]()
        torch.cuda.synchronize()
        want.append([c[n].clone() for n in ("q", "out", "tables", "kept")])
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                c["step"]()
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        for n, t in zip(("q", "out", "tables", "kept"), w):
            assert torch.equal(c[n], t), n


def test_scores_of_infinite_values(B):
    """An infinite query or bound makes its own head's or page's scores infinite or NaN, and no other."""
    for dtype in ("bf16", "e4m3"):
        g = gen(24)
        k, v, ks, vs, cache = make_cache(B, g, 4, 16, 2, 64, dtype)
        bounds = B.new_page_bounds(cache)
        table, seq = torch.tensor([[0, 1, 2, 3]], **INT), torch.tensor([64], **INT)
        B.moe_page_bounds(cache, bounds, table, seq)
        q, scores = normal(g, 1, 4, 64), torch.zeros(1, 2, 4, device="cuda")
        if dtype == "bf16":
            bounds[2, 0, 1, 7] = math.inf
        q[0, 3, 5] = -math.inf
        B.moe_page_scores(q, cache, bounds, table, seq, scores)
        assert not torch.isfinite(scores[0, 1]).any()
        assert torch.isfinite(scores[0, 0]).tolist() == [True, True, dtype == "e4m3", True]


# ------------------------------------------------------------------ far and odd places


def test_far_pages(B):
    """Pages whose offset passes 2^32 elements: append, bounds and attention."""
    D, page = 64, 16
    stride = 1 << 28
    buf = torch.zeros((17 * stride + page * D,), dtype=torch.uint8, device="cuda")
    k = buf.view(torch.float8_e4m3fn).as_strided((18, page, 1, D), (stride, D, D, 1))
    s = torch.ones(1, device="cuda")
    cache = B.KvCache(k, k, s, s)
    g = gen(20)
    rows, table, req = normal(g, 2, 1, D), torch.tensor([[17]], **INT), torch.zeros(2, **INT)
    B.moe_qk_norm_append(None, rows, rows, None, None, 1e-6, cache, table, torch.tensor([0, 1], **INT), None, req=req)
    got = O.f64(buf[17 * stride:17 * stride + 2 * D].view(torch.float8_e4m3fn)).view(2, 1, D)
    assert (got != 0).any()
    bounds = B.new_page_bounds(cache)
    B.moe_page_bounds(cache, bounds, table, torch.tensor([2], **INT))
    assert torch.equal(O.f64(bounds[17]), torch.stack([got.min(0).values, got.max(0).values], 1))
    q, o = normal(g, 1, 1, D), torch.empty(1, 1, D, device="cuda")
    B.moe_attn_pages(q, cache, table.view(1, 1, 1), torch.tensor([[2]], **INT), 0.125, o, B.new_attn_workspace(1, 1, 1, D))
    want, _ = O.decode_attention(q[0], (got, got), 0.125)
    assert_within(o[0], want, 4e-4, "far page")


def test_far_bounds(B):
    """Bounds of 2^22 pages and more, beyond 2^32 bytes; the cache is a view of one page."""
    pages, hkv, D = (1 << 22) + 8, 4, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    g = gen(21)
    k = normal(g, 1, 16, hkv, D, dtype=torch.bfloat16).expand(pages, 16, hkv, D)
    cache = B.KvCache(k, k)
    bounds = B.new_page_bounds(cache)
    table = torch.tensor([[pages - 1, 3, pages - 8]], **INT)
    seq = torch.tensor([40], **INT)
    B.moe_page_bounds(cache, bounds, table, seq)
    assert torch.equal(bounds[pages - 1, :, 0], k[0].amin(0)) and torch.equal(bounds[pages - 8, :, 1], k[0, :8].amax(0))
    q, scores = normal(g, 1, 8, D), torch.zeros(1, hkv, 3, device="cuda")
    B.moe_page_scores(q, cache, bounds, table, seq, scores)
    at = torch.tensor([pages - 1, 3, pages - 8], device="cuda")
    want, size = O.page_scores(q[0], bounds[at, :, 0], bounds[at, :, 1])
    assert_within(scores[0], want, 30 * U * size + 1e-4, "far bounds")


def test_scores_lengths_near_the_limit_of_int(B):
    """2^31 - 1 tokens in two pages of 2^30 slots, of a cache that is a view of one row."""
    k = normal(gen(22), 1, 1, 2, 64, dtype=torch.bfloat16).expand(3, 2**30, 2, 64)
    cache = B.KvCache(k, k)
    bounds = torch.stack([k[:, 0], k[:, 0]], 2).contiguous()
    q, scores = normal(gen(23), 1, 2, 64), torch.zeros(1, 2, 2, device="cuda")
    B.moe_page_scores(q, cache, bounds, torch.tensor([[2, 0]], **INT), torch.tensor([2**31 - 1], **INT), scores)
    want = (O.f64(q[0]) * O.f64(k[0, 0])).sum(1)
    assert_within(scores[0, :, 0], want, 1e-4, "first page")
    assert_within(scores[0, :, 1], want, 1e-4, "second page")


# ------------------------------------------------------------------------- example


@pytest.fixture(scope="module")
def example(B):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block_pages", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_example_block_with_selected_pages(B, example, cache):
    """Eager steps and replays of a captured one give the same bits; with every page kept, attention is that over
    the whole cache."""
    T, runs = 3, []
    for captured, keep in ((False, 3), (True, 3), (False, 10)):
        blk = example.DecodeBlock(synth.TINY_VANILLA, T, 80, 4, 2, 64, page=8, adapters=2, rank=8, cache=cache, seed=5, keep=keep)
        x, delta = torch.zeros(T, 256, device="cuda"), synth.hidden(T, 256, 2, "cuda")
        positions = torch.tensor([0, 9, 60], **INT)
        seq, adapter = positions + 1, torch.tensor([1, -1, 0], **INT)
        g = gen(1)
        for c in blk.cache.tensors[:2]:
            c.copy_(normal(g, *c.shape, std=0.5).to(c.dtype))
        blk.prompt(positions)

        def one():
            blk.step(delta, x, positions, seq, adapter)
            positions.add_(1)
            seq.add_(1)

        step = one
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
            step = graph.replay
        for i in range(5):
            step()
        torch.cuda.synchronize()
        assert blk.status() == 0
        runs.append((blk.attn.clone(), blk.tables.clone(), blk.lens.clone()))
        if keep == 10:
            q = blk.qkv.view(T, -1, 64)[:, :4]
            out = torch.empty_like(blk.attn)
            B.moe_attn_decode(q, blk.cache, blk.block_table, seq - 1, 64 ** -0.5, out, B.new_attn_workspace(T, 4, 2, 64))
            top = O.f64(blk.cache.tensors[1]).abs().max().item() * (8 / 448 if cache == "e4m3" else 1.0)
            assert_within(blk.attn, O.f64(out), 1e-4 * top + 2.02 * BF * O.f64(out).abs(), "all pages")
    for a, b in zip(runs[0], runs[1]):
        assert torch.equal(a, b)


def test_example_runs(B):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "decode_block.py"), "--requests", "3", "--context", "500",
                        "--steps", "4", "--keep", "8"], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "8 pages of each" in r.stdout

"""moe_page_scores at the ends of fp32, and its error against a bound that its arithmetic has.

The bound, with u = 2^-24, G query heads to a key-value head, and S the sum of the absolute values of what is added up, the lower
and the upper side taken apart:
- a channel's sum of G queries of one sign: G - 1 roundings, (G - 1) u S;
- its terms: three truncated bf16 ones have its 24 bits; over an E4M3 cache a power of two brings the greatest sum to 2^14 and
  more (a greatest sum below 2^-112 by 2^126), and three f16 terms leave 2^-25: 2^-39 of the greatest sum for every channel;
- an MMA adds 16 products to a running sum.  The tensor cores cut each of the 17 to a multiple of 2^-23 of the
  greatest of them or less, possibly in two steps of 8, and cut the result: 20 cuts of 2 u of the terms' absolute sum, 40 u.
  A chain has n = D / 16 MMAs (D rounded up to 64, over bf16 to 32, then to 64, 128 or 256): 40 n u S; second and third terms are under
  2^-7 of it: 41 n u S together;
- two chains, three terms, and the scale as two factors: 5 u S.
Together (G + 41 n + 4) u S, and the terms' 2^-39.
"""

import math

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import DT, U, assert_within, gen, normal

pytestmark = pytest.mark.gpu

INT = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def mmas(D, dtype):
    """Of a chain."""
    return next(w for w in ((64, 128, 256) if dtype == "e4m3" else (32, 64, 128, 256)) if D <= w) // 16


def run(B, q, bounds, scale, dtype):
    """(scores, 64-bit scores, bound on their difference) [hkv, pages] of one request with a page of one slot for each of bounds."""
    pages, hkv, _, D = bounds.shape
    k = torch.zeros(pages, 1, hkv, D, dtype=DT[dtype], device="cuda")
    cache = B.KvCache(k, k, scale, scale)
    scores, status = torch.full((1, hkv, pages), 77.0, device="cuda"), torch.zeros(1, **INT)
    B.moe_page_scores(q, cache, bounds, torch.arange(pages, **INT).view(1, -1), torch.tensor([pages], **INT), scores, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    s = O.f64(scale)[:, None] if scale is not None else 1.0
    lo, hi = (O.f64(bounds[:, :, i]) * s for i in (0, 1))
    want, _ = O.page_scores(q[0], lo, hi)
    G = q.shape[1] // hkv
    qd = O.f64(q[0]).view(hkv, G, D)
    below, above = qd.clamp(max=0).sum(1).abs(), qd.clamp(min=0).sum(1)
    size = (below[None] * lo.abs() + above[None] * hi.abs()).sum(2).T
    most = torch.maximum(below, above).amax(1).clamp(min=2.0 ** -112)
    left = 2.0 ** -39 * most[:, None] * (lo.abs() + hi.abs()).sum(2).T if dtype == "e4m3" else 0.0
    # where a result or the one before it is below the normal numbers, half of their last step
    return scores[0], want, (G + 41 * mmas(D, dtype) + 4) * U * size + left + 2.0 ** -149


def edges(g, pages, hkv, D, dtype, mid=1.0, wide=1.0):
    m, w = mid * normal(g, pages, hkv, D), wide * normal(g, pages, hkv, D).abs()
    e = torch.stack([m - w, m + w], 2)
    return (e * 100).clamp(-448, 448).to(DT[dtype]) if dtype == "e4m3" else e.to(DT[dtype])


@pytest.mark.parametrize("D", [16, 32, 48, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (14, 2), (40, 1)])
def test_scores_within_what_their_arithmetic_has(B, D, dtype, q, hq, hkv):
    """Bounds of both signs, and of one: all terms alike in sign, and terms that cancel."""
    g = gen(D + hq)
    scale = (0.5 + torch.rand(hkv, generator=g, device="cuda")) / 100 if dtype == "e4m3" else None
    for mid, wide in ((1.0, 1.0), (0.1, 2.0), (3.0, 0.01)):
        qt = normal(g, 1, hq, D, std=1.5, dtype=DT[q])
        got, want, bound = run(B, qt, edges(g, 300, hkv, D, dtype, mid, wide), scale, dtype)
        assert_within(got, want, bound, f"mid {mid}, wide {wide}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_exp,scale_exp", [(0, -122), (0, -125), (-100, -6), (-116, -6), (-125, -3), (-60, -60), (100, -100),
                                             (-100, 100), (-110, 0), (60, 30)])
def test_scores_of_small_scales_and_queries(B, D, q_exp, scale_exp):
    """Queries and scales of E4M3 keys whose product with a power of two is below the normal numbers, though the scores are not."""
    g = gen(D)
    scale = (1 + torch.rand(2, generator=g, device="cuda")) * 2.0 ** scale_exp
    qt = normal(g, 1, 6, D).clamp(-4, 4) * 2.0 ** q_exp
    got, want, bound = run(B, qt, edges(g, 50, 2, D, "e4m3"), scale, "e4m3")
    assert_within(got, want, bound, f"2^{q_exp}, 2^{scale_exp}")


def test_scores_of_zero_bounds_beside_infinite_ones(B):
    """A page of zeros scores 0 where others pass fp32's range."""
    g = gen(3)
    bounds = edges(g, 40, 2, 64, "e4m3", 0.1, 3.0)
    bounds.view(torch.uint8)[7] = 0
    scale = torch.full((2,), 2.0 ** 120, device="cuda")
    got, _, _ = run(B, normal(g, 1, 4, 64) * 2.0 ** 30, bounds, scale, "e4m3")
    assert (got[:, 7] == 0).all()
    assert got[:, :7].eq(math.inf).all() and got[:, 8:].eq(math.inf).all()


def test_scores_of_no_query(B):
    """Queries of 0 (a padded slot): every page scores 0."""
    for dtype in ("bf16", "e4m3"):
        g = gen(4)
        scale = torch.full((2,), 0.01, device="cuda") if dtype == "e4m3" else None
        got, _, _ = run(B, torch.zeros(1, 4, 64, device="cuda"), edges(g, 40, 2, 64, dtype), scale, dtype)
        assert (got == 0).all()

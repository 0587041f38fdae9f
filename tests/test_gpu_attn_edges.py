"""Attention over the paged cache at the ends of its range, against the fp64 oracle: NaN and infinite
queries, keys and values, large caps, queries and scales far from 1, lengths near 2^31, and the digits that
fp32 queries and outputs keep."""

import math

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import BF, DT, U, assert_within, attn_case, gen, make_cache, normal, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


class One:
    """One request of n keys, pages in order; `run` returns (out, lse) and `want` the oracle's."""

    def __init__(self, B, n, hq, hkv, D, q="bf16", dtype="bf16", seed=0, page=16):
        self.B, self.n, self.hq = B, n, hq
        g = gen(seed)
        pages = (n + page - 1) // page
        self.k, self.v, self.ks, self.vs, self.cache = make_cache(B, g, pages, page, hkv, D, dtype)
        self.table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, pages)
        self.q = normal(g, 1, hq, D, dtype=DT[q])
        self.page, self.D = page, D

    def put(self, t, key, head, dim, value):
        raw(t)[key // self.page, key % self.page, head, dim] = raw(torch.tensor([value]).to(t.dtype))[0].item()

    def run(self, softcap=0.0, scale=None, out=None):
        o = torch.empty(self.q.shape, dtype=DT[out] if out else self.q.dtype, device="cuda")
        lse = torch.empty(1, self.hq, device="cuda")
        ws = self.B.new_attn_workspace(1, self.hq, self.k.shape[2], self.D)
        self.scale = self.D ** -0.5 if scale is None else scale
        self.B.moe_attn_decode(self.q, self.cache, self.table, torch.tensor([self.n], dtype=torch.int32, device="cuda"),
                               self.scale, o, ws, softcap=softcap, lse=lse)
        torch.cuda.synchronize()
        assert self.B.moe_read_status(ws)[0] == 0
        return o[0], lse[0]

    def rows(self):
        return (O.cached_rows(self.k, self.ks, self.table[0], 0, self.n),
                O.cached_rows(self.v, self.vs, self.table[0], 0, self.n))

    def want(self, softcap=0.0):
        return O.decode_attention(self.q[0], self.rows(), self.scale, softcap)


def bound_of(want, out_dtype, top):
    return 1e-4 * top + (1.01 * BF * want.abs() if out_dtype == torch.bfloat16 else 0.0)


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("q", ["bf16", "f32"])
def test_attn_nan_queries_and_keys(B, q, hq, dtype, softcap):
    """A NaN in a query spoils its own head, one in a key all heads of its key-value head, with a cap or without."""
    for n in (100, 3000):
        c = One(B, n, 2 * hq, 2, 64, q, dtype, seed=n)
        c.q[0, 1, 7] = math.nan
        o, lse = c.run(softcap)
        want, _ = c.want(softcap)
        bad = torch.zeros(2 * hq, dtype=torch.bool)
        bad[1] = True
        assert torch.isnan(o[1]).all() and torch.isnan(lse[1])
        top = c.rows()[1].abs().max().item()
        assert_within(o.cpu()[~bad], want[~bad], bound_of(want[~bad], o.dtype, top), "other heads")
        c.put(c.k, n // 2, 1, 9, math.nan)
        o, _ = c.run(softcap)
        want, _ = c.want(softcap)
        bad[hq:] = True
        assert torch.isnan(o[hq:]).all()
        assert_within(o.cpu()[~bad], want[~bad], bound_of(want[~bad], o.dtype, top), "the other key-value head")


@pytest.mark.parametrize("hq", [4, 16])
def test_attn_infinite_bf16_queries(B, hq):
    """Over a bf16 cache the scores are infinite (+-cap with a cap); over an E4M3 cache the head gets NaN."""
    for dtype in ("bf16", "e4m3"):
        c = One(B, 200, hq, 1, 64, "bf16", dtype, seed=hq)
        c.q[0, 2, 3] = math.inf
        for i in range(200):      # no zero beside the infinity
            c.put(c.k, i, 0, 3, 1.0 if i % 3 else -1.0)
        others = [h for h in range(hq) if h != 2]
        for cap in (0.0, 30.0):
            o, _ = c.run(cap)
            want, _ = c.want(cap)
            assert_within(o[others], want[others], bound_of(want[others], o.dtype, c.rows()[1].abs().max().item()), "others")
            if dtype == "e4m3" or cap == 0.0:
                assert torch.isnan(o[2]).all()
            else:
                assert_within(o[2], want[2], bound_of(want[2], o.dtype, 4.0), "capped")


@pytest.mark.parametrize("softcap", [300.0, 1e5])
@pytest.mark.parametrize("q,dtype", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "bf16")])
@pytest.mark.parametrize("hq", [8, 32])
def test_attn_large_softcap(B, softcap, q, dtype, hq):
    attn_case(B, [1, 64, 300, 3000], hq, 2, 128, 32, q=q, dtype=dtype, softcap=softcap, seed=9)


@pytest.mark.parametrize("q,out", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("hq", [4, 16])
def test_attn_infinite_values(B, q, out, hq):
    """An infinite cached value makes its column infinite and leaves the others alone."""
    for n in (5, 100, 3000):
        c = One(B, n, 2 * hq, 2, 64, q, "bf16", seed=n)
        c.put(c.v, n // 2, 1, 9, math.inf)
        c.put(c.v, n - 1, 1, 40, -math.inf)
        o, _ = c.run(out=out)
        want, _ = c.want()
        assert torch.equal(torch.isinf(want), torch.isinf(o.cpu())), "infinities"
        at = torch.isinf(want)
        assert torch.equal(O.f64(o)[at], want[at])
        rest = torch.where(at, torch.zeros_like(want), want)
        assert_within(torch.where(at, torch.zeros_like(want), O.f64(o)), rest, bound_of(rest, o.dtype, 5.0), "the others")


@pytest.mark.parametrize("q", ["bf16", "f32"])
@pytest.mark.parametrize("power", [-116, -110, 110, 122])
def test_attn_e4m3_queries_far_from_one(B, q, power):
    """q of 2^power over keys whose scale is 2^-power."""
    c = One(B, 200, 4, 1, 64, q, "e4m3", seed=3)
    c.q.mul_(2.0 ** power)
    c.ks.mul_(2.0 ** -power)
    o, lse = c.run()
    want, wl = c.want()
    assert_within(o[:], want, bound_of(want, o.dtype, c.rows()[1].abs().max().item()), "out")
    assert_within(lse, wl, 1e-4 + 4 * U * wl.abs(), "lse")


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_lengths_near_the_limit_of_int(B, window, dtype):
    """2^31 - 1 keys, all in one row of memory (a page whose slots have stride 0)."""
    n, D = 2 ** 31 - 1, 16
    g = gen(5)
    row = normal(g, 1, D).to(DT[dtype])
    kv = row.view(torch.uint8 if dtype == "e4m3" else torch.int16).as_strided((1, n, 1, D), (D, 0, D, 1)).view(DT[dtype])
    s = torch.full((1,), 0.5, device="cuda") if dtype == "e4m3" else None
    cache = B.KvCache(kv, kv, s, s)
    q, o = normal(g, 1, 2, D, dtype=torch.bfloat16), torch.empty(1, 2, D, device="cuda")
    lse, ws = torch.empty(1, 2, device="cuda"), B.new_attn_workspace(1, 2, 1, D)
    table, seq = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32, device="cuda")
    B.moe_attn_decode(q, cache, table, seq, 0.25, o, ws, window=window, lse=lse)
    torch.cuda.synchronize()
    assert B.moe_read_status(ws)[0] == 0
    v = O.f64(row)[0] * (0.5 if s is not None else 1.0)
    # a warp adds up 2^31 / 1216 equal weights in tiles of 32 (one addition to o, four to a thread's part of
    # the sum), each rounded to 2^-24
    tol = 5 * 2 ** 31 / 1216 / 32 * U if not window else 1e-5
    assert_within(o[0], v.expand(2, D), tol * v.abs().expand(2, D) + 1e-30, "out")
    score = (O.f64(q)[0] @ v) * 0.25
    want = score + math.log(window or n)
    assert_within(lse[0], want, 1e-4 + tol, "lse")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_fp32_keeps_its_digits(B, dtype):
    """fp32 queries and outputs keep 22 bits.  A score of one key is the logarithm of its sum: one product
    (2^-22), a scale or two and the change of base and back (with 7 added to it and taken off again), under 16
    roundings of 2^-24.  And with scores of one product each, up to 1, over positive values: 2^-22 for q's
    terms and for the exponential, 2^-23 for p's, 4 cuts of 2^-23 in a tile's sum, and 2^-24 for each of 6
    roundings of the score, 8 tiles, 8 parts and 8 terms of the sum of weights: 48 2^-24, under 2^-18
    (weights of 16 bits, truncated, would be off by 2^-17 on average)."""
    c = One(B, 1, 4, 1, 64, "f32", dtype, seed=1)
    c.q.mul_(4.0)
    raw(c.k).zero_()
    c.put(c.k, 0, 0, 5, 1.625)
    _, lse = c.run(scale=3.7 / (c.ks[0].item() if c.ks is not None else 1.0))
    _, wl = c.want()
    assert_within(lse, wl, 16 * U * (wl.abs() + 7), "score")
    c = One(B, 900, 4, 1, 64, "f32", dtype, seed=2)
    c.q.uniform_(-1.0, 1.0, generator=gen(4))
    k5, v = raw(c.k)[..., 5].clone(), c.v.float().abs()
    raw(c.k).zero_()
    raw(c.k)[..., 5] = k5
    c.v.copy_(v.to(c.v.dtype))
    kmax = c.rows()[0].abs().max().item()
    o, lse = c.run(scale=1.0 / kmax)
    want, wl = c.want()
    assert (want > 0).all()
    assert_within(o, want, 2.0 ** -18 * want, "out")


def test_attn_views_with_a_size_of_one(B):
    """The stride of a dimension of size one means nothing."""
    g = gen(6)
    # one request out of a wider, odd row; one head of an odd number of elements in between
    wide = normal(g, 4 * 64 + 3, dtype=torch.bfloat16)
    for q in (wide[:256].as_strided((1, 4, 64), (259, 64, 1)), normal(g, 3, 1, 64, dtype=torch.bfloat16).as_strided((3, 1, 64), (64, 77, 1))):
        nb, hq, _ = q.shape
        kb, vb = normal(g, 8, 16, 1, 64, dtype=torch.bfloat16), normal(g, 8, 16, 1, 64, dtype=torch.bfloat16)
        odd = [t.as_strided((8, 16, 1, 64), (16 * 64, 64, 13, 1)) for t in (kb, vb)]
        cache = B.KvCache(*odd)
        table = torch.arange(2 * nb, dtype=torch.int32, device="cuda").view(nb, 2)
        seq = torch.full((nb,), 27, dtype=torch.int32, device="cuda")
        o = torch.empty(nb * hq * 64 + 8, dtype=torch.bfloat16, device="cuda")[:nb * hq * 64].as_strided(q.shape, q.stride())
        B.moe_attn_decode(q, cache, table, seq, 0.125, o, B.new_attn_workspace(nb, hq, 1, 64))
        for b in range(nb):
            rk, rv = (O.cached_rows(t, None, table[b], 0, 27) for t in (kb, vb))
            want, _ = O.decode_attention(q[b], (rk, rv), 0.125)
            assert_within(o[b], want, bound_of(want, o.dtype, rv.abs().max().item()), f"request {b}")
    # a cache of one page, and one of pages of one slot
    for shape, strides in (((1, 16, 2, 64), (5, 128, 64, 1)), ((16, 1, 2, 64), (128, 3, 64, 1))):
        kb, vb = normal(g, 16 * 128, dtype=torch.bfloat16), normal(g, 16 * 128, dtype=torch.bfloat16)
        k, v = kb.as_strided(shape, strides), vb.as_strided(shape, strides)
        table = torch.arange(shape[0], dtype=torch.int32, device="cuda").view(1, -1)
        q, o = normal(g, 1, 2, 64), torch.empty(1, 2, 64, device="cuda")
        B.moe_attn_decode(q, B.KvCache(k, v), table, torch.tensor([11], dtype=torch.int32, device="cuda"), 0.125, o,
                          B.new_attn_workspace(1, 2, 2, 64))
        rows = [O.f64(t).view(16, 2, 64)[:11] for t in (kb, vb)]
        want, _ = O.decode_attention(q[0], rows, 0.125)
        assert_within(o[0], want, bound_of(want, o.dtype, rows[1].abs().max().item()), str(shape))

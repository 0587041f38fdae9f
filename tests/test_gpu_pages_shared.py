"""Attention over pages where the heads of a key-value head are several units, divided between blocks; and the calls of a step
repeated over outputs that were overwritten before, so that a call which writes nothing shows.

Tolerances: see test_gpu_block.py.
"""

import math

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import BF, DT, gen, make_cache, normal, raw
from tests.test_gpu_pages import chain

pytestmark = pytest.mark.gpu

INT = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


class Lists:
    """A cache, a workspace for ``most`` requests of ``group`` query heads to a key-value head, and calls over lists of pages."""

    def __init__(self, B, group, D, q, dtype, most, hkv=2, pages=300, page=16, seed=0):
        self.B, self.group, self.D, self.q, self.hkv, self.pages, self.page = B, group, D, q, hkv, pages, page
        self.g = gen(seed)
        k, v, ks, vs, self.cache = make_cache(B, self.g, pages, page, hkv, D, dtype)
        self.kd, self.vd = ((O.f64(c) * (O.f64(s)[:, None] if s is not None else 1.0)).cuda() for c, s in ((k, ks), (v, vs)))
        self.ws = B.new_attn_workspace(most, group * hkv, hkv, D)

    def attend(self, lens, runs=2, dense=False, what=""):
        """lens [B, hkv] (host): ``runs`` calls, each against 64 bits; ``dense``: one over all heads' same lists in between."""
        nb, hkv, group, D, page = lens.shape[0], self.hkv, self.group, self.D, self.page
        width = max(1, -(-int(lens.max()) // page))
        tables = torch.randint(0, self.pages, (nb, 1 if dense else hkv, width), generator=self.g, device="cuda", dtype=torch.int32)
        table = tables[:, 0]
        tables = tables.expand(nb, hkv, width).contiguous()
        lens = lens.to(torch.int32).cuda()
        qt = normal(self.g, nb, hkv * group, D, std=1.5, dtype=DT[self.q])
        want = torch.zeros(nb, hkv, group, D, dtype=torch.float64, device="cuda")
        log = torch.full((nb, hkv, group), -math.inf, dtype=torch.float64, device="cuda")
        for b in range(nb):
            for h in range(hkv):
                n = int(lens[b, h])
                if n <= 0:
                    continue
                at = torch.arange(n, device="cuda")
                rows = tables[b, h].long()[at // page]
                s = qt[b].double().view(hkv, group, D)[h] @ self.kd[rows, at % page, h].T * D ** -0.5
                log[b, h] = torch.logsumexp(s, -1)
                want[b, h] = torch.exp(s - log[b, h, :, None]) @ self.vd[rows, at % page, h]
        bound = 1e-4 * self.vd.abs().max().item() + (1.01 * BF * want.abs() if self.q == "bf16" else 0.0)
        out, lse = torch.empty_like(qt), torch.empty(nb, hkv * group, device="cuda")

        def check(kind):
            off = (out.double().view_as(want) - want).abs()
            assert (off <= bound).all(), f"{what} {kind}: off by {off.max().item():.3g}"
            seen = torch.isfinite(log)
            got = lse.double().view_as(log)
            assert (got[~seen] == -math.inf).all() and ((got - log).abs()[seen] <= 1e-4 + 2.0 ** -22 * log.abs()[seen]).all(), f"{what} {kind}: lse"

        for _ in range(runs):
            if dense:
                out.fill_(9.0)
                lse.fill_(9.0)
                self.B.moe_attn_decode(qt, self.cache, table, lens[:, 0].contiguous(), D ** -0.5, out, self.ws, lse=lse)
                check("dense")
            out.fill_(9.0)
            lse.fill_(9.0)
            self.B.moe_attn_pages(qt, self.cache, tables, lens, D ** -0.5, out, self.ws, lse=lse)
            check("pages")
        assert self.B.moe_read_status(self.ws)[0] == 0


def mixes(seed, count, most, hkv=2):
    """Lengths of lists: empty, within a tile, of up to some tiles, of thousands of keys."""
    host = torch.Generator()
    host.manual_seed(seed)

    def pick(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=host))

    for _ in range(count):
        lens = torch.zeros(pick(1, most), hkv, dtype=torch.int32)
        for i in range(lens.numel()):
            kind = pick(0, 6)
            lens.view(-1)[i] = 0 if kind == 0 else pick(1, 64) if kind == 1 else pick(1, 800) if kind < 5 else pick(800, 5000)
        yield lens


@pytest.mark.parametrize("group", [9, 16, 17, 40])
@pytest.mark.parametrize("q", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_pages_divided_units_of_wide_groups(B, group, q, dtype):
    """Units that several blocks share next to units that one takes whole, several of them to a list."""
    lists = Lists(B, group, 64, q, dtype, 24, seed=group)
    for i, lens in enumerate(mixes(group, 10, 24)):
        lists.attend(lens, what=f"mix {i}")


@pytest.mark.parametrize("D,group", [(128, 17), (128, 40), (256, 3), (256, 16), (256, 20)])
@pytest.mark.parametrize("q,dtype", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_attn_pages_divided_units_of_wide_heads(B, D, group, q, dtype):
    lists = Lists(B, group, D, q, dtype, 12, seed=D + group)
    for i, lens in enumerate(mixes(D + group, 6, 12)):
        lists.attend(lens, what=f"mix {i}")


@pytest.mark.parametrize("group", [16, 17, 40])
@pytest.mark.parametrize("q", ["bf16", "f32"])
def test_attn_pages_of_more_parts_than_one_join(B, group, q):
    """Lists so long that a unit's parts are joined in groups first; each of several units to a list."""
    lists = Lists(B, group, 64, q, "bf16", 4, hkv=1, seed=group)
    lists.attend(torch.tensor([[40000]]), what="alone")
    lists.attend(torch.tensor([[130], [60001], [0], [300]]), what="between short ones")
    two = Lists(B, group, 64, q, "e4m3", 4, seed=group + 1)
    two.attend(torch.tensor([[33333, 700], [0, 45000]]), what="two long ones")


@pytest.mark.parametrize("group", [4, 17])
@pytest.mark.parametrize("q,dtype", [("f32", "bf16"), ("bf16", "e4m3")])
def test_attn_pages_and_decode_in_turn(B, group, q, dtype):
    """One workspace for both, each behind the other."""
    lists = Lists(B, group, 64, q, dtype, 20, seed=50)
    for i, lens in enumerate(mixes(51, 8, 20)):
        lists.attend(lens[:, :1].expand(-1, 2).contiguous(), dense=True, what=f"mix {i}")


@pytest.mark.parametrize("group", [4, 17])
@pytest.mark.parametrize("q,dtype", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "e4m3"), ("f32", "e4m3")])
def test_attn_pages_what_lies_behind_a_list(B, group, q, dtype):
    """NaN in the slots behind a list's last key, and no page behind its last one: neither is read."""
    g = gen(60)
    page, hkv, D = 16, 2, 64
    lens = torch.tensor([[1, 17], [16, 0], [1000, 333], [63, 64]], **INT)
    width = 70
    pages = 1 + int(((lens + page - 1) // page).sum())
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype)
    qt = normal(g, 4, hkv * group, D, dtype=DT[q])
    tables, at = torch.full((4, hkv, width), -7, **INT), 0
    for b in range(4):
        for h in range(hkv):
            n = int(lens[b, h])
            need = -(-n // page)
            tables[b, h, :need] = torch.arange(at, at + need, **INT)
            at += need
    ws, runs = B.new_attn_workspace(4, hkv * group, hkv, D), []
    for spoil in (False, True):
        if spoil:
            for b in range(4):
                for h in range(hkv):
                    n = int(lens[b, h])
                    last = int(tables[b, h, (n - 1) // page]) if n else pages - 1
                    for c in (k, v):
                        bits(c)[last, (n - 1) % page + 1 if n else 0:] = 0x7F if dtype == "e4m3" else 0x7FC0
        out = torch.full_like(qt, 9.0)
        B.moe_attn_pages(qt, cache, tables, lens, 0.125, out, ws)
        runs.append(out)
    assert torch.isfinite(runs[0].float()).all() and torch.equal(bits(runs[0]), bits(runs[1]))
    assert (runs[1][1, group:] == 0).all() and B.moe_read_status(ws)[0] == 0


# ------------------------------------------------------------------------ repeats

PARTS = ("q", "out", "tables", "kept", "bounds", "k", "v", "scores")


def bits(t):
    return raw(t) if t.dtype.itemsize < 4 else t.view(torch.int32)


def overwrite(c):
    """Everything that a step writes."""
    seq = c["seq"].long()
    b = torch.arange(len(seq), device="cuda")
    last = c["table"][b, (seq - 1) // c["page"]].long()
    for n in ("q", "out", "tables", "kept"):
        c[n].fill_(7)
    c["scores"].fill_(math.nan)
    bits(c["bounds"])[last] = 17
    for n in ("k", "v"):
        bits(c[n])[last, (seq - 1) % c["page"]] = 17


def results(c):
    return {n: bits(c[n]).clone() for n in PARTS}


def first_step(c):
    """What a step leaves, over overwritten outputs."""
    overwrite(c)
    before = results(c)
    c["step"]()
    torch.cuda.synchronize()
    after = results(c)
    for n in PARTS:
        assert not torch.equal(before[n], after[n]), n
    return after


def same(got, want, what):
    for n in PARTS:
        assert torch.equal(got[n], want[n]), f"{what}: {n}"


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_steps_over_overwritten_outputs(B, dtype):
    """On a side stream, and captured and replayed: every output is written again, with the bits of the eager step."""
    c = chain(B, dtype, T=7, seed=3)
    want = first_step(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        overwrite(c)
        c["step"]()
    torch.cuda.synchronize()
    same(results(c), want, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c["step"]()
    for i in range(4):
        overwrite(c)
        graph.replay()
        torch.cuda.synchronize()
        same(results(c), want, f"replay {i}")


def test_captured_steps_in_turn_over_overwritten_outputs(B):
    both = [chain(B, seed=4), chain(B, "e4m3", T=9, seed=5, prompt=600)]
    want = [first_step(c) for c in both]
    graphs = []
    for c in both:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c["step"]()
    for i in range(4):
        for c, graph in zip(both, graphs):
            overwrite(c)
            graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(both, want):
            same(results(c), w, f"replay {i}")


def test_steps_on_two_streams_at_once_each_checked(B):
    both = [chain(B, seed=8), chain(B, "e4m3", T=9, seed=9, prompt=700)]
    want = [first_step(c) for c in both]
    streams = [torch.cuda.Stream() for _ in both]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    kept = []
    for _ in range(12):
        for i, (c, s) in enumerate(zip(both, streams)):
            with torch.cuda.stream(s):
                overwrite(c)
                c["step"]()
                kept.append((i, results(c)))
    torch.cuda.synchronize()
    for i, r in kept:
        same(r, want[i], f"stream {i}")

"""moe_qk_norm_append against the fp64 oracle on the same inputs.

Tolerances, u = 2^-24: the sum of a head's squares is one of positive terms, 16 serial additions
and 5 levels at most with a rounding per square, 22 u of it, half of which reaches the root;
division, addition of eps, root, and the products with it and the weight are 7 roundings: 18 u
of an element.  The rotation adds 3 of |a| + |b|, the scale of an E4M3 row 2: under 24 u of twice the
largest normed element.  Storing rounds once more (bf16 2^-8, E4M3 2^-4 or half its least step).
"""

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import BF, DT, U, assert_within, cos_sin_table, gen, make_cache, normal, raw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def axes_of(T, A, half, seed, most=60):
    """Positions of A axes and the axis of each pair (runs of the first, then in turn)."""
    g = torch.Generator()
    g.manual_seed(seed)
    at = torch.randint(0, most, (A, T), generator=g, dtype=torch.int32).cuda()
    return at, bytes(0 if i < half // 3 else i % A for i in range(half))


def run(B, T=19, R=5, hq=6, hkv=3, D=128, rot=128, A=0, x="bf16", dtype="bf16", w="bf16", page=8, heads_first=False,
        eps=1e-6, pad=0, shift=0, with_q=True, in_place=False, cols=6, seed=0, spoil=None):
    """One call, all of whose outputs are checked; ``spoil(pos, axis_positions, req, table)`` makes
    tokens that are dropped (it returns their numbers)."""
    g = gen(seed)
    pages = R * cols
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype, heads_first)
    room = normal(g, T * (hq + 2 * hkv) * (D + pad) + shift, std=2.0, dtype=DT[x])
    qkv = room[shift:].view(T, hq + 2 * hkv, D + pad)[..., :D]
    q, kn, vn = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    weights = [(1 + 0.2 * normal(g, D)).to(DT[w]) if w else None for _ in range(2)]
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(R, cols)
    req = torch.tensor([t % R for t in range(T)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([(11 * (t % R)) % 17 + t // R for t in range(T)], dtype=torch.int32, device="cuda")
    assert int(pos.max()) < cols * page
    if T > 7:
        pos[7] = -1
    cs = cos_sin_table(64, rot) if rot else None
    at, axis = axes_of(T, A, rot // 2, seed) if A else (None, None)
    lost = spoil(pos, at, req, table) if spoil else []
    qo = q if in_place else torch.empty(T, hq, D, dtype=DT[x], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = raw(k).clone(), raw(v).clone()

    def turned(y):
        if not rot:
            return y
        return O.rotate_axes(y, pos, cs, at, axis) if A else O.rotate(y, pos, cs)

    qn, kn_ = O.qk_norm(q, weights[0], eps), O.qk_norm(kn, weights[1], eps)
    qr, kr, vr = turned(qn), turned(kn_), O.f64(vn)
    B.moe_qk_norm_append(q if with_q else None, kn, vn, weights[0], weights[1], eps, cache, table, pos,
                         qo if with_q else None, req=req, cos_sin=cs, axis_positions=at, axis=axis, status=status)
    torch.cuda.synchronize()
    assert status.item() == (-6 if lost else 0)
    mag = 2 * max(qn.abs().max().item(), kn_.abs().max().item())
    if with_q:
        assert_within(qo, qr, 24 * U * mag + (BF if x == "bf16" else U) * qr.abs() * 1.01, "q")
    touched = torch.zeros(k.shape[:2], dtype=torch.bool)
    for t in range(T):
        if pos[t] < 0 or t in lost:
            continue
        p, i = O.slot_of(table, int(req[t]), int(pos[t]), page)
        touched[p, i] = True
        for name, c, s, want in (("k", k, ks, kr[t]), ("v", v, vs, vr[t])):
            row = raw(c)[p, i].view(c.dtype)
            slack = 24 * U * mag if name == "k" else 4 * U * want.abs()
            if s is not None:
                sd = O.f64(s)[:, None]
                want = want.clamp(-448 * sd, 448 * sd)
                assert_within(O.f64(row) * sd, want, want.abs() * 2.0 ** -4 * 1.0001 + sd * 2.0 ** -10 * 1.0001 + slack,
                              f"{name} of token {t}")
            else:
                assert_within(row, want, BF * want.abs() * 1.01 + slack, f"{name} of token {t}")
    for c, b in ((k, before[0]), (v, before[1])):
        assert torch.equal(raw(c).cpu()[~touched], b.cpu()[~touched])


@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (80, 40), (80, 80), (256, 256), (256, 32), (16, 2), (128, 0),
                                   (48, 6), (16, 16), (96, 96), (240, 16)])
@pytest.mark.parametrize("x,dtype", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("A", [0, 3])
def test_qk_append(B, D, rot, x, dtype, A):
    run(B, D=D, rot=rot, x=x, dtype=dtype, A=A if rot else 0, heads_first=A > 0, seed=D + rot)


@pytest.mark.parametrize("D", [8, 24, 56, 72, 136, 200, 248])
def test_qk_append_head_dims_of_eight(B, D):
    run(B, D=D, rot=0, seed=D)
    run(B, D=D, rot=D // 16 * 16, x="f32", A=2 if D >= 16 else 0, seed=D)
    run(B, D=D, rot=D, seed=D)


@pytest.mark.parametrize("w", [None, "f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_qk_append_weights(B, w, eps):
    run(B, w=w, eps=eps, seed=3)
    run(B, w=w, eps=eps, D=80, rot=40, A=2, seed=4)


def test_qk_append_one_weight(B):
    """Ones for the keys, and the other way round; types of the only weight."""
    g = gen(5)
    k, v, _, _, cache = make_cache(B, g, 4, 4, 2, 64, "bf16")
    q, kn, vn = (normal(g, 1, h, 64, dtype=torch.bfloat16) for h in (4, 2, 2))
    table, pos = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4), torch.tensor([9], dtype=torch.int32, device="cuda")
    for name in ("q", "k"):
        for dt in (torch.float32, torch.bfloat16):
            w = (1 + 0.2 * normal(g, 64)).to(dt)
            qw, kw = (w, None) if name == "q" else (None, w)
            qo = torch.empty_like(q)
            B.moe_qk_norm_append(q, kn, vn, qw, kw, 1e-6, cache, table, pos, qo)
            for got, want in ((qo[0], O.qk_norm(q, qw, 1e-6)[0]), (k[2, 1], O.qk_norm(kn, kw, 1e-6)[0])):
                assert_within(got, want, 1.01 * BF * want.abs() + 1e-5, name)
            assert torch.equal(v[2, 1], vn[0])


@pytest.mark.parametrize("A", [1, 2, 4, 7])
@pytest.mark.parametrize("rot", [128, 32, 24])
def test_qk_append_axes(B, A, rot):
    run(B, A=A, rot=rot, seed=A)
    run(B, A=A, rot=rot, D=256, hq=2, hkv=2, x="f32", seed=A)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (7, 1), (56, 8), (40, 20), (3, 3)])
@pytest.mark.parametrize("T", [1, 2, 40])
def test_qk_append_heads(B, hq, hkv, T):
    run(B, T=T, R=min(T, 5), hq=hq, hkv=hkv, A=3, seed=T + hq)
    run(B, T=T, R=min(T, 5), hq=hq, hkv=hkv, D=64, rot=64, x="f32", seed=T + hq)


def test_qk_append_strides_in_place_and_without_q(B):
    run(B, pad=8, seed=6)
    run(B, pad=4, seed=6)                    # rows that are not a multiple of 16 bytes apart, but of 8
    run(B, shift=4, A=3, rot=64, seed=6)
    run(B, pad=4, x="f32", D=80, rot=80, hq=9, seed=6)
    run(B, pad=3, seed=6)                    # nor of 8
    run(B, shift=1, seed=7)                  # nor aligned
    run(B, shift=1, x="f32", A=2, seed=7)
    run(B, in_place=True, seed=8)
    run(B, in_place=True, rot=24, seed=8)
    run(B, with_q=False, seed=9)
    run(B, with_q=False, rot=24, A=2, seed=9)


@pytest.mark.parametrize("T,hq,hkv,D,rot,x,A", [(2600, 8, 2, 64, 32, "bf16", 3), (1500, 40, 20, 256, 256, "f32", 0),
                                                (2100, 9, 3, 80, 80, "bf16", 4), (700, 9, 3, 80, 40, "f32", 2)])
def test_qk_append_many_tokens(B, T, hq, hkv, D, rot, x, A):
    """Blocks that take several tokens, or slices of their heads, with padding and dropped tokens in between."""
    R, page, g = 7, 16, gen(T)
    per = (T + R - 1) // R
    cols = (per + page - 1) // page
    k, v, _, _, cache = make_cache(B, g, R * cols, page, hkv, D, "bf16", fill=0)
    qkv = normal(g, T, hq + 2 * hkv, D, dtype=DT[x])
    q, kn, vn = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    qw, kw = (1 + 0.2 * normal(g, D) for _ in range(2))
    table = torch.randperm(R * cols, generator=g, device="cuda").to(torch.int32).view(R, cols)
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    req, pos = i % R, i // R
    pos[5::11] = -1
    req[7::301] = R
    rows = 64 if A else per
    at, axis = axes_of(T, A, rot // 2, T) if A else (None, None)
    bad = torch.zeros(T, dtype=torch.bool)
    if A:
        at[axis[rot // 2 - 1], 9::97] = rows          # no such row of cos_sin
        at[axis[0], 13::201] = -1
        bad[9::97] = True
        bad[13::201] = True
    cs = cos_sin_table(rows, rot)
    qo = torch.empty(T, hq, D, dtype=DT[x], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_qk_norm_append(q, kn, vn, qw, kw, 1e-6, cache, table, pos, qo, req=req, cos_sin=cs, axis_positions=at, axis=axis,
                         status=status)
    torch.cuda.synchronize()
    assert status.item() == -6

    def turned(y):
        return O.rotate_axes(y, pos, cs, at, axis) if A else O.rotate(y, pos, cs)

    qn, kn_ = O.qk_norm(q, qw, 1e-6), O.qk_norm(kn, kw, 1e-6)
    mag = 2 * max(qn.abs().max().item(), kn_.abs().max().item())
    qr = turned(qn)
    assert_within(qo, qr, 24 * U * mag + (BF if x == "bf16" else U) * qr.abs() * 1.01, "q")
    kept = ((pos >= 0) & (req < R)).cpu() & ~bad
    t = torch.nonzero(kept).flatten()
    where = table.cpu().long()[req.cpu()[t].long(), pos.cpu()[t].long() // page], pos.cpu()[t].long() % page
    for name, c, want in (("k", k, turned(kn_)), ("v", v, O.f64(vn))):
        full = torch.zeros(c.shape, dtype=torch.float64)
        full[where] = want.cpu()[t]
        assert_within(c, full, BF * full.abs() * 1.01 + 24 * U * mag * (full != 0), name)


@pytest.mark.parametrize("T,hq,hkv,D,rot,x,A", [(700, 16, 4, 128, 128, "f32", 3), (650, 32, 8, 64, 64, "bf16", 0),
                                                (1300, 5, 5, 16, 16, "f32", 2), (640, 6, 2, 80, 40, "bf16", 3)])
def test_qk_append_few_heads_of_many_tokens(B, T, hq, hkv, D, rot, x, A):
    """Heads of q that narrow blocks take, for just as many tokens as they need and more."""
    test_qk_append_many_tokens(B, T, hq, hkv, D, rot, x, A)
    run(B, T=T, R=200, hq=hq, hkv=hkv, D=D, rot=rot, x=x, A=A, dtype="e4m3", seed=T)
    run(B, T=T, R=200, hq=hq, hkv=hkv, D=D, rot=rot, x=x, A=A, pad=4, seed=T)


@pytest.mark.parametrize("bad", ["req", "table", "page_high", "page_negative", "position_cos", "axis_high", "axis_negative"])
@pytest.mark.parametrize("rot", [128, 24])
def test_qk_append_drops_tokens_without_a_slot(B, bad, rot):
    def spoil(pos, at, req, table):
        if bad == "req":
            req[3] = 5
        elif bad == "table":
            pos[3] = 48
        elif bad == "page_high":
            table[3, int(pos[3]) // 8] = 30
        elif bad == "page_negative":
            table[3, int(pos[3]) // 8] = -1
        elif bad == "position_cos":
            pos[3] = 64
        elif bad == "axis_high":
            at[1, 3] = 64
        else:
            at[0, 3] = -1
        lost = [3]
        if bad.startswith("page"):
            # every token of that page of request 3
            lost = [t for t in range(3, 19, 5) if int(pos[t]) // 8 == int(pos[3]) // 8]
        return lost

    run(B, rot=rot, A=3 if bad.startswith("axis") else 0, cols=9 if bad == "position_cos" else 6, spoil=spoil, seed=11)


def test_qk_append_slots_beyond_the_axes(B):
    """With axes `positions` only names slots: it may pass the rows of cos_sin."""
    def spoil(pos, at, req, table):
        pos[3] = 70
        return []

    run(B, A=2, cols=9, spoil=spoil, seed=12)


def test_qk_append_rows_that_are_not_finite(B):
    """NaN, infinities and zeros stay in their own head."""
    g = gen(13)
    k, v, _, _, cache = make_cache(B, g, 2, 4, 2, 64, "bf16", fill=0)
    q, kn, vn = (normal(g, 2, h, 64) for h in (2, 2, 2))
    q[0, 1, 5] = float("nan")
    kn[1, 0] = 0.0
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    qo = torch.empty_like(q)
    B.moe_qk_norm_append(q, kn, vn, None, None, 1e-6, cache, table, pos, qo, cos_sin=cos_sin_table(4, 64))
    assert torch.isnan(qo[0, 1]).all() and torch.isfinite(qo[0, 0]).all() and torch.isfinite(qo[1]).all()
    assert (k[1, 0, 0] == 0).all() and torch.isfinite(k).all()


def test_qk_append_no_tokens(B):
    _, _, _, _, cache = make_cache(B, gen(0), 2, 4, 2, 64, "bf16")
    q, kn = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    B.moe_qk_norm_append(q, kn, kn, None, None, 1e-6, cache, i.view(0, 1), i, q, cos_sin=cos_sin_table(4, 64),
                         axis_positions=i.view(2, 0), axis=bytes(32))

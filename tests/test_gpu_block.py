"""The decode-block operators against the fp64 oracle on the same inputs.

Tolerances come from the arithmetic, u = 2^-24 (fp32) and 2^-8 (bf16: 8 significant bits, round to
nearest):
- norm: a row's sum of squares is a tree of at most 32 serial additions per
  thread, then 5 shuffles and at most 32 warps, half of which reaches y, plus
  six roundings: under 40 u = 2.4e-6 relative to each element;
- rotation: two products and an addition: 4 u of |a| + |b|;
- attention: a score is off by at most about (D / 8 + 8) u sum |q k| scale and
  a weight by as much relatively; with the inputs here (sum |q k| scale < 40,
  D <= 256) that is under 1e-4 of the largest |v|, and bf16 output adds 2^-8
  of |o|;
- projection: fp32 accumulation in blocks: 64 u of sum |w x|.
"""

import math

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def e4m3(v):
    return v.clamp(-448, 448).to(torch.float8_e4m3fn)


def assert_within(got, want, bound, what=""):
    got = O.f64(got)
    off = (got - want).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = (off - bound).max().item()
    assert worst <= 0, f"{what}: off by {off.max().item():.3g}, {worst:.3g} over the bound"


# ------------------------------------------------------------------------ norm


def run_norm(B, T, d, x="f32", res=None, y="f32", weight="bf16", group=0, seed=0, eps=1e-5, pad=0, inplace=False):
    g = gen(seed)

    def matrix(dtype, std=1.0):
        return normal(g, T, d + pad, std=std, dtype=dtype)[:, :d]

    xt = matrix(DT[x])
    rt = matrix(DT[res], 3.0) if res else None
    ro = None if rt is None else rt.clone() if pad == 0 else torch.empty_like(matrix(DT[res]))
    if inplace and rt is not None:
        ro.copy_(rt)
        res_arg = ro
    else:
        res_arg = rt
    w = (1 + 0.1 * normal(g, d)).to(DT[weight]) if weight else None
    yt = torch.empty(T, d + pad, dtype=DT[y], device="cuda")[:, :d]
    sc = None
    if y == "e4m3":
        sc = torch.empty((T, d // group) if group else (T,), device="cuda")
    yr, zr = O.rms_norm(xt, w, eps, rt)
    B.moe_rmsnorm(xt, w, eps, yt, residual=res_arg, residual_out=ro, y_scale=sc)
    torch.cuda.synchronize()
    if ro is not None:
        assert_within(ro, zr, zr.abs() * (BF if res == "bf16" else U) * 1.01 + 1e-30, "residual_out")
    # an element's own addition x + residual is rounded relative to the sum
    tol = 40 * U * yr.abs()
    if y == "e4m3":
        sr = O.e4m3_scales(yr, group)
        assert_within(sc, sr, 40 * U * sr, "scale")
        s = O.f64(sc).repeat_interleave(group, 1) if group else O.f64(sc)[:, None]
        got = O.f64(yt) * s
        assert_within(got, yr, yr.abs() * 2.0 ** -4 * 1.0001 + s * 2.0 ** -10 * 1.0001, "codes")
        assert O.f64(yt).abs().max() <= 448
    else:
        assert_within(yt, yr, tol + (yr.abs() * BF * 1.01 if y == "bf16" else 0), "y")


@pytest.mark.parametrize("T", [1, 2, 33])
@pytest.mark.parametrize("d", [8, 24, 256, 1000, 2048, 2056, 7168, 8200, 16384, 32768])
def test_norm_sizes(B, T, d):
    run_norm(B, T, d, res="f32", seed=T + d)
    run_norm(B, T, d, x="bf16", y="bf16", seed=T + d)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("res", [None, "f32", "bf16"])
@pytest.mark.parametrize("y", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("weight", [None, "f32", "bf16"])
def test_norm_types(B, x, res, y, weight):
    run_norm(B, 5, 1024, x=x, res=res, y=y, weight=weight, seed=1)


@pytest.mark.parametrize("T,d", [(1, 128), (3, 256), (130, 1152), (7, 7168), (2, 32768)])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_e4m3_scales(B, T, d, group):
    run_norm(B, T, d, res="bf16", x="bf16", y="e4m3", group=group, seed=d)


@pytest.mark.parametrize("T,d", [(700, 64), (3000, 256), (2500, 512), (1200, 2048), (400, 7168)])
def test_norm_many_rows(B, T, d):
    run_norm(B, T, d, x="bf16", res="bf16", y="bf16", seed=T)
    run_norm(B, T, d, x="f32", y="e4m3", seed=T)


@pytest.mark.parametrize("T,d", [(400, 8200), (311, 12288), (170, 16384)])
def test_norm_many_wide_rows(B, T, d):
    run_norm(B, T, d, res="f32", seed=d)
    run_norm(B, T, d, x="bf16", res="bf16", y="bf16", seed=d)


def test_norm_strides_and_in_place(B):
    run_norm(B, 9, 520, res="f32", y="bf16", pad=24, seed=3)
    run_norm(B, 9, 512, res="f32", y="f32", inplace=True, seed=4)
    run_norm(B, 9, 512, res="bf16", x="bf16", y="e4m3", inplace=True, seed=4)
    # y is x itself, and residual_out is x itself
    x = normal(gen(5), 7, 768)
    r = normal(gen(6), 7, 768)
    yr, zr = O.rms_norm(x, None, 1e-6, r)
    a = x.clone()
    B.moe_rmsnorm(a, None, 1e-6, a, residual=r)
    assert_within(a, yr, 40 * U * yr.abs(), "y in x")
    a, y = x.clone(), torch.empty_like(x)
    B.moe_rmsnorm(a, None, 1e-6, y, residual=r, residual_out=a)
    assert_within(a, zr, U * zr.abs(), "sum in x")
    assert_within(y, yr, 40 * U * yr.abs(), "y")


def test_norm_zero_rows_and_extremes(B):
    """Rows of zeros (with eps 0 they are 0 / 0), one large row, tiny rows."""
    x = torch.zeros(4, 256, device="cuda")
    x[1, 3] = 1e18
    x[2] = 1e-20
    x[3] = 3.0
    y, q = torch.empty_like(x), torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(4, 2, device="cuda")
    B.moe_rmsnorm(x, None, 1e-5, y)
    yr, _ = O.rms_norm(x, None, 1e-5)
    assert_within(y, yr, 40 * U * yr.abs() + 1e-44, "y")
    B.moe_rmsnorm(x, None, 1e-5, q, y_scale=sc)
    assert sc[0].tolist() == [1.0, 1.0] and sc[1, 1].item() == 1.0
    assert O.f64(q)[0].abs().max() == 0 and O.f64(q)[1, 3] == 448 and O.f64(q)[3].eq(448).all()
    x[0, 0] = float("nan")
    B.moe_rmsnorm(x, None, 1e-5, y)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1:]).all()


# ---------------------------------------------------------------------- append


def make_cache(B, g, pages, page, heads, D, dtype, heads_first=False, fill=None):
    shape = (pages, heads, page, D) if heads_first else (pages, page, heads, D)
    out = []
    for _ in range(2):
        s = None
        v = normal(g, *shape)
        if dtype == "e4m3":
            s = (0.5 + torch.rand(heads, generator=g, device="cuda")) * (4 / 448)
            v = e4m3(v / (s[:, None, None] if heads_first else s[:, None]))
        else:
            v = v.to(torch.bfloat16)
        if fill is not None:
            v = v.float().fill_(fill).to(v.dtype)
        out.append((v.transpose(1, 2) if heads_first else v, s))
    (k, ks), (v, vs) = out
    return k, v, ks, vs, B.KvCache(k, v, ks, vs)


def cos_sin_table(n, rot):
    half = rot // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def raw(cache):
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache.view(torch.int16)


@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (80, 40), (80, 80), (256, 256), (16, 2), (128, 0), (48, 6)])
@pytest.mark.parametrize("x,dtype", [("bf16", "bf16"), ("f32", "bf16"), ("bf16", "e4m3"), ("f32", "e4m3")])
@pytest.mark.parametrize("heads_first", [False, True])
def test_append(B, D, rot, x, dtype, heads_first):
    T, R, hq, hkv, page = 19, 5, 6, 3, 8
    g = gen(D + rot)
    k, v, ks, vs, cache = make_cache(B, g, 32, page, hkv, D, dtype, heads_first)
    qkv = normal(g, T, hq + 2 * hkv, D, dtype=DT[x])
    q, kn, vn = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    table = torch.randperm(32, generator=g, device="cuda").to(torch.int32)[:R * 6].view(R, 6)
    req = torch.tensor([t % R for t in range(T)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([(11 * (t % R)) % 30 + t // R for t in range(T)], dtype=torch.int32, device="cuda")
    pos[7] = -1
    cs = cos_sin_table(64, rot) if rot else None
    qo = torch.empty(T, hq, D, dtype=DT[x], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = raw(k).clone(), raw(v).clone()
    B.moe_kv_append(kn, vn, cache, table, pos, req=req, cos_sin=cs, q=q, q_out=qo, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    qr, kr = O.rotate(q, pos, cs), O.rotate(kn, pos, cs)
    mag = O.f64(qkv).abs().max().item() * 2
    out_u = BF if x == "bf16" else 0.0
    assert_within(qo, qr, 4 * U * mag + out_u * qr.abs() * 1.01, "q")
    touched = torch.zeros(k.shape[:2], dtype=torch.bool)
    for t in range(T):
        if pos[t] < 0:
            continue
        p, i = O.slot_of(table, int(req[t]), int(pos[t]), page)
        touched[p, i] = True
        for name, c, s, want in (("k", k, ks, kr[t]), ("v", v, vs, O.f64(vn[t]))):
            row = raw(c)[p, i].view(c.dtype)
            if s is not None:
                sd = O.f64(s)[:, None]
                got = O.f64(row) * sd
                bound = want.abs() * 2.0 ** -4 * 1.0001 + sd * 2.0 ** -10 * 1.0001 + 4 * U * mag
                want = want.clamp(-448 * sd, 448 * sd)
            else:
                got, bound = row, BF * want.abs() * 1.01 + 4 * U * mag
            assert_within(got, want, bound, f"{name} of token {t}")
    # nothing else moved
    for c, b in ((k, before[0]), (v, before[1])):
        assert torch.equal(raw(c).cpu()[~touched], b.cpu()[~touched])


@pytest.mark.parametrize("T,hq,hkv,D,rot,x", [(2600, 8, 2, 64, 32, "bf16"), (1500, 40, 20, 256, 256, "f32"),
                                              (3001, 0, 1, 16, 16, "f32"), (2100, 9, 3, 80, 80, "bf16"), (700, 9, 3, 80, 40, "f32")])
def test_append_many_tokens(B, T, hq, hkv, D, rot, x):
    """Blocks that take several tokens, or slices of their heads, with padding and tokens dropped in between."""
    R, page, g = 7, 16, gen(T)
    per = (T + R - 1) // R
    cols = (per + page - 1) // page
    k, v, _, _, cache = make_cache(B, g, R * cols, page, hkv, D, "bf16", fill=0)
    qkv = normal(g, T, hq + 2 * hkv, D, dtype=DT[x])
    q, kn, vn = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    table = torch.randperm(R * cols, generator=g, device="cuda").to(torch.int32).view(R, cols)
    i = torch.arange(T, dtype=torch.int32, device="cuda")
    req, pos = i % R, i // R
    pos[5::11] = -1                                   # padding
    req[7::301] = R                                   # no such request
    qo = torch.empty(T, hq, D, dtype=DT[x], device="cuda")
    cs = cos_sin_table(per, rot)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_kv_append(kn, vn, cache, table, pos, req=req, cos_sin=cs, q=q if hq else None, q_out=qo if hq else None, status=status)
    torch.cuda.synchronize()
    assert status.item() == -6
    mag = O.f64(qkv).abs().max().item() * 2
    if hq:
        qr = O.rotate(q, pos, cs)
        assert_within(qo, qr, 4 * U * mag + (BF if x == "bf16" else 0.0) * qr.abs() * 1.01, "q")
    kept = ((pos >= 0) & (req < R)).cpu()
    t = torch.nonzero(kept).flatten()
    at = table.cpu().long()[req.cpu()[t].long(), pos.cpu()[t].long() // page], pos.cpu()[t].long() % page
    for name, c, want in (("k", k, O.rotate(kn, pos, cs)), ("v", v, O.f64(vn))):
        full = torch.zeros(c.shape, dtype=torch.float64)
        full[at] = want.cpu()[t]
        assert_within(c, full, BF * full.abs() * 1.01 + 4 * U * mag * (full != 0), name)


def test_append_default_requests_in_place_and_without_q(B):
    g = gen(1)
    k, v, _, _, cache = make_cache(B, g, 9, 4, 2, 64, "bf16")
    kn, vn = normal(g, 3, 2, 64, dtype=torch.bfloat16), normal(g, 3, 2, 64, dtype=torch.bfloat16)
    q = normal(g, 3, 4, 64, dtype=torch.bfloat16)
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    pos = torch.tensor([0, 4, 11], dtype=torch.int32, device="cuda")
    cs = cos_sin_table(12, 64)
    qr = O.rotate(q, pos, cs)
    B.moe_kv_append(kn, vn, cache, table, pos, cos_sin=cs, q=q, q_out=q)
    assert_within(q, qr, 1e-5 + 1.01 * BF * qr.abs(), "q in place")
    assert torch.equal(v[0, 0], vn[0]) and torch.equal(v[4, 0], vn[1]) and torch.equal(v[8, 3], vn[2])
    v.zero_()
    B.moe_kv_append(kn, vn, cache, table, pos)
    assert torch.equal(k[8, 3], kn[2]) and torch.equal(v[8, 3], vn[2])


@pytest.mark.parametrize("bad", ["req_high", "req_negative", "position_table", "position_cos", "page_high", "page_negative"])
def test_append_drops_tokens_without_a_slot(B, bad):
    g = gen(2)
    k, v, _, _, cache = make_cache(B, g, 4, 4, 2, 64, "bf16")
    kn, vn = normal(g, 2, 2, 64, dtype=torch.bfloat16), normal(g, 2, 2, 64, dtype=torch.bfloat16)
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    req = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    cs = cos_sin_table(7, 64)
    if bad == "req_high":
        req[1] = 2
    elif bad == "req_negative":
        req[1] = -1
    elif bad == "position_table":
        pos[1] = 8
        cs = cos_sin_table(20, 64)
    elif bad == "position_cos":
        pos[1] = 7
    elif bad == "page_high":
        table[1, 0] = 4
    else:
        table[1, 0] = -1
    before_k, before_v = k.clone(), v.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.moe_kv_append(kn, vn, cache, table, pos, req=req, cos_sin=cs, status=status)
    torch.cuda.synchronize()
    assert status.item() == -6
    assert torch.equal(v[0, 1], vn[0])
    before_v[0, 1] = vn[0]
    assert torch.equal(v, before_v) and torch.equal(k[1:], before_k[1:])
    B.moe_kv_append(kn, vn, cache, table, pos, req=req, cos_sin=cs)     # without a status word


# ------------------------------------------------------------------- attention


def attn_case(B, lens, hq, hkv, D, page, q="bf16", dtype="bf16", out=None, heads_first=False, window=0, softcap=0.0,
              seed=0, poison=True, lse=True, pad=0):
    g = gen(seed)
    nb = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    k, v, ks, vs, cache = make_cache(B, g, pages, page, hkv, D, dtype, heads_first)
    ids = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).tolist()
    width = max(max(need), 1) + pad
    # entries past a request's pages and slots past its length hold nonsense
    table = torch.full((nb, width), -12345, dtype=torch.int32)
    seen = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        for j in range(need[b]):
            table[b, j] = ids[at]
            at += 1
        first = max(0, n - window) if window else 0
        for i in range(first, n):
            seen[table[b, i // page], i % page] = True
        for j in range(first // page):
            table[b, j] = 1 << 30
    if poison:
        nan = torch.tensor(0x7FC0 if dtype == "bf16" else 0x7F).to(torch.int16 if dtype == "bf16" else torch.uint8)
        raw(k)[~seen.cuda()] = nan.cuda()
        raw(v)[~seen.cuda()] = nan.cuda()
    table = table.cuda()
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    qt = normal(g, nb, hq, D, std=1.5, dtype=DT[q])
    ot = torch.full((nb, hq, D), 7.0, dtype=DT[out or q], device="cuda")
    lt = torch.empty(nb, hq, device="cuda") if lse else None
    ws = B.new_attn_workspace(nb, hq, hkv, D)
    scale = D ** -0.5

    def go():
        B.moe_attn_decode(qt, cache, table, seq, scale, ot, ws, window=window, softcap=softcap, lse=lt)

    go()
    torch.cuda.synchronize()
    assert B.moe_read_status(ws)[0] == 0
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        n = max(n, 0)
        rk = O.cached_rows(k, ks, table[b], first, n)
        rv = O.cached_rows(v, vs, table[b], first, n)
        want, wl = O.decode_attention(qt[b], (rk, rv), scale, softcap)
        top = rv.abs().max().item() if n else 0.0
        bound = 1e-4 * top + (1.01 * BF * want.abs() if ot.dtype == torch.bfloat16 else 0.0)
        assert_within(ot[b], want, bound, f"request {b} of length {n}")
        if lse:
            if n == 0:
                assert lt[b].eq(-math.inf).all()
            else:
                assert_within(lt[b], wl, 1e-4 + 4 * U * wl.abs(), f"lse of request {b}")
    return go, ot, lt, ws


LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("q", ["f32", "bf16"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_lengths(B, q, dtype):
    attn_case(B, LENGTHS, 8, 2, 128, 16, q=q, dtype=dtype, seed=1)
    attn_case(B, [0, 5, 0, 0, 700, 0], 8, 2, 128, 16, q=q, dtype=dtype, seed=2)
    attn_case(B, [0], 4, 4, 64, 16, q=q, dtype=dtype, seed=3)
    attn_case(B, [3], 4, 4, 64, 16, q=q, dtype=dtype, seed=3)


@pytest.mark.parametrize("D", [16, 48, 64, 80, 96, 112, 128, 144, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_head_dims(B, D, dtype):
    attn_case(B, [1, 40, 333], 6, 2, D, 16, dtype=dtype, seed=D)
    attn_case(B, [70, 129], 6, 2, D, 16, q="f32", dtype=dtype, seed=D)


@pytest.mark.parametrize("D", [8, 24, 72, 136, 248])
def test_attn_head_dims_of_eight(B, D):
    attn_case(B, [1, 40, 333], 6, 2, D, 16, seed=D)
    attn_case(B, [200], 6, 2, D, 16, q="f32", seed=D)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (3, 1), (5, 1), (7, 1), (8, 1), (9, 1), (16, 1), (17, 1), (24, 1),
                                    (32, 1), (56, 8), (40, 2), (128, 1)])
@pytest.mark.parametrize("q", ["f32", "bf16"])
def test_attn_head_groups(B, hq, hkv, q):
    attn_case(B, [1, 100, 513], hq, hkv, 64, 16, q=q, seed=hq)
    attn_case(B, [290], hq, hkv, 128, 16, q=q, dtype="e4m3", seed=hq)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 64, 100, 128, 1000])
@pytest.mark.parametrize("heads_first", [False, True])
def test_attn_pages(B, page, heads_first):
    attn_case(B, [1, 99, 100, 101, 640], 4, 2, 64, page, heads_first=heads_first, seed=page)
    attn_case(B, [130, 5], 4, 2, 128, page, dtype="e4m3", heads_first=heads_first, seed=page, pad=3)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
@pytest.mark.parametrize("q", ["f32", "bf16"])
def test_attn_window(B, window, q):
    attn_case(B, [0, 1, 16, 50, 117, 1024], 4, 2, 64, 16, q=q, window=window, seed=window)


@pytest.mark.parametrize("softcap", [1.0, 30.0])
@pytest.mark.parametrize("q,dtype", [("f32", "bf16"), ("bf16", "e4m3")])
def test_attn_softcap(B, softcap, q, dtype):
    attn_case(B, [1, 64, 300], 8, 2, 128, 32, q=q, dtype=dtype, softcap=softcap, seed=9)


@pytest.mark.parametrize("lens,hq,hkv,D", [([20000], 8, 2, 128), ([9000, 1, 30000], 4, 1, 64), ([5000] * 40, 8, 4, 64),
                                           ([17] * 700, 4, 2, 64), ([40000], 1, 1, 256), ([3] * 2000, 2, 1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_attn_long_and_many(B, lens, hq, hkv, D, dtype):
    attn_case(B, lens, hq, hkv, D, 64, dtype=dtype, seed=len(lens))


def test_attn_output_types_and_no_lse(B):
    attn_case(B, [100, 7], 4, 2, 64, 16, q="bf16", out="f32", seed=1)
    attn_case(B, [100, 7], 4, 2, 64, 16, q="f32", out="bf16", lse=False, seed=1)


def test_attn_equal_calls_give_equal_bits(B):
    """The same workspace over and over, and another one."""
    for q, dtype in (("f32", "bf16"), ("bf16", "e4m3")):
        go, o, l, _ = attn_case(B, [3000, 0, 17, 50000], 8, 2, 128, 16, q=q, dtype=dtype, seed=5)
        o0, l0 = o.clone(), l.clone()
        for _ in range(5):
            o.fill_(3)
            go()
            torch.cuda.synchronize()
            assert torch.equal(o, o0) and torch.equal(l, l0)


def test_attn_large_scores_and_sinks(B):
    """One key far above the others at the start or the end, and scores all very low."""
    g = gen(7)
    D, n, page = 64, 600, 16
    for where in (0, 17, n - 1):
        k, v, _, _, cache = make_cache(B, g, 40, page, 1, D, "bf16")
        table = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
        q = torch.ones(1, 2, D, device="cuda")
        q[0, 1] = -1.0
        k.zero_()
        k[where // page, where % page] = 40.0
        seq = torch.tensor([n], dtype=torch.int32, device="cuda")
        o, ws = torch.empty(1, 2, D, device="cuda"), B.new_attn_workspace(1, 2, 1, D)
        B.moe_attn_decode(q, cache, table, seq, 1.0, o, ws)
        want, _ = O.decode_attention(q[0], (O.cached_rows(k, None, table[0], 0, n), O.cached_rows(v, None, table[0], 0, n)), 1.0)
        assert_within(o[0], want, 1e-4, f"sink at {where}")


def test_attn_infinite_and_nan_inputs(B):
    """A key of minus infinity weighs nothing; a NaN query spoils its own head alone."""
    g = gen(8)
    k, v, _, _, cache = make_cache(B, g, 8, 16, 1, 64, "bf16")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    k[0, 3, 0, 5] = -math.inf
    q = normal(g, 1, 3, 64).abs()
    q[0, 2, 0] = math.nan
    o, ws = torch.empty(1, 3, 64, device="cuda"), B.new_attn_workspace(1, 3, 1, 64)
    B.moe_attn_decode(q, cache, table, torch.tensor([100], dtype=torch.int32, device="cuda"), 0.1, o, ws)
    want, _ = O.decode_attention(q[0, :2], (O.cached_rows(k, None, table[0], 0, 100), O.cached_rows(v, None, table[0], 0, 100)), 0.1)
    assert_within(o[0, :2], want, 1e-3, "with a key of -inf")
    assert torch.isnan(o[0, 2]).all()


def test_attn_strided_q_and_out(B):
    g = gen(9)
    k, v, _, _, cache = make_cache(B, g, 8, 16, 2, 64, "bf16")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    big = normal(g, 2, 9, 72, dtype=torch.bfloat16)
    q = big[:, 1:5, 8:]
    out = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    seq = torch.tensor([60, 33], dtype=torch.int32, device="cuda")
    wide = torch.full((2, 11), -1, dtype=torch.int32, device="cuda")
    wide[:, :4] = table
    B.moe_attn_decode(q, cache, wide[:, :5], seq, 0.125, out, B.new_attn_workspace(5, 4, 2, 64))
    for b in range(2):
        n = int(seq[b])
        want, _ = O.decode_attention(q[b], (O.cached_rows(k, None, table[b], 0, n), O.cached_rows(v, None, table[b], 0, n)), 0.125)
        assert_within(out[b], want, 4e-4 + 1.01 * BF * want.abs(), f"request {b}")


def test_attn_reports_what_it_cannot_read(B):
    """A length beyond the table, or a page outside the cache: status, and the other keys count."""
    g = gen(10)
    k, v, _, _, cache = make_cache(B, g, 8, 16, 1, 64, "bf16")
    q = normal(g, 2, 2, 64)
    o = torch.empty_like(q)
    for bad in ("length", "page_high", "page_negative"):
        table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
        seq = torch.tensor([64, 64], dtype=torch.int32, device="cuda")
        left = list(range(64))
        if bad == "length":
            seq[1] = 2_000_000_000
        else:
            table[1, 2] = 8 if bad == "page_high" else -3
            left = [i for i in left if i // 16 != 2]
        ws = B.new_attn_workspace(2, 2, 1, 64)
        B.moe_attn_decode(q, cache, table, seq, 0.125, o, ws)
        torch.cuda.synchronize()
        assert B.moe_read_status(ws)[0] == -6
        for b, rows in ((0, list(range(64))), (1, left)):
            fk = torch.cat([O.f64(k[p]) for p in range(4 * b, 4 * b + 4)])[rows]
            fv = torch.cat([O.f64(v[p]) for p in range(4 * b, 4 * b + 4)])[rows]
            want, _ = O.decode_attention(q[b], (fk, fv), 0.125)
            assert_within(o[b], want, 4e-4, f"{bad}, request {b}")


def test_cache_beyond_32_bit_offsets(B):
    """Pages whose offset passes 2^32 elements."""
    D, page, heads = 64, 16, 1
    stride = 1 << 28
    buf = torch.zeros((17 * stride + page * D,), dtype=torch.uint8, device="cuda")
    k = buf.view(torch.float8_e4m3fn).as_strided((18, page, heads, D), (stride, D, D, 1))
    v = buf.view(torch.float8_e4m3fn).as_strided((18, page, heads, D), (stride, D, D, 1), storage_offset=0)
    s = torch.ones(1, device="cuda")
    cache = B.KvCache(k, v, s, s)
    g = gen(11)
    rows = normal(g, 2, 1, D)
    table = torch.tensor([[17]], dtype=torch.int32, device="cuda")
    req = torch.zeros(2, dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    B.moe_kv_append(rows, rows, cache, table, pos, req=req)
    got = buf[17 * stride:17 * stride + 2 * D].view(torch.float8_e4m3fn).float()
    assert torch.equal(got, e4m3(rows).float().flatten())
    q, o = normal(g, 1, 1, D), torch.empty(1, 1, D, device="cuda")
    B.moe_attn_decode(q, cache, table, torch.tensor([2], dtype=torch.int32, device="cuda"), 0.125, o,
                      B.new_attn_workspace(1, 1, 1, D))
    kv = O.f64(got).view(2, 1, D)
    want, _ = O.decode_attention(q[0], (kv, kv), 0.125)
    assert_within(o[0], want, 4e-4, "far page")


# ------------------------------------------------------------------ projection


def lora_case(B, T, d, N, x="bf16", y="f32", r=16, na=5, adapter=None, seed=0, pad=0):
    g = gen(seed)
    xs = ws_ = None
    if x == "e4m3":
        xf, wf = normal(g, T, d), normal(g, N, d, std=0.02)
        xs, ws_ = xf.abs().amax(1) / 448, wf.abs().amax(1) / 448
        xt, wt = e4m3(xf / xs[:, None]), e4m3(wf / ws_[:, None])
    else:
        xt = normal(g, T, d + pad, dtype=DT[x])[:, :d]
        wt = normal(g, N, d + 2 * pad, std=0.02, dtype=torch.bfloat16)[:, :d]
    lora = ad = None
    if r:
        lora = (normal(g, na, r, d, std=0.05, dtype=torch.bfloat16), normal(g, na, N, r, std=0.05, dtype=torch.bfloat16),
                0.5 + torch.rand(na, generator=g, device="cuda"))
        ad = adapter if adapter is not None else [(3 * t) % (na + 1) - 1 for t in range(T)]
        ad = torch.tensor(ad, dtype=torch.int32, device="cuda")
    yt = torch.full((T, N + pad), 9.0, dtype=DT[y], device="cuda")[:, :N]
    ws = B.new_lora_workspace(T, d, r)

    def go():
        B.moe_lora_project(xt, wt, yt, ws, lora=lora, adapter=ad, x_scale=xs, w_scale=ws_)

    go()
    torch.cuda.synchronize()
    assert B.moe_read_status(ws)[0] == 0
    want, size = O.lora_project(xt, wt, lora, ad, xs, ws_)
    assert_within(yt, want, 64 * U * size + (1.01 * BF * want.abs() if y == "bf16" else 0.0), "y")
    return go, yt


@pytest.mark.parametrize("x", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 127, 128])
def test_lora_tokens(B, x, T):
    lora_case(B, T, 512, 384, x=x, seed=T)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("d,N", [(8, 8), (16, 128), (56, 24), (64, 136), (72, 1000), (264, 256), (1000, 120),
                                 (2048, 2560), (7168, 264), (32768, 128)])
def test_lora_sizes(B, x, d, N):
    lora_case(B, 3, d, N, x=x, seed=d)
    lora_case(B, 40, d, N, x=x, y="bf16", r=8, seed=d)


@pytest.mark.parametrize("d,N", [(16, 8), (48, 24), (144, 136), (1008, 1000), (7168, 264)])
def test_lora_e4m3_sizes(B, d, N):
    lora_case(B, 3, d, N, x="e4m3", seed=d)
    lora_case(B, 70, d, N, x="e4m3", y="bf16", r=32, seed=d)


@pytest.mark.parametrize("r", [0, 8, 16, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("T,x", [(1, "f32"), (7, "bf16"), (50, "f32"), (128, "bf16"), (20, "e4m3")])
def test_lora_ranks(B, r, T, x):
    lora_case(B, T, 256, 320, x=x, r=r, seed=r)


@pytest.mark.parametrize("x", ["f32", "e4m3"])
@pytest.mark.parametrize("kind", ["none", "one", "all", "few", "last"])
def test_lora_adapter_mixes(B, kind, x):
    T, na = 37, 37
    ad = {"none": [-1] * T, "one": [3] * T, "all": list(range(T)), "few": [t % 2 * 30 - (t % 2 == 0) for t in range(T)],
          "last": [-1] * (T - 1) + [na - 1]}[kind]
    lora_case(B, T, 256, 264, x=x, na=na, adapter=ad, seed=1)


@pytest.mark.parametrize("x", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("r", [8, 24, 64, 72, 128])
def test_lora_many_tokens_and_ranks(B, x, r):
    """Tokens times rank large enough for the tensor-core form of A x; adapters shared by many tokens or by
    none, small and large d, ranks that do not divide 128."""
    lora_case(B, 128, 16, 136, x=x, r=r, na=40, seed=r)
    lora_case(B, 128, 1040, 264, x=x, r=r, na=3, y="bf16", seed=r)
    lora_case(B, 77, 512, 128, x=x, r=r, na=100, adapter=[(t * 13) % 101 - 1 for t in range(77)], seed=r)
    lora_case(B, 128, 256, 136, x=x, r=r, na=2, adapter=[1] * 128, seed=r)


@pytest.mark.parametrize("x", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("T,r", [(3, 16), (100, 16), (128, 128)])
def test_lora_rows_in_threes(B, x, T, r):
    """As many tiles of rows as make three CTAs share each."""
    lora_case(B, T, 1168, 5120, x=x, r=r, na=9, seed=T + r)


def test_lora_keeps_adapters_apart(B):
    """An adapter of NaN and infinite weights spoils its own tokens alone, whichever kernel forms A x."""
    for T, r in ((6, 8), (96, 64)):
        g = gen(T)
        na, d, N = 8, 256, 256
        x, w = normal(g, T, d, dtype=torch.bfloat16), normal(g, N, d, dtype=torch.bfloat16)
        lora = [normal(g, na, r, d, dtype=torch.bfloat16), normal(g, na, N, r, dtype=torch.bfloat16), torch.ones(na, device="cuda")]
        lora[0][2], lora[1][2] = math.nan, math.nan
        lora[0][5], lora[1][5] = math.inf, -math.inf
        ad = torch.tensor([t % na for t in range(T)], dtype=torch.int32, device="cuda")
        y = torch.empty(T, N, device="cuda")
        B.moe_lora_project(x, w, y, B.new_lora_workspace(T, d, r), lora=tuple(lora), adapter=ad)
        good = [t for t in range(T) if t % na not in (2, 5)]
        clean = [lora[0].clone(), lora[1].clone(), lora[2]]
        for i in (2, 5):
            clean[0][i], clean[1][i] = 0, 0
        want, size = O.lora_project(x, w, clean, ad)
        assert_within(y[good], want[good], 64 * U * size[good], "the other tokens")
        assert not torch.isfinite(y[[t for t in range(T) if t % na in (2, 5)]]).any()


def test_lora_large(B):
    lora_case(B, 1, 7168, 9216, x="f32", seed=1)
    lora_case(B, 128, 7168, 7168, x="f32", y="bf16", r=64, na=20, seed=2)
    lora_case(B, 128, 7168, 9216, x="e4m3", y="bf16", r=16, seed=3)


def test_lora_strides_and_equal_bits(B):
    for x in ("f32", "bf16"):
        go, y = lora_case(B, 21, 1024, 520, x=x, pad=8, seed=2)
        y0 = y.clone()
        for _ in range(3):
            y.fill_(0)
            go()
            torch.cuda.synchronize()
            assert torch.equal(y, y0)


@pytest.mark.parametrize("x,T", [("bf16", 3), ("bf16", 48), ("e4m3", 128), ("f32", 70), ("bf16", 2)])
def test_lora_inputs_of_the_kernel_before(B, x, T):
    """x comes from the norm right before, the adapters' numbers from a copy before that; what an earlier
    call left in a cache must not be seen."""
    g, d, N, r, na = gen(T), 1024, 768, 32, 6
    src = [normal(g, T, d) for _ in range(2)]
    ids = [torch.randint(-1, na, (T,), generator=g, device="cuda", dtype=torch.int32) for _ in range(2)]
    w = normal(g, N, d, std=0.02)
    w, ws_ = (e4m3(w / 0.0004), torch.full((N,), 0.0004, device="cuda")) if x == "e4m3" else (w.to(torch.bfloat16), None)
    lora = (normal(g, na, r, d, std=0.05, dtype=torch.bfloat16), normal(g, na, N, r, std=0.05, dtype=torch.bfloat16),
            torch.rand(na, generator=g, device="cuda"))
    h = torch.empty(T, d, dtype=torch.float8_e4m3fn if x == "e4m3" else DT[x], device="cuda")
    hs = torch.empty(T, device="cuda") if x == "e4m3" else None
    ad, ws = torch.empty(T, dtype=torch.int32, device="cuda"), B.new_lora_workspace(T, d, r)
    y = torch.empty(T, N, device="cuda")

    def step(i):
        ad.copy_(ids[i])
        B.moe_rmsnorm(src[i], None, 1e-6, h, y_scale=hs)
        B.moe_lora_project(h, w, y, ws, lora=lora, adapter=ad, x_scale=hs, w_scale=ws_)

    want = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        ref, size = O.lora_project(h, w, lora, ad, hs, ws_)
        assert_within(y, ref, 64 * U * size, "y")
        want.append(y.clone())
    got = []
    for k in range(60):
        step(k % 2)
        got.append(y.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k % 2]) for k in range(60))


def test_lora_reports_adapters_out_of_range(B):
    g = gen(3)
    x, w = normal(g, 3, 64, dtype=torch.bfloat16), normal(g, 32, 64, dtype=torch.bfloat16)
    lora = (normal(g, 2, 8, 64, dtype=torch.bfloat16), normal(g, 2, 32, 8, dtype=torch.bfloat16), torch.ones(2, device="cuda"))
    ad = torch.tensor([1, 2, -7], dtype=torch.int32, device="cuda")
    y, ws = torch.empty(3, 32, device="cuda"), B.new_lora_workspace(3, 64, 8)
    B.moe_lora_project(x, w, y, ws, lora=lora, adapter=ad)
    torch.cuda.synchronize()
    assert B.moe_read_status(ws)[0] == -6
    want, size = O.lora_project(x, w, lora, ad)
    assert_within(y, want, 64 * U * size, "y")


# ------------------------------------------------------- streams and graphs


def test_block_calls_on_another_stream_and_in_a_graph(B):
    """norm -> projection -> append -> attention on a side stream and replayed
    from a CUDA graph give the bits of the eager run."""
    g = gen(4)
    T, d, hq, hkv, D = 6, 256, 4, 2, 64
    x, w = normal(g, T, d), normal(g, (hq + 2 * hkv) * D, d, std=0.05, dtype=torch.bfloat16)
    k, v, _, _, cache = make_cache(B, g, 12, 16, hkv, D, "bf16")
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(6, 2)
    pos = torch.tensor([0, 5, 9, 16, 30, 31], dtype=torch.int32, device="cuda")
    seq, cs = pos + 1, cos_sin_table(32, D)
    h, qkv = torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, w.shape[0], dtype=torch.bfloat16, device="cuda")
    out = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    ws1, ws2 = B.new_lora_workspace(T, d), B.new_attn_workspace(T, hq, hkv, D)

    def block():
        B.moe_rmsnorm(x, None, 1e-5, h)
        B.moe_lora_project(h, w, qkv, ws1)
        heads = qkv.view(T, -1, D)
        q = heads[:, :hq]
        B.moe_kv_append(heads[:, hq:hq + hkv], heads[:, hq + hkv:], cache, table, pos, cos_sin=cs, q=q, q_out=q)
        B.moe_attn_decode(q, cache, table, seq, 0.125, out, ws2)

    block()
    torch.cuda.synchronize()
    want, kw = out.clone(), k.clone()
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(k, kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(k, kw)

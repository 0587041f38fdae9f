"""Timed cases of the operators around the MoE layer in a decode block.

Four operators, each in two forms.  With ``own`` false, ``run`` computes an
operator in its plain form: elementary torch operations in fp32, rounded once
at the end.  With ``own`` true it makes the library calls:

- ``norm``:    root-mean-square norm of x + residual, its output in fp32, bf16
               or E4M3 codes with fp32 scales (``moe_rmsnorm``);
- ``append``:  rotary position encoding of q and k, and k, v written into a
               paged cache in bf16 or E4M3 (``moe_kv_append``);
- ``attn``:    attention of one new token per request over the paged cache,
               requests of different lengths (``moe_attn_decode``);
- ``project``: a shared projection with low-rank adapters of many requests
               (``moe_lora_project``).

Hidden sizes and batch sizes are those of the layer shapes in
``moe_decode_layer_fp32_gb300/synth.py`` (d = 256, 1024, 2048 and 7168, 1 to
128 tokens); head counts are d / 128 query heads with 2 to 8 key-value heads.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-5


def _binding():
    from moe_decode_layer_fp32_gb300 import binding
    return binding


_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # One stream of a 2048-wide model: the norm before the MoE layer, which takes fp32.
        {"name": "norm-1x2048-f32", "op": "norm", "T": 1, "d": 2048, "x": "f32", "y": "f32", "residual": True,
         "group": 0},
        # A full decode batch of a 7168-wide model, quantised for an E4M3 projection.
        {"name": "norm-128x7168-e4m3", "op": "norm", "T": 128, "d": 7168, "x": "bf16", "y": "e4m3",
         "residual": True, "group": 0},
        # A prompt of that model, with one scale per 128 columns.
        {"name": "norm-8191x7168-e4m3-blocks", "op": "norm", "T": 8191, "d": 7168, "x": "bf16", "y": "e4m3",
         "residual": True, "group": 128},
        # The new tokens of 16 requests of the 2048-wide model, bf16 cache.
        {"name": "append-16-bf16", "op": "append", "T": 16, "R": 16, "hq": 16, "hkv": 4, "D": 128, "rot": 128,
         "page": 16, "x": "bf16", "cache": "bf16", "heads_first": False},
        # Prompts of four requests of the 7168-wide model, E4M3 cache.
        {"name": "append-12345-e4m3", "op": "append", "T": 12345, "R": 4, "hq": 56, "hkv": 8, "D": 128, "rot": 64,
         "page": 64, "x": "bf16", "cache": "e4m3", "heads_first": True},
        # One short conversation: latency.
        {"name": "attn-1x777-bf16", "op": "attn", "B": 1, "L": 777, "ragged": False, "hq": 16, "hkv": 4, "D": 128,
         "page": 16, "q": "bf16", "cache": "bf16", "heads_first": False, "window": 0, "softcap": 0.0},
        # A serving batch of mixed lengths, two slots of it idle or new.
        {"name": "attn-16x4096-ragged-f32", "op": "attn", "B": 16, "L": 4096, "ragged": True, "hq": 16, "hkv": 4,
         "D": 128, "page": 32, "q": "f32", "cache": "bf16", "heads_first": False, "window": 0, "softcap": 0.0},
        # One document of 128k tokens on the 7168-wide model.
        {"name": "attn-1x131071-bf16", "op": "attn", "B": 1, "L": 131071, "ragged": False, "hq": 56, "hkv": 8,
         "D": 128, "page": 64, "q": "bf16", "cache": "bf16", "heads_first": True, "window": 0, "softcap": 0.0},
        # The largest serving batch, E4M3 cache, capped scores.
        {"name": "attn-128x4096-ragged-e4m3", "op": "attn", "B": 128, "L": 4096, "ragged": True, "hq": 56, "hkv": 8,
         "D": 128, "page": 64, "q": "bf16", "cache": "e4m3", "heads_first": False, "window": 0, "softcap": 30.0},
        # One stream's q, k, v projection (16 + 2 * 2 heads of 128).
        {"name": "project-1-2048-2560-r16", "op": "project", "T": 1, "d": 2048, "N": 2560, "x": "f32", "y": "f32",
         "r": 16, "adapters": 1, "used": 1},
        # 32 streams of the 7168-wide model, 9 adapters among them (56 + 2 * 8 heads of 128).
        {"name": "project-32-7168-9216-r16", "op": "project", "T": 32, "d": 7168, "N": 9216, "x": "bf16",
         "y": "bf16", "r": 16, "adapters": 12, "used": 9},
        # The E4M3 projection of a full batch, an adapter of its own for every second request.
        {"name": "project-128-7168-7168-e4m3-r64", "op": "project", "T": 128, "d": 7168, "N": 7168, "x": "e4m3",
         "y": "bf16", "r": 64, "adapters": 64, "used": 64},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size8(rng, lo, hi, step=8):
    """A multiple of ``step``, log-uniform in [lo, hi]."""
    n = max(lo // step, min(hi // step, _log(rng, lo, hi) // step)) * step
    return n + step if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "attn", "project", "project"])
    if op == "norm":
        group = rng.choice([0, 0, 128])
        y = "e4m3" if group else rng.choice(["f32", "bf16", "e4m3"])
        return {"op": op, "T": _log(rng, 1, 8000), "d": _size8(rng, 256, 7168, 128 if group else 8),
                "x": rng.choice(["f32", "bf16"]), "y": y, "residual": rng.random() < 0.7, "group": group}
    if op == "append":
        R = _log(rng, 1, 128)
        D = rng.choice([64, 80, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": op, "T": R * _log(rng, 1, 12000 // R), "R": R, "hq": hkv * rng.choice([1, 2, 4, 7]) if D < 256 else hkv,
                "hkv": hkv, "D": D, "rot": rng.choice([0, D // 2, D]), "page": rng.choice([1, 16, 24, 64, 128]),
                "x": rng.choice(["f32", "bf16"]), "cache": rng.choice(["bf16", "e4m3"]),
                "heads_first": rng.random() < 0.5}
    if op == "attn":
        D = rng.choice([64, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 7, 8, 16] if D < 256 else [1, 2, 4])
        B = _log(rng, 1, 128)
        # no more cached values than the largest listed case
        most = min(131072, 128 * 4096 * 8 * 128 // (3 * B * hkv * D))
        return {"op": op, "B": B, "L": _log(rng, 1, most), "ragged": rng.random() < 0.7, "hq": hq, "hkv": hkv,
                "D": D, "page": rng.choice([1, 16, 24, 32, 64, 128]), "q": rng.choice(["f32", "bf16"]),
                "cache": rng.choice(["bf16", "e4m3"]), "heads_first": rng.random() < 0.5,
                "window": rng.choice([0, 0, 0, 1, 512]), "softcap": rng.choice([0.0, 0.0, 30.0])}
    x = rng.choice(["f32", "bf16", "e4m3"])
    T = _log(rng, 1, 128)
    adapters = _log(rng, 1, 64)
    step = 16 if x == "e4m3" else 8
    return {"op": op, "T": T, "d": _size8(rng, 256, 7168, step), "N": _size8(rng, 256, 7168), "x": x,
            "y": rng.choice(["f32", "bf16"]), "r": rng.choice([0, 8, 16, 32, 64]), "adapters": adapters,
            "used": rng.randint(1, min(adapters, T))}


def _lens(case):
    """Cached tokens per request, the new one included (before shuffling)."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    lens = [max(1, round(L * ((i + 1) / B) ** 1.5)) for i in range(B)]
    if B >= 8:
        lens[0] = 0    # an idle slot of the batch
        lens[1] = 1    # a request that has just begun
    return lens


def _seen(case, n):
    return min(n, case["window"]) if case["window"] else n


def _adapter_of(case):
    """Adapter of each token (before shuffling): ``used`` of them in turn, -1 (none) now and then."""
    T, used = case["T"], case["used"]
    ids = [i * case["adapters"] // used for i in range(used)]
    return [-1 if used < T and t % 8 == 7 else ids[t % used] for t in range(T)]


def _with_adapters(case):
    return case["r"] > 0


# ------------------------------------------------------------------ inputs


class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.host = random.Random(seed)

    def normal(self, *shape, std=1.0):
        return torch.randn(shape, generator=self.g, device="cuda", dtype=torch.float32).mul_(std)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.g, device="cuda", dtype=torch.float32)

    def perm(self, n):
        return torch.randperm(n, generator=self.g, device="cuda")

    def shuffled(self, values):
        values = list(values)
        self.host.shuffle(values)
        return torch.tensor(values, dtype=torch.int32, device="cuda")


def _hidden(g, T, d):
    """Residual-stream rows: a few channels are much larger than the others."""
    big = 1.0 + 15.0 * (g.uniform(d) < 0.004).float()
    return g.normal(T, d) * big


def _to_e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _cache(g, pages, page, heads, D, dtype, heads_first):
    """(cache viewed as [pages, page, heads, D], scale per head or None)."""
    shape = (pages, heads, page, D) if heads_first else (pages, page, heads, D)
    values = torch.empty(shape, dtype=_DT[dtype], device="cuda")
    scale = (0.5 + g.uniform(heads)) * (4.0 / E4M3_MAX) if dtype == "e4m3" else None
    per = max(1, (1 << 26) // (page * heads * D))
    for p in range(0, pages, per):
        v = g.normal(*((min(per, pages - p),) + shape[1:]))
        if scale is not None:
            v = _to_e4m3(v / (scale[:, None, None] if heads_first else scale[:, None]))
        values[p:p + per].copy_(v)
    return (values.transpose(1, 2) if heads_first else values), scale


def _caches(g, s, pages):
    """One layer's key and value caches, and the library's handle of them."""
    case = s["case"]
    for name in ("k", "v"):
        s[name + "_cache"], s[name + "_scale"] = _cache(g, pages, case["page"], case["hkv"], case["D"], case["cache"],
                                                        case["heads_first"])
    if own:
        s["cache"] = _binding().KvCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def _tables(g, counts, page, spare=1):
    """Block table [R, most] of requests with ``counts`` tokens: pages in random order, -1 past a request's last."""
    need = [-(-c // page) for c in counts]
    pages, width = sum(need) + spare, max(max(need), 1)
    ids = g.perm(pages).to(torch.int32)
    slots = torch.tensor(need, device="cuda")
    first = torch.cumsum(slots, 0) - slots
    col = torch.arange(width, device="cuda")
    table = ids[(first[:, None] + col).clamp(max=pages - 1)]
    return torch.where(col < slots[:, None], table, torch.full_like(table, -1)).contiguous(), pages


def prepare(case, seed):
    g = _Draws(seed)
    return {"norm": _prepare_norm, "append": _prepare_append, "attn": _prepare_attn,
            "project": _prepare_project}[case["op"]](case, g)


def _prepare_norm(case, g):
    T, d = case["T"], case["d"]
    dt = _DT[case["x"]]
    s = {"case": case, "x": (0.3 * _hidden(g, T, d)).to(dt), "weight": (1.0 + 0.1 * g.normal(d)).to(torch.bfloat16)}
    s["residual"] = _hidden(g, T, d).to(dt) if case["residual"] else None
    s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
    s["y"] = torch.empty((T, d), dtype=_DT[case["y"]], device="cuda")
    s["y_scale"] = None
    if case["y"] == "e4m3":
        s["y_scale"] = torch.empty((T, d // case["group"]) if case["group"] else (T,), dtype=torch.float32,
                                   device="cuda")
    return s


def _prepare_append(case, g):
    T, R, hq, hkv, D = (case[k] for k in ("T", "R", "hq", "hkv", "D"))
    # each request gets T / R new tokens after the ones it has
    new = T // R + 1
    old = [(37 * i) % 100 for i in range(R)]
    g.host.shuffle(old)
    req = torch.tensor([t % R for t in range(T)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([old[t % R] + t // R for t in range(T)], dtype=torch.int32, device="cuda")
    table, pages = _tables(g, [o + new for o in old], case["page"])
    # one q, k, v projection's output, sliced by heads
    qkv = g.normal(T, hq + 2 * hkv, D).to(_DT[case["x"]])
    s = {"case": case, "req": req if R != T else None, "positions": pos, "block_table": table,
         "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "cos_sin": None}
    s["q_out"] = torch.empty((T, hq, D), dtype=_DT[case["x"]], device="cuda")
    if case["rot"]:
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ang = torch.arange(max(old) + new, device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    _caches(g, s, pages)
    return s


def _prepare_attn(case, g):
    B, hq, hkv, D = (case[k] for k in ("B", "hq", "hkv", "D"))
    seq = g.shuffled(_lens(case))
    table, pages = _tables(g, seq.tolist(), case["page"])
    s = {"case": case, "seq_lens": seq, "block_table": table, "scale": D ** -0.5}
    s["q"] = (1.5 * g.normal(B, hq, D)).to(_DT[case["q"]])
    s["out"] = torch.empty_like(s["q"])
    _caches(g, s, pages)
    if own:
        s["ws"] = _binding().new_attn_workspace(B, hq, hkv, D)
    return s


def _prepare_project(case, g):
    T, d, N, r, na = (case[k] for k in ("T", "d", "N", "r", "adapters"))
    x, w = g.normal(T, d), g.normal(N, d, std=0.02)
    s = {"case": case, "x_scale": None, "w_scale": None, "lora": None, "adapter": None}
    if case["x"] == "e4m3":
        s["x_scale"] = x.abs().amax(1) / E4M3_MAX
        s["w_scale"] = w.abs().amax(1) / E4M3_MAX
        s["x"], s["w"] = _to_e4m3(x / s["x_scale"][:, None]), _to_e4m3(w / s["w_scale"][:, None])
    else:
        s["x"], s["w"] = x.to(_DT[case["x"]]), w.to(torch.bfloat16)
    if _with_adapters(case):
        a = g.normal(na, r, d, std=0.02).to(torch.bfloat16)
        b = g.normal(na, N, r, std=0.02).to(torch.bfloat16)
        s["lora"] = (a, b, 1.0 + g.uniform(na))
        s["adapter"] = g.shuffled(_adapter_of(case))
    s["y"] = torch.empty((T, N), dtype=_DT[case["y"]], device="cuda")
    if own:
        s["ws"] = _binding().new_lora_workspace(T, d, r)
    return s


# ------------------------------------------------------------------- passes


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_norm(s):
    _binding().moe_rmsnorm(s["x"], s["weight"], EPS, s["y"], residual=s["residual"], residual_out=s["residual_out"],
                           y_scale=s["y_scale"])
    return {"y": s["y"], "scale": s["y_scale"], "sum": s["residual_out"]}


def _own_append(s):
    _binding().moe_kv_append(s["k"], s["v"], s["cache"], s["block_table"], s["positions"], req=s["req"],
                             cos_sin=s["cos_sin"], q=s["q"], q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_attn(s):
    c = s["case"]
    _binding().moe_attn_decode(s["q"], s["cache"], s["block_table"], s["seq_lens"], s["scale"], s["out"], s["ws"],
                               window=c["window"], softcap=c["softcap"])
    return s["out"]


def _own_project(s):
    _binding().moe_lora_project(s["x"], s["w"], s["y"], s["ws"], lora=s["lora"], adapter=s["adapter"],
                                x_scale=s["x_scale"], w_scale=s["w_scale"])
    return s["y"]


def _plain_norm(s):
    c, T = s["case"], s["case"]["T"]
    z = s["x"].float()
    out = {"sum": None, "scale": None}
    if c["residual"]:
        z = z + s["residual"].float()
        out["sum"] = z.to(s["x"].dtype)
    y = z * torch.rsqrt((z * z).mean(1, keepdim=True) + EPS) * s["weight"].float()
    if c["y"] == "e4m3":
        blocks = y.view(T, -1, c["group"] or c["d"])
        amax = blocks.abs().amax(2)
        scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        y = _to_e4m3(blocks / scale[:, :, None]).view(T, -1)
        out["scale"] = scale.view(s["y_scale"].shape)
    out["y"] = y.to(_DT[c["y"]])
    return out


def _rotated(v, cos_sin, pos, rot):
    if not rot:
        return v
    h = rot // 2
    cs = cos_sin[pos.long()]
    cos, sin = cs[:, None, :h], cs[:, None, h:]
    a, b = v[..., :h], v[..., h:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, v[..., rot:]], dim=-1)


def _put(cache, page, offset, rows, scale):
    if scale is not None:
        cache.view(torch.uint8)[page, offset] = _to_e4m3(rows / scale[:, None]).view(torch.uint8)
    else:
        cache[page, offset] = rows.to(cache.dtype)


def _plain_append(s):
    c, pos = s["case"], s["positions"]
    req = s["req"].long() if s["req"] is not None else torch.arange(c["T"], device="cuda")
    page = s["block_table"][req, (pos // c["page"]).long()].long()
    offset = (pos % c["page"]).long()
    _put(s["k_cache"], page, offset, _rotated(s["k"].float(), s["cos_sin"], pos, c["rot"]), s["k_scale"])
    _put(s["v_cache"], page, offset, s["v"].float(), s["v_scale"])
    q = _rotated(s["q"].float(), s["cos_sin"], pos, c["rot"]).to(s["q"].dtype)
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _gathered(cache, page, offset, scale):
    if scale is not None:
        return cache.view(torch.uint8)[page, offset].view(torch.float8_e4m3fn).float() * scale[:, None]
    return cache[page, offset].float()


def _plain_attn(s):
    c = s["case"]
    B, hq, hkv, D = c["B"], c["hq"], c["hkv"], c["D"]
    n = s["seq_lens"].long()[:, None]
    at = torch.arange(s["block_table"].shape[1] * c["page"], device="cuda")
    page = s["block_table"].clamp(min=0)[:, at // c["page"]].long()
    k = _gathered(s["k_cache"], page, at % c["page"], s["k_scale"])
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    score = torch.einsum("bhgd,blhd->bhgl", q, k) * s["scale"]
    del k
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    seen = at < n
    if c["window"]:
        seen = seen & (at >= n - c["window"])
    seen = seen[:, None, None, :]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    v = _gathered(s["v_cache"], page, at % c["page"], s["v_scale"])
    # what an unwritten slot holds takes no part, whatever it is
    v = torch.where(seen[:, 0, 0, :, None, None], v, torch.zeros_like(v))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, hq, D).to(s["out"].dtype)


def _plain_project(s):
    x, w = s["x"].float(), s["w"].float()
    if s["x_scale"] is not None:
        x, w = x * s["x_scale"][:, None], w * s["w_scale"][:, None]
    y = x @ w.t()
    if s["lora"] is not None:
        a, b, scale = s["lora"]
        at = s["adapter"].clamp(min=0).long()
        v = torch.einsum("trd,td->tr", a[at].float(), x)
        low = torch.einsum("tnr,tr->tn", b[at].float(), v) * scale[at][:, None]
        y = y + torch.where((s["adapter"] >= 0)[:, None], low, torch.zeros_like(low))
    return y.to(s["y"].dtype)


_OWN = {"norm": _own_norm, "append": _own_append, "attn": _own_attn, "project": _own_project}
_PLAIN = {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn, "project": _plain_project}


# --------------------------------------------------------------------- work


def work(case):
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        b = T * d * (_SIZE[case["x"]] * (3 if case["residual"] else 1) + _SIZE[case["y"]]) + 2 * d
        if case["y"] == "e4m3":
            b += 4 * T * (d // case["group"] if case["group"] else 1)
        return {"bytes": b, "flops": 4 * T * d}
    if case["op"] == "append":
        T, hq, hkv, D = (case[k] for k in ("T", "hq", "hkv", "D"))
        values = T * D
        b = values * _SIZE[case["x"]] * (2 * hq + 2 * hkv) + values * 2 * hkv * _SIZE[case["cache"]]
        b += 4 * T * (1 if case["R"] == T else 2) + 4 * case["rot"] * (T // case["R"])
        return {"bytes": b, "flops": 3 * T * (hq + hkv) * case["rot"] + 1}
    if case["op"] == "attn":
        B, hq, hkv, D = (case[k] for k in ("B", "hq", "hkv", "D"))
        seen = sum(_seen(case, n) for n in _lens(case))
        pages = sum(-(-_seen(case, n) // case["page"]) for n in _lens(case))
        b = 2 * seen * hkv * D * _SIZE[case["cache"]] + 2 * B * hq * D * _SIZE[case["q"]] + 4 * (pages + B)
        return {"bytes": b, "flops": 4 * seen * hq * D}
    T, d, N, r = (case[k] for k in ("T", "d", "N", "r"))
    size = _SIZE[case["x"]] if case["x"] == "e4m3" else 2
    b = N * d * size + T * d * _SIZE[case["x"]] + T * N * _SIZE[case["y"]]
    f = 2 * T * N * d
    if case["x"] == "e4m3":
        b += 4 * (N + T)
    if _with_adapters(case):
        ids = [i for i in _adapter_of(case) if i >= 0]
        b += len(set(ids)) * r * (d + N) * 2 + 4 * T
        f += 2 * len(ids) * r * (d + N)
    return {"bytes": b, "flops": f}


# -------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attn, "project": _exact_project}[case["op"]](s)


def _exact_norm(s):
    c = s["case"]
    ys, sums, scales = [], [], []
    for t in range(0, c["T"], 512):
        z = s["x"][t:t + 512].double()
        if c["residual"]:
            z = z + s["residual"][t:t + 512].double()
            sums.append(z)
        y = z / ((z.square().sum(1) / c["d"] + EPS).sqrt())[:, None] * s["weight"].double()
        if c["y"] == "e4m3":
            y = y.unflatten(1, (-1, c["group"] or c["d"]))
            top = y.abs().amax(2)
            scale = (top / E4M3_MAX).masked_fill(top == 0, 1.0)
            scales.append(scale)
            y = (y / scale[..., None]).flatten(1)
        ys.append(y)
    return {"y": torch.cat(ys), "sum": torch.cat(sums) if sums else None,
            "scale": torch.cat(scales).view(s["y_scale"].shape) if scales else None}


def _exact_turn(v, s):
    """Each pair (i, i + rot/2) as a complex number, turned by its angle."""
    h = s["case"]["rot"] // 2
    if not h:
        return v
    cs = s["cos_sin"].double()[s["positions"].long()]
    z = torch.complex(v[..., :h], v[..., h:2 * h]) * torch.complex(cs[:, :h], cs[:, h:])[:, None]
    return torch.cat([z.real, z.imag, v[..., 2 * h:]], dim=-1)


def _exact_append(s):
    c = s["case"]
    T, page = c["T"], c["page"]
    req = (s["req"] if s["req"] is not None else torch.arange(T, device="cuda")).long()
    pos = s["positions"].long()
    slot = s["block_table"].long()[req, torch.div(pos, page, rounding_mode="floor")] * page + pos.remainder(page)
    out = {"q": _exact_turn(s["q"].double(), s)}
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        flat = cache.to(torch.float32).double().contiguous().flatten(0, 1)
        rows = s[name].double()
        if name == "k":
            rows = _exact_turn(rows, s)
        if s[name + "_scale"] is not None:
            rows = rows / s[name + "_scale"].double()[:, None]
            rows = rows.clamp(-E4M3_MAX, E4M3_MAX)
        flat[slot] = rows
        out[name] = flat.view(cache.shape)
    return out


def _exact_attn(s):
    c = s["case"]
    hq, hkv, D, page = c["hq"], c["hkv"], c["D"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["seq_lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == first:
            continue
        at = torch.arange(first, n, device="cuda")
        slot = s["block_table"][b].long()[at // page]
        rows = []
        for name in ("k", "v"):
            cache = s[name + "_cache"]
            if cache.dtype == torch.float8_e4m3fn:
                kv = cache.view(torch.uint8)[slot, at % page].view(torch.float8_e4m3fn).to(torch.float32).double()
                kv = kv * s[name + "_scale"].double()[None, :, None]
            else:
                kv = cache[slot, at % page].double()
            rows.append(kv.transpose(0, 1))
        k, v = rows
        q = s["q"][b].double().unflatten(0, (hkv, hq // hkv))
        score = (q @ k.transpose(1, 2)) * s["scale"]
        if c["softcap"]:
            score = torch.tanh(score / c["softcap"]) * c["softcap"]
        out[b] = (torch.softmax(score, -1) @ v).flatten(0, 1)
    return out


def _exact_project(s):
    x, w = s["x"].to(torch.float32).double(), s["w"].to(torch.float32).double()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].double()[:, None]
        w = w * s["w_scale"].double()[:, None]
    y = torch.mm(x, w.t())
    if s["lora"] is not None:
        a, b, scale = s["lora"]
        for t, i in enumerate(s["adapter"].tolist()):
            if i >= 0:
                y[t] += scale[i].double() * (b[i].double() @ (a[i].double() @ x[t]))
    return y

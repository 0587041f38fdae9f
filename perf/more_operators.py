"""Timed cases of the operators for long contexts in a decode block.

Five operators, each in two forms.  With ``own`` false, ``run`` computes an
operator in its plain form: elementary torch operations in fp32, rounded once
at the end.  With ``own`` true it makes the library calls:

- ``append``: root-mean-square norm of every head of q and k, rotation by
              positions of one or several axes, and k, v written into the paged
              cache (``moe_qk_norm_append``);
- ``bounds``: per channel the least and greatest key of each page
              (``moe_page_bounds``);
- ``scores``: for each page and key-value head an upper bound of what the new
              token's queries can score in it (``moe_page_scores``);
- ``select``: the pages with the best scores, with the request's first and
              last ones, as a table per key-value head (``moe_page_select``);
- ``attn``:   attention of one new token per request over a table of pages per
              key-value head (``moe_attn_pages``).

Sizes are those of the layer shapes in ``moe_decode_layer_fp32_gb300/synth.py``
(d = 2048 and 7168, 1 to 128 tokens) with d / 128 query heads and 2 to 8
key-value heads, and contexts of up to 131072 tokens.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
THETA = 1000000.0


def _binding():
    from moe_decode_layer_fp32_gb300 import binding
    return binding


_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases


def listed():
    return [
        # One stream of the 2048-wide model, text only: latency.
        {"name": "append-1-bf16", "op": "append", "T": 1, "R": 1, "hq": 16, "hkv": 4, "D": 128, "rot": 128, "axes": 1,
         "page": 16, "x": "bf16", "cache": "bf16", "heads_first": False},
        # 97 streams with images in their prompts: positions of time, height and width.
        {"name": "append-97-f32-axes", "op": "append", "T": 97, "R": 97, "hq": 16, "hkv": 4, "D": 128, "rot": 128,
         "axes": 3, "page": 32, "x": "f32", "cache": "bf16", "heads_first": False},
        # Prompts of five videos of the 7168-wide model, E4M3 cache.
        {"name": "append-12345-e4m3-axes", "op": "append", "T": 12345, "R": 5, "hq": 56, "hkv": 8, "D": 128, "rot": 64,
         "axes": 3, "page": 64, "x": "bf16", "cache": "e4m3", "heads_first": True},
        # A decode step of 33 requests: only the page that each has just written to.
        {"name": "bounds-33-new", "op": "bounds", "B": 33, "L": 4096, "ragged": True, "new": 1, "hkv": 4, "D": 128,
         "page": 32, "cache": "bf16", "heads_first": False},
        # Seven prompts after their append, all pages.
        {"name": "bounds-7x16383", "op": "bounds", "B": 7, "L": 16383, "ragged": False, "new": 0, "hkv": 8, "D": 128,
         "page": 64, "cache": "bf16", "heads_first": True},
        # One document of 128k tokens.
        {"name": "scores-1x131071", "op": "scores", "B": 1, "L": 131071, "ragged": False, "hq": 16, "hkv": 4, "D": 128,
         "page": 64, "q": "f32", "cache": "bf16"},
        # The largest batch with long, uneven contexts, E4M3 cache.
        {"name": "scores-128x32768-e4m3", "op": "scores", "B": 128, "L": 32768, "ragged": True, "hq": 56, "hkv": 8,
         "D": 128, "page": 32, "q": "bf16", "cache": "e4m3"},
        # The pages of one document of 128k tokens, 64 of 2048 kept.
        {"name": "select-1x2048", "op": "select", "B": 1, "L": 131071, "ragged": False, "hkv": 4, "page": 64, "keep": 64,
         "sinks": 1, "recent": 2},
        # The largest batch, small pages, 128 of up to 2048 kept.
        {"name": "select-128x2048", "op": "select", "B": 128, "L": 32768, "ragged": True, "hkv": 8, "page": 16,
         "keep": 128, "sinks": 4, "recent": 8},
        # One document of the 2048-wide model, 2048 keys of it: latency.
        {"name": "attn-1x32-pages", "op": "attn", "B": 1, "L": 131071, "ragged": False, "hq": 16, "hkv": 4, "D": 128,
         "page": 64, "keep": 32, "q": "f32", "cache": "bf16", "heads_first": False, "softcap": 0.0},
        # A serving batch of mixed lengths, two slots of it idle or new.
        {"name": "attn-16x64-pages", "op": "attn", "B": 16, "L": 32768, "ragged": True, "hq": 56, "hkv": 8, "D": 128,
         "page": 32, "keep": 64, "q": "bf16", "cache": "bf16", "heads_first": True, "softcap": 0.0},
        # The largest batch, E4M3 cache.
        {"name": "attn-128x64-pages-e4m3", "op": "attn", "B": 128, "L": 16384, "ragged": True, "hq": 56, "hkv": 8,
         "D": 128, "page": 64, "keep": 64, "q": "bf16", "cache": "e4m3", "heads_first": False, "softcap": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "bounds", "scores", "select", "attn", "attn"])
    D = rng.choice([64, 80, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 16] if D < 256 else [1, 2, 4])
    page = rng.choice([16, 24, 32, 64, 128])
    cache, x = rng.choice(["bf16", "e4m3"]), rng.choice(["f32", "bf16"])
    if op == "append":
        R = _log(rng, 1, 128)
        hq = hkv * (group if D < 256 else 1)
        token = D * (2 * (hq + hkv) * _SIZE[x] + 2 * hkv * _SIZE[cache])
        most = max(R, min(12345, 430000000 // token))
        rot = rng.choice([D // 2, D, D])
        return {"op": op, "T": R * _log(rng, 1, max(1, most // R)), "R": R, "hq": hq, "hkv": hkv, "D": D, "rot": rot,
                "axes": rng.choice([1, 2, 3, 4]), "page": rng.choice([1, page]), "x": x, "cache": cache,
                "heads_first": rng.random() < 0.5}
    B = _log(rng, 1, 128)
    if op == "bounds":
        L = _log(rng, 1, min(131072, 7 * 16383 * 8 * 128 // (B * hkv * D)))
        return {"op": op, "B": B, "L": L, "ragged": rng.random() < 0.7, "new": rng.choice([0, 1, 1, 5]), "hkv": hkv,
                "D": D, "page": page, "cache": cache, "heads_first": rng.random() < 0.5}
    if op == "scores":
        L = _log(rng, 1, min(131072, 128 * 32768 // 3 * 8 * 128 // 32 * page // (B * hkv * D * _SIZE[cache])))
        return {"op": op, "B": B, "L": L, "ragged": rng.random() < 0.7, "hq": hkv * group, "hkv": hkv, "D": D,
                "page": page, "q": x, "cache": cache}
    if op == "select":
        keep = _log(rng, 1, 256)
        sinks = min(rng.choice([0, 1, 4]), keep - 1)
        return {"op": op, "B": B, "L": _log(rng, 1, min(131072, 128 * 32768 // 3 * 8 // 16 * page // (B * hkv))),
                "ragged": rng.random() < 0.7, "hkv": hkv, "page": page, "keep": keep, "sinks": sinks,
                "recent": min(rng.choice([0, 1, 2, 8]), keep - sinks)}
    # no more pages than the largest listed case, and no more cached values
    keep = _log(rng, 1, max(1, min(16384, 128 * 8 * 4096 * 128 // (2 * B * hkv * D)) // page))
    L = _log(rng, 1, min(131072, 128 * 16384 * 8 * 128 // (3 * B * hkv * D)))
    return {"op": op, "B": B, "L": L, "ragged": rng.random() < 0.7, "hq": hkv * group, "hkv": hkv, "D": D, "page": page,
            "keep": keep, "q": x, "cache": cache, "heads_first": rng.random() < 0.5,
            "softcap": rng.choice([0.0, 0.0, 30.0])}


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


def _pages(n, page):
    return -(-n // page)


def _first(case, n):
    """The first token of a request that ``bounds`` has not seen."""
    return max(0, n - case["new"]) if case["new"] else 0


def _kept_keys(case, n):
    """Keys in the pages that a request of n tokens keeps, its last page among them."""
    pages = _pages(n, case["page"])
    return n - (pages - min(pages, case["keep"])) * case["page"]


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


def _to_e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _channels(g, D):
    """Keys have channels with a mean of their own and a few much larger than the others."""
    return 1.0 + 7.0 * (g.uniform(D) < 0.03).float(), g.normal(D, std=0.5)


def _cache(g, pages, page, heads, D, dtype, heads_first, keys):
    """(cache viewed as [pages, page, heads, D], scale per head or None)."""
    shape = (pages, heads, page, D) if heads_first else (pages, page, heads, D)
    values = torch.empty(shape, dtype=_DT[dtype], device="cuda")
    scale = (0.5 + g.uniform(heads)) * ((40.0 if keys else 5.0) / E4M3_MAX) if dtype == "e4m3" else None
    std, mean = _channels(g, D) if keys else (1.0, 0.0)
    per = max(1, (1 << 26) // (page * heads * D))
    for p in range(0, pages, per):
        v = (g.normal(*((min(per, pages - p),) + shape[1:])) + mean) * std
        if scale is not None:
            v = _to_e4m3(v / (scale[:, None, None] if heads_first else scale[:, None]))
        values[p:p + per].copy_(v)
    return (values.transpose(1, 2) if heads_first else values), scale


def _caches(g, s, pages, values=True):
    """One layer's key and value caches, and the library's handle of them."""
    case = s["case"]
    for name in ("k", "v"):
        if name == "v" and not values:
            # a call that reads no values has them all the same, in the least room
            s["v_cache"], s["v_scale"] = s["k_cache"], s["k_scale"]
            continue
        s[name + "_cache"], s[name + "_scale"] = _cache(g, pages, case["page"], case["hkv"], case["D"], case["cache"],
                                                        case.get("heads_first", False), name == "k")
    if own:
        s["cache"] = _binding().KvCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def _tables(g, counts, page, spare=1):
    """Block table [R, most] of requests with ``counts`` tokens: pages in random order, -1 past a request's last."""
    need = [_pages(c, page) for c in counts]
    pages, width = sum(need) + spare, max(max(need), 1)
    ids = g.perm(pages).to(torch.int32)
    slots = torch.tensor(need, device="cuda")
    first = torch.cumsum(slots, 0) - slots
    col = torch.arange(width, device="cuda")
    table = ids[(first[:, None] + col).clamp(max=pages - 1)]
    return torch.where(col < slots[:, None], table, torch.full_like(table, -1)).contiguous(), pages


def prepare(case, seed):
    g = _Draws(seed)
    return {"append": _prepare_append, "bounds": _prepare_bounds, "scores": _prepare_scores,
            "select": _prepare_select, "attn": _prepare_attn}[case["op"]](case, g)


def _prepare_append(case, g):
    T, R, hq, hkv, D, A = (case[k] for k in ("T", "R", "hq", "hkv", "D", "axes"))
    # each request gets T / R new tokens after the ones it has
    new = T // R
    old = [(37 * i) % 100 for i in range(R)]
    g.host.shuffle(old)
    req = torch.tensor([t % R for t in range(T)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([old[t % R] + t // R for t in range(T)], dtype=torch.int32, device="cuda")
    table, pages = _tables(g, [o + new for o in old], case["page"])
    # one q, k, v projection's output, sliced by heads
    qkv = (g.normal(T, hq + 2 * hkv, D) * (0.5 + 2.0 * g.uniform(T, hq + 2 * hkv, 1))).to(_DT[case["x"]])
    s = {"case": case, "req": req if R != T else None, "positions": pos, "block_table": table,
         "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:]}
    s["q_weight"] = (1.0 + 0.2 * g.normal(D)).to(torch.bfloat16)
    s["k_weight"] = (1.0 + 0.2 * g.normal(D)).to(torch.bfloat16)
    s["q_out"] = torch.empty((T, hq, D), dtype=_DT[case["x"]], device="cuda")
    half = case["rot"] // 2
    freq = THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(max(old) + new, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float()
    s["axis_positions"] = s["axis"] = None
    if A > 1:
        # frames of 24 x 20 patches: time moves on with the frame, height and width within it; a fourth
        # axis counts the frames' tiles
        at = pos.long()
        axes = [at // 480, at // 20 % 24, at % 20, at // 120 % 4][:A]
        s["axis_positions"] = torch.stack(axes).to(torch.int32).contiguous()
        # the slow pairs belong to time, the fast ones to the places in turn
        s["axis"] = bytes((0 if A == 1 or 4 * i >= 3 * half else i % A) for i in range(half))
    _caches(g, s, pages)
    return s


def _prepare_bounds(case, g):
    lens = g.shuffled(_lens(case))
    table, pages = _tables(g, lens.tolist(), case["page"])
    s = {"case": case, "seq_lens": lens, "block_table": table, "pages": pages}
    s["first"] = (lens - case["new"]).clamp(min=0).to(torch.int32) if case["new"] else None
    _caches(g, s, pages, values=False)
    s["bounds"] = torch.zeros((pages, case["hkv"], 2, case["D"]), dtype=_DT[case["cache"]], device="cuda")
    return s


def _prepare_scores(case, g):
    B, hq, hkv, D = (case[k] for k in ("B", "hq", "hkv", "D"))
    lens = g.shuffled(_lens(case))
    table, pages = _tables(g, lens.tolist(), case["page"])
    s = {"case": case, "seq_lens": lens, "block_table": table, "q": (1.5 * g.normal(B, hq, D)).to(_DT[case["q"]])}
    # what moe_page_bounds leaves: of a few normal keys, the least and the greatest
    scale = (0.5 + g.uniform(hkv)) * (40.0 / E4M3_MAX) if case["cache"] == "e4m3" else None
    std, mean = _channels(g, D)
    s["bounds"] = torch.empty((pages, hkv, 2, D), dtype=_DT[case["cache"]], device="cuda")
    per = max(1, (1 << 25) // (hkv * D))
    for p in range(0, pages, per):
        n = min(per, pages - p)
        mid, wide = g.normal(n, hkv, D, std=0.4) + mean, 1.5 + g.uniform(n, hkv, D)
        v = torch.stack([(mid - wide) * std, (mid + wide) * std], dim=2)
        s["bounds"][p:p + n].copy_(_to_e4m3(v / scale[:, None, None]) if scale is not None else v)
    s["k_scale"] = scale
    s["scores"] = torch.full((B, hkv, table.shape[1]), -math.inf, device="cuda")
    if own:
        # the handle of a cache of these pages; the call reads its sizes and scales, not its rows
        k = torch.empty((pages, case["page"], hkv, D), dtype=_DT[case["cache"]], device="cuda")
        s["cache"] = _binding().KvCache(k, k, scale, scale)
    return s


def _prepare_select(case, g):
    lens = g.shuffled(_lens(case))
    table, pages = _tables(g, lens.tolist(), case["page"])
    B, hkv, n = case["B"], case["hkv"], table.shape[1]
    scores = 40.0 + 12.0 * g.normal(B, hkv, n)
    # pages of a repeated text have equal scores
    same = (g.uniform(B, hkv, n) * n).long().clamp(max=n - 1)
    scores = torch.where(g.uniform(B, hkv, n) < 0.2, scores.gather(2, same), scores)
    return {"case": case, "seq_lens": lens, "block_table": table, "scores": scores.contiguous(),
            "tables": torch.empty((B, hkv, case["keep"]), dtype=torch.int32, device="cuda"),
            "lens": torch.empty((B, hkv), dtype=torch.int32, device="cuda")}


def _prepare_attn(case, g):
    B, hq, hkv, D, P, keep = (case[k] for k in ("B", "hq", "hkv", "D", "page", "keep"))
    lens = g.shuffled(_lens(case))
    table, pages = _tables(g, lens.tolist(), P)
    # what moe_page_select leaves: some pages of each request in order, the last one among them
    have = (lens.long() + P - 1) // P
    width = table.shape[1]
    rank = g.uniform(B, hkv, max(width, keep))
    col = torch.arange(rank.shape[2], device="cuda")
    rank = torch.where(col == (have - 1)[:, None, None], torch.full_like(rank, 2.0), rank)
    rank = torch.where(col < have[:, None, None], rank, torch.full_like(rank, -1.0))
    best, at = rank.topk(keep, dim=2)
    at = torch.where(best >= 0, at, torch.full_like(at, 1 << 30)).sort(dim=2).values
    chosen = torch.gather(table.long()[:, None].expand(B, hkv, width), 2, at.clamp(max=width - 1))
    s = {"case": case, "scale": D ** -0.5,
         "tables": torch.where(at < (1 << 30), chosen, torch.full_like(chosen, -1)).to(torch.int32).contiguous(),
         "lens": (lens.long() - (have - have.clamp(max=keep)) * P)[:, None].expand(B, hkv).to(torch.int32).contiguous()}
    s["q"] = (1.5 * g.normal(B, hq, D)).to(_DT[case["q"]])
    s["out"] = torch.empty_like(s["q"])
    _caches(g, s, pages)
    if own:
        s["ws"] = _binding().new_attn_workspace(B, hq, hkv, D)
    return s


# ------------------------------------------------------------------- passes


def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_append(s):
    _binding().moe_qk_norm_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["cache"],
                                  s["block_table"], s["positions"], s["q_out"], req=s["req"], cos_sin=s["cos_sin"],
                                  axis_positions=s["axis_positions"], axis=s["axis"])
    return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}


def _own_bounds(s):
    _binding().moe_page_bounds(s["cache"], s["bounds"], s["block_table"], s["seq_lens"], first=s["first"])
    return s["bounds"]


def _own_scores(s):
    _binding().moe_page_scores(s["q"], s["cache"], s["bounds"], s["block_table"], s["seq_lens"], s["scores"])
    return s["scores"]


def _own_select(s):
    c = s["case"]
    _binding().moe_page_select(s["scores"], s["block_table"], s["seq_lens"], c["page"], s["tables"], s["lens"],
                               sinks=c["sinks"], recent=c["recent"])
    return {"tables": s["tables"], "lens": s["lens"]}


def _own_attn(s):
    _binding().moe_attn_pages(s["q"], s["cache"], s["tables"], s["lens"], s["scale"], s["out"], s["ws"],
                              softcap=s["case"]["softcap"])
    return s["out"]


def _normed(x, weight):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _turned(v, cos, sin, half):
    a, b = v[..., :half], v[..., half:2 * half]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, v[..., 2 * half:]], dim=-1)


def _put(cache, page, offset, rows, scale):
    if scale is not None:
        cache.view(torch.uint8)[page, offset] = _to_e4m3(rows / scale[:, None]).view(torch.uint8)
    else:
        cache[page, offset] = rows.to(cache.dtype)


def _plain_append(s):
    c, pos = s["case"], s["positions"].long()
    half = c["rot"] // 2
    req = s["req"].long() if s["req"] is not None else torch.arange(c["T"], device="cuda")
    pair = torch.arange(half, device="cuda")
    if s["axis"] is None:
        row = pos[:, None].expand(-1, half)
    else:
        row = s["axis_positions"].long()[torch.tensor(list(s["axis"]), device="cuda")].t()
    cos, sin = s["cos_sin"][row, pair][:, None], s["cos_sin"][row, half + pair][:, None]
    page = s["block_table"][req, pos // c["page"]].long()
    offset = pos % c["page"]
    _put(s["k_cache"], page, offset, _turned(_normed(s["k"], s["k_weight"]), cos, sin, half), s["k_scale"])
    _put(s["v_cache"], page, offset, s["v"].float(), s["v_scale"])
    q = _turned(_normed(s["q"], s["q_weight"]), cos, sin, half).to(s["q"].dtype)
    return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}


def _plain_bounds(s):
    c, P = s["case"], s["case"]["page"]
    n = s["seq_lens"].long()
    first = s["first"].long() if s["first"] is not None else torch.zeros_like(n)
    cols = torch.arange(s["block_table"].shape[1], device="cuda")
    b, col = torch.nonzero((cols * P < n[:, None]) & (cols * P + P > first[:, None]) & (first < n)[:, None], as_tuple=True)
    page = s["block_table"][b, col].long()
    slot = torch.arange(P, device="cuda")
    seen = (col[:, None] * P + slot < n[b, None])[:, :, None, None]
    if s["k_scale"] is not None:
        k = s["k_cache"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
    else:
        k = s["k_cache"][page].float()
    lo = torch.where(seen, k, math.inf).amin(1)
    hi = torch.where(seen, k, -math.inf).amax(1)
    found = torch.stack([lo, hi], dim=2).to(s["bounds"].dtype)
    if s["k_scale"] is not None:
        s["bounds"].view(torch.uint8)[page] = found.view(torch.uint8)
    else:
        s["bounds"][page] = found
    return s["bounds"]


def _plain_scores(s):
    c = s["case"]
    B, hq, hkv, D = c["B"], c["hq"], c["hkv"], c["D"]
    cols = torch.arange(s["block_table"].shape[1], device="cuda")
    page = s["block_table"].long().clamp(min=0)
    if s["k_scale"] is not None:
        edge = s["bounds"].view(torch.uint8)[page].view(torch.float8_e4m3fn).float() * s["k_scale"][:, None, None]
    else:
        edge = s["bounds"][page].float()
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    up, down = q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)
    found = torch.einsum("bgd,bjgd->bgj", down, edge[:, :, :, 0]) + torch.einsum("bgd,bjgd->bgj", up, edge[:, :, :, 1])
    seen = (cols * c["page"] < s["seq_lens"].long()[:, None])[:, None]
    return torch.where(seen, found, s["scores"])


def _plain_select(s):
    c, P, keep = s["case"], s["case"]["page"], s["case"]["keep"]
    n = s["seq_lens"].long()[:, None, None]
    pages = (n + P - 1) // P
    width = s["scores"].shape[2]
    cols = torch.arange(width, device="cuda")
    must = (cols < c["sinks"]) | (cols >= pages - c["recent"])
    score = torch.where(must, math.inf, s["scores"])
    score = torch.where(cols < pages, score, -math.inf)
    order = score.sort(dim=2, descending=True, stable=True).indices
    if width < keep:
        order = torch.nn.functional.pad(order, (0, keep - width), value=width)
    order = order[:, :, :keep]
    order = torch.where(order < pages, order, torch.full_like(order, 1 << 30)).sort(dim=2).values
    kept = order < (1 << 30)
    table = s["block_table"].long()[:, None].expand(-1, order.shape[1], -1)
    tables = torch.where(kept, table.gather(2, order.clamp(max=width - 1)), -1).to(torch.int32)
    keys = torch.where(kept, (n - order * P).clamp(max=P), 0)
    return {"tables": tables, "lens": keys.sum(2).to(torch.int32)}


def _rows(cache, page, slot, head, scale):
    if scale is not None:
        return cache.view(torch.uint8)[page, slot, head].view(torch.float8_e4m3fn).float() * scale[:, None, None]
    return cache[page, slot, head].float()


def _plain_attn(s):
    c = s["case"]
    B, hq, hkv, D, P = c["B"], c["hq"], c["hkv"], c["D"], c["page"]
    at = torch.arange(c["keep"] * P, device="cuda")
    page = s["tables"].long().clamp(min=0)[:, :, at // P]
    head = torch.arange(hkv, device="cuda")[:, None]
    seen = at < s["lens"].long()[:, :, None]
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    score = torch.einsum("bghd,bgld->bghl", q, _rows(s["k_cache"], page, at % P, head, s["k_scale"])) * s["scale"]
    if c["softcap"]:
        score = c["softcap"] * torch.tanh(score / c["softcap"])
    score = torch.where(seen[:, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    # what an unwritten slot holds takes no part, whatever it is
    v = torch.where(seen[..., None], _rows(s["v_cache"], page, at % P, head, s["v_scale"]), 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bghl,bgld->bghd", p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.view(B, hq, D).to(s["out"].dtype)


_OWN = {"append": _own_append, "bounds": _own_bounds, "scores": _own_scores, "select": _own_select, "attn": _own_attn}
_PLAIN = {"append": _plain_append, "bounds": _plain_bounds, "scores": _plain_scores, "select": _plain_select,
          "attn": _plain_attn}


# --------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "append":
        T, hq, hkv, D, rot, A = (case[k] for k in ("T", "hq", "hkv", "D", "rot", "axes"))
        b = T * D * _SIZE[case["x"]] * (2 * hq + 2 * hkv) + T * D * 2 * hkv * _SIZE[case["cache"]]
        b += 4 * T * (1 if case["R"] == T else 2) + 4 * T * (A if A > 1 else 0) + 4 * D
        rows = T // case["R"] if A == 1 else min(T // case["R"], 24)
        return {"bytes": b + 4 * rot * rows, "flops": T * (hq + hkv) * (4 * D + 3 * rot)}
    page, hkv = case["page"], case["hkv"]
    if op == "bounds":
        D, size = case["D"], _SIZE[case["cache"]]
        rows = pages = 0
        for n in _lens(case):
            if n:
                col = _first(case, n) // page
                rows += n - col * page
                pages += _pages(n, page) - col
        b = (rows + 2 * pages) * hkv * D * size + 4 * pages + 8 * case["B"]
        return {"bytes": b, "flops": 2 * rows * hkv * D}
    pages = sum(_pages(n, page) for n in _lens(case))
    if op == "scores":
        B, hq, D = (case[k] for k in ("B", "hq", "D"))
        b = pages * hkv * 2 * D * _SIZE[case["cache"]] + B * hq * D * _SIZE[case["q"]] + 4 * pages * (hkv + 1) + 4 * B
        return {"bytes": b, "flops": 4 * pages * hkv * D + 2 * B * hq * D}
    if op == "select":
        kept = sum(min(_pages(n, page), case["keep"]) for n in _lens(case))
        b = 4 * pages * hkv + 4 * kept * (hkv + 1) + 4 * case["B"] * (hkv + 1)
        return {"bytes": b, "flops": pages * hkv}
    B, hq, D = (case[k] for k in ("B", "hq", "D"))
    keys = sum(_kept_keys(case, n) for n in _lens(case)) * hkv
    kept = sum(min(_pages(n, page), case["keep"]) for n in _lens(case)) * hkv
    b = 2 * keys * D * _SIZE[case["cache"]] + 2 * B * hq * D * _SIZE[case["q"]] + 4 * (kept + B * hkv)
    return {"bytes": b, "flops": 4 * keys * (hq // hkv) * D}


# -------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "scores": _exact_scores, "select": _exact_select,
            "attn": _exact_attn}[case["op"]](s)


def _double(t):
    return t.to(torch.float32).double()


def _exact_append(s):
    c = s["case"]
    T, P, h = c["T"], c["page"], c["rot"] // 2
    req = (s["req"] if s["req"] is not None else torch.arange(T, device="cuda")).long()
    pos = s["positions"].long()
    # each pair (i, i + h) as a complex number, turned by its axis's angle
    turn = torch.empty((T, h), dtype=torch.complex128, device="cuda")
    for i in range(h):
        at = pos if s["axis"] is None else s["axis_positions"][s["axis"][i]].long()
        turn[:, i] = torch.complex(s["cos_sin"][at, i].double(), s["cos_sin"][at, h + i].double())

    def head(x, weight):
        x = _double(x)
        x = x / (x.square().sum(-1) / c["D"] + EPS).sqrt()[..., None] * weight.double()
        z = torch.complex(x[..., :h], x[..., h:2 * h]) * turn[:, None]
        return torch.cat([z.real, z.imag, x[..., 2 * h:]], dim=-1)

    slot = s["block_table"].long()[req, torch.div(pos, P, rounding_mode="floor")] * P + pos.remainder(P)
    out = {"q": head(s["q"], s["q_weight"])}
    for name in ("k", "v"):
        cache = s[name + "_cache"]
        flat = _double(cache).contiguous().flatten(0, 1)
        rows = head(s["k"], s["k_weight"]) if name == "k" else _double(s["v"])
        if s[name + "_scale"] is not None:
            rows = (rows / s[name + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        flat[slot] = rows
        out[name] = flat.view(cache.shape)
    return out


def _exact_bounds(s):
    c, P = s["case"], s["case"]["page"]
    out = _double(s["bounds"])
    k = s["k_cache"].transpose(1, 2)
    first = s["first"].tolist() if s["first"] is not None else [0] * c["B"]
    for b, n in enumerate(s["seq_lens"].tolist()):
        if first[b] >= n:
            continue
        whole = n // P
        ids = s["block_table"][b].long()
        col = first[b] // P
        for a in range(col, whole, 512):
            page = ids[a:min(whole, a + 512)]
            rows = _double(k.view(torch.uint8)[page].view(k.dtype) if k.dtype == torch.float8_e4m3fn else k[page])
            out[page] = torch.stack(torch.aminmax(rows, dim=2), dim=2)
        if n % P:
            rows = _double(k[int(ids[whole])])[:, :n % P]
            out[ids[whole]] = torch.stack([rows.min(1).values, rows.max(1).values], dim=1)
    return out


def _exact_scores(s):
    c = s["case"]
    hq, hkv = c["hq"], c["hkv"]
    out = s["scores"].double()
    for b, n in enumerate(s["seq_lens"].tolist()):
        j = _pages(n, c["page"])
        if not j:
            continue
        page = s["block_table"][b, :j].long()
        edge = s["bounds"]
        edge = edge.view(torch.uint8)[page].view(edge.dtype) if c["cache"] == "e4m3" else edge[page]
        edge = _double(edge)
        if s["k_scale"] is not None:
            edge = edge * s["k_scale"].double()[:, None, None]
        q = _double(s["q"][b]).unflatten(0, (hkv, hq // hkv))
        for h in range(hq // hkv):
            best = torch.maximum(q[:, h] * edge[:, :, 0], q[:, h] * edge[:, :, 1]).sum(-1).t()
            if h == 0:
                out[b, :, :j] = best
            else:
                out[b, :, :j] += best
    return out


def _exact_select(s):
    c, P, keep = s["case"], s["case"]["page"], s["case"]["keep"]
    table, scores = s["block_table"].tolist(), s["scores"].tolist()
    tables = torch.full_like(s["tables"], -1)
    lens = torch.zeros_like(s["lens"])
    kept_all, len_all = [], []
    for b, n in enumerate(s["seq_lens"].tolist()):
        pages = _pages(n, P)
        for g in range(c["hkv"]):
            must = set(range(min(c["sinks"], pages))) | set(range(max(0, pages - c["recent"]), pages))
            rest = sorted((j for j in range(pages) if j not in must), key=lambda j: (-scores[b][g][j], j))
            kept = sorted(must | set(rest[:max(0, keep - len(must))]))
            kept_all.append([table[b][j] for j in kept] + [-1] * (keep - len(kept)))
            len_all.append(sum(min(P, n - j * P) for j in kept))
    tables.copy_(torch.tensor(kept_all, dtype=torch.int32).view(tables.shape))
    lens.copy_(torch.tensor(len_all, dtype=torch.int32).view(lens.shape))
    return {"tables": tables, "lens": lens}


def _exact_attn(s):
    c = s["case"]
    hq, hkv, P = c["hq"], c["hkv"], c["page"]
    group = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, row in enumerate(s["lens"].tolist()):
        for g, n in enumerate(row):
            if n == 0:
                continue
            at = torch.arange(n, device="cuda")
            page = s["tables"][b, g].long()[torch.div(at, P, rounding_mode="floor")]
            kv = []
            for name in ("k", "v"):
                cache = s[name + "_cache"][:, :, g]
                if cache.dtype == torch.float8_e4m3fn:
                    rows = cache.view(torch.uint8)[page, at.remainder(P)].view(cache.dtype)
                    kv.append(_double(rows) * s[name + "_scale"][g].double())
                else:
                    kv.append(cache[page, at.remainder(P)].double())
            score = (s["q"][b, g * group:(g + 1) * group].double() @ kv[0].t()) * s["scale"]
            if c["softcap"]:
                score = torch.tanh(score / c["softcap"]) * c["softcap"]
            out[b, g * group:(g + 1) * group] = torch.softmax(score, -1) @ kv[1]
    return out

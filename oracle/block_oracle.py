"""fp64 CPU oracle of the decode-block operators (test infrastructure only).

Written from the definitions in ``include/moe_block.h``: no code is shared
with the CUDA path.  Inputs are torch tensors (any device, any type); results
are float64 CPU tensors.
"""

from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def f64(t) -> torch.Tensor:
    """Exact float64 copy on the CPU."""
    t = t.detach().cpu()
    return t.to(torch.float32).to(torch.float64) if t.dtype != torch.float64 else t


def rms_norm(x, weight, eps, residual=None):
    """(y, z): z = x + residual, y = z / sqrt(mean z^2 + eps) * weight."""
    z = f64(x)
    if residual is not None:
        z = z + f64(residual)
    y = z / torch.sqrt((z * z).mean(dim=1, keepdim=True) + eps)
    if weight is not None:
        y = y * f64(weight)
    return y, z


def e4m3_scales(y, group):
    """amax / 448 of each row (group 0) or of each ``group`` columns; 1 where it is 0."""
    T, d = y.shape
    amax = y.abs().view(T, -1, group or d).amax(dim=2)
    scale = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return scale if group else scale[:, 0]


def rotate(v, positions, cos_sin):
    """v [T, heads, D] by rows of cos_sin; tokens of negative position stay."""
    v = f64(v).clone()
    if cos_sin is None:
        return v
    half = cos_sin.shape[1] // 2
    for t, p in enumerate(positions.tolist()):
        if p < 0 or p >= cos_sin.shape[0]:
            continue
        c, s = f64(cos_sin[p, :half]), f64(cos_sin[p, half:])
        a, b = v[t, :, :half].clone(), v[t, :, half:2 * half].clone()
        v[t, :, :half] = a * c - b * s
        v[t, :, half:2 * half] = b * c + a * s
    return v


def slot_of(table, req, pos, page_size):
    """(page, slot) of position ``pos`` of request ``req``."""
    return int(table[req, pos // page_size]), pos % page_size


def decode_attention(q, rows, scale, softcap=0.0):
    """One request: q [hq, D]; rows = (k, v), each [n, heads, D] fp64, in cache
    order.  Returns (o [hq, D], lse [hq])."""
    q = f64(q)
    k, v = rows
    hq, D = q.shape
    n, heads, _ = k.shape
    o = torch.zeros(hq, D, dtype=torch.float64)
    lse = torch.full((hq,), -math.inf, dtype=torch.float64)
    if n == 0:
        return o, lse
    for h in range(hq):
        g = h // (hq // heads)
        s = (k[:, g] @ q[h]) * scale
        if softcap > 0:
            s = softcap * torch.tanh(s / softcap)
        lse[h] = torch.logsumexp(s, 0)
        o[h] = torch.exp(s - lse[h]) @ v[:, g]
    return o, lse


def cached_rows(cache, scale, table_row, first, n):
    """fp64 rows [n - first, heads, D] of positions first .. n - 1; cache viewed
    [pages, page_size, heads, D]."""
    page = cache.shape[1]
    at = torch.arange(first, n)
    pages = table_row.cpu().long()[at // page]
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    got = raw[pages.to(cache.device), (at % page).to(cache.device)]
    if cache.dtype == torch.float8_e4m3fn:
        got = got.view(torch.float8_e4m3fn)
    got = f64(got)
    return got * f64(scale)[:, None] if scale is not None else got


def lora_project(x, w, lora=None, adapter=None, x_scale=None, w_scale=None):
    """(y, size): y = W x + s B (A x) and the same sum over absolute values,
    which scales rounding errors."""
    x, w = f64(x), f64(w)
    if x_scale is not None:
        x, w = x * f64(x_scale)[:, None], w * f64(w_scale)[:, None]
    y, size = x @ w.T, x.abs() @ w.abs().T
    if lora is not None:
        A, B, s = (f64(t) for t in lora)
        for t, i in enumerate(adapter.tolist()):
            if 0 <= i < A.shape[0]:
                y[t] += s[i] * (B[i] @ (A[i] @ x[t]))
                size[t] += s[i].abs() * (B[i].abs() @ (A[i].abs() @ x[t].abs()))
    return y, size

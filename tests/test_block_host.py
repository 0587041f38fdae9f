"""Host-side checks of the decode-block calls (no GPU needed): bad arguments
are refused with a code and a message before anything is launched, empty
batches are accepted, and the binding refuses what the C side cannot see."""

import ctypes as C

import pytest
import torch

from tests.helpers import ensure_built

F32, BF16, FP8 = 0, 1, 2
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
P = 1 << 20   # an aligned address that is never dereferenced on the host


@pytest.fixture(scope="module")
def B():
    return ensure_built()


def _call(fn, args, over):
    args = dict(args, **over)
    return fn(*args.values())


NORM = dict(x=P, x_dt=F32, x_ld=64, res=None, r_dt=0, r_ld=0, ro=None, ro_ld=0, w=P, w_dt=BF16, eps=1e-5, T=2, d=64,
            y=P, y_dt=BF16, y_ld=64, ys=None, group=0, stream=None)


@pytest.mark.parametrize("over,code,text", [
    (dict(T=-1), INVALID, "T"),
    (dict(d=12), INVALID, "d=12"),
    (dict(d=32776, x_ld=32776, y_ld=32776), UNSUPPORTED, "32768"),
    (dict(x=None), INVALID, "x null"),
    (dict(x=P + 2), INVALID, "x null or unaligned"),
    (dict(y=P + 8), INVALID, "y null or unaligned"),
    (dict(x_ld=60), INVALID, "row stride"),
    (dict(y_ld=68), INVALID, "row stride"),
    (dict(w=P + 4), INVALID, "weight"),
    (dict(x_dt=FP8), UNSUPPORTED, "dtypes"),
    (dict(y_dt=7), UNSUPPORTED, "dtypes"),
    (dict(res=P, r_dt=FP8, r_ld=64), UNSUPPORTED, "dtypes"),
    (dict(res=P, r_dt=BF16, r_ld=32), INVALID, "residual"),
    (dict(ro=P + 2, r_dt=BF16, ro_ld=64), INVALID, "residual_out"),
    (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(y_dt=FP8), INVALID, "y_scale"),
    (dict(ys=P), INVALID, "y_scale"),
    (dict(y_dt=FP8, ys=P, group=64), INVALID, "group"),
    (dict(y_dt=FP8, ys=P, group=128), INVALID, "group"),
])
def test_norm_refusals(B, over, code, text):
    assert _call(B.lib().moe_rmsnorm, NORM, over) == code
    assert text in B.lib().moe_last_error().decode()


def _cache(B, **over):
    f = dict(k=P, v=P, k_scale=None, v_scale=None, k_page_stride=4096, k_slot_stride=256, k_head_stride=64,
             v_page_stride=4096, v_slot_stride=256, v_head_stride=64, dtype=BF16, num_pages=8, page_size=16, heads=4,
             head_dim=64)
    f.update(over)
    return C.byref(B.KvCacheArgs(**f))


BAD_CACHES = [
    (dict(dtype=F32), UNSUPPORTED, "cache dtype"),
    (dict(k=None), INVALID, "cache null"),
    (dict(v=P + 2), INVALID, "unaligned"),
    (dict(k_scale=P, v_scale=P), INVALID, "k_scale"),
    (dict(dtype=FP8), INVALID, "k_scale"),
    (dict(dtype=FP8, k_scale=P), INVALID, "k_scale"),
    (dict(dtype=FP8, k_scale=P, v_scale=P, head_dim=72), INVALID, "head_dim"),
    (dict(head_dim=0), INVALID, "head_dim"),
    (dict(head_dim=60), INVALID, "head_dim"),
    (dict(head_dim=264), UNSUPPORTED, "head_dim"),
    (dict(page_size=0), INVALID, "page_size"),
    (dict(heads=0), INVALID, "heads"),
    (dict(num_pages=0), INVALID, "num_pages"),
    (dict(k_slot_stride=4), INVALID, "strides"),
    (dict(v_head_stride=-64), INVALID, "strides"),
]

APPEND = dict(k=P, kts=256, khs=64, v=P, vts=256, vhs=64, dt=BF16, T=2, cache=None, table=P, ld=4, R=2, pages=4, pos=P,
              req=None, cs=P, rot=64, max_pos=100, q=P, qts=512, qhs=64, qo=P, ots=512, ohs=64, hq=8, status=None,
              stream=None)


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(T=-1), INVALID, "T"),
    (dict(R=-1), INVALID, "R"),
    (dict(ld=3), INVALID, "table_ld"),
    (dict(rot=66), INVALID, "rot"),
    (dict(rot=7), INVALID, "rot"),
    (dict(rot=-2), INVALID, "rot"),
    (dict(rot=0), INVALID, "rot"),
    (dict(cs=None), INVALID, "rot"),
    (dict(max_pos=0), INVALID, "max_pos"),
    (dict(q=None), INVALID, "q_out"),
    (dict(qo=None), INVALID, "q_out"),
    (dict(hq=0), INVALID, "q_heads"),
    (dict(k=None), INVALID, "null"),
    (dict(pos=None), INVALID, "null"),
    (dict(table=None), INVALID, "null"),
    (dict(v=P + 1), INVALID, "aligned"),
])
def test_append_refusals(B, over, code, text):
    assert _call(B.lib().moe_kv_append, dict(APPEND, cache=_cache(B)), over) == code
    assert text in B.lib().moe_last_error().decode()


ATTN = dict(q=P, dt=BF16, qb=512, qh=64, B=2, hq=8, cache=None, table=P, ld=4, pages=4, lens=P, scale=0.1, window=0,
            cap=0.0, out=P, odt=BF16, ob=512, oh=64, lse=None, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=FP8), UNSUPPORTED, "dtypes"),
    (dict(odt=FP8), UNSUPPORTED, "dtypes"),
    (dict(B=-1), INVALID, "B"),
    (dict(hq=6), INVALID, "q_heads"),
    (dict(hq=0), INVALID, "q_heads"),
    (dict(ld=3), INVALID, "table_ld"),
    (dict(pages=-1), INVALID, "max_pages"),
    (dict(window=-1), INVALID, "window"),
    (dict(cap=-1.0), INVALID, "softcap"),
    (dict(cap=float("nan")), INVALID, "softcap"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(q=None), INVALID, "q or out"),
    (dict(out=P + 2), INVALID, "q or out"),
    (dict(qh=60), INVALID, "stride"),
    (dict(table=None), INVALID, "null"),
    (dict(lens=None), INVALID, "null"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws=P + 4), INVALID, "workspace"),
    (dict(ws_bytes=64), WORKSPACE, "required"),
])
def test_attn_refusals(B, over, code, text):
    assert _call(B.lib().moe_attn_decode, dict(ATTN, cache=_cache(B)), over) == code
    assert text in B.lib().moe_last_error().decode()


@pytest.mark.parametrize("over,code,text", BAD_CACHES)
def test_cache_refusals(B, over, code, text):
    for fn, args in ((B.lib().moe_kv_append, APPEND), (B.lib().moe_attn_decode, ATTN)):
        assert _call(fn, dict(args, cache=_cache(B, **over)), {}) == code
        assert text in B.lib().moe_last_error().decode()
    assert _call(B.lib().moe_attn_decode, dict(ATTN, cache=None), {}) == INVALID


LORA = dict(x=P, x_dt=BF16, x_ld=64, xs=None, T=2, d=64, w=P, w_dt=BF16, w_ld=64, wsc=None, N=32, la=P, lb=P, ls=P,
            na=3, r=16, ad=P, y=P, y_dt=F32, y_ld=32, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,code,text", [
    (dict(x_dt=FP8), UNSUPPORTED, "dtypes"),
    (dict(w_dt=F32), UNSUPPORTED, "dtypes"),
    (dict(w_dt=FP8), UNSUPPORTED, "dtypes"),
    (dict(y_dt=FP8), UNSUPPORTED, "dtypes"),
    (dict(xs=P), INVALID, "x_scale"),
    (dict(x_dt=FP8, w_dt=FP8, xs=P), INVALID, "w_scale"),
    (dict(x_dt=FP8, w_dt=FP8, xs=P, wsc=P, d=72, x_ld=80, w_ld=80), INVALID, "d"),
    (dict(T=-1), INVALID, "T"),
    (dict(T=129), UNSUPPORTED, "T=129"),
    (dict(d=60), INVALID, "d"),
    (dict(d=32776, x_ld=32776, w_ld=32776), UNSUPPORTED, "32768"),
    (dict(N=36), INVALID, "N"),
    (dict(r=12), INVALID, "r=12"),
    (dict(r=136), UNSUPPORTED, "r=136"),
    (dict(r=0), INVALID, "adapters"),
    (dict(la=None), INVALID, "adapters"),
    (dict(ad=None), INVALID, "adapters"),
    (dict(na=0), INVALID, "adapters"),
    (dict(na=1 << 27), UNSUPPORTED, "2^31"),
    (dict(la=P + 2), INVALID, "lora_a"),
    (dict(x=None), INVALID, "x null"),
    (dict(w=P + 8), INVALID, "w null or unaligned"),
    (dict(w_ld=68), INVALID, "row stride"),
    (dict(x_ld=32), INVALID, "row stride"),
    (dict(y_ld=24), INVALID, "row stride"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(ws_bytes=600), WORKSPACE, "required"),
])
def test_lora_refusals(B, over, code, text):
    assert _call(B.lib().moe_lora_project, LORA, over) == code
    assert text in B.lib().moe_last_error().decode()


def test_empty_batches_launch_nothing(B):
    L = B.lib()
    assert _call(L.moe_rmsnorm, NORM, dict(T=0)) == 0
    assert _call(L.moe_kv_append, dict(APPEND, cache=_cache(B)), dict(T=0)) == 0
    assert _call(L.moe_attn_decode, dict(ATTN, cache=_cache(B)), dict(B=0)) == 0
    assert _call(L.moe_lora_project, LORA, dict(T=0)) == 0


@pytest.mark.parametrize("args", [(-1, 8, 4, 64), (2, 0, 4, 64), (2, 6, 4, 64), (2, 8, 0, 64), (2, 8, 4, 60),
                                  (2, 8, 4, 264)])
def test_attn_workspace_refuses_bad_sizes(B, args):
    assert B.lib().moe_attn_workspace_bytes(*args) == 0
    with pytest.raises(B.MoeError):
        B.moe_attn_workspace_bytes(*args)


@pytest.mark.parametrize("args", [(-1, 64, 16), (129, 64, 16), (2, 60, 16), (2, 32776, 16), (2, 64, 12), (2, 64, 136)])
def test_lora_workspace_refuses_bad_sizes(B, args):
    assert B.lib().moe_lora_workspace_bytes(*args) == 0
    with pytest.raises(B.MoeError):
        B.moe_lora_workspace_bytes(*args)


def test_workspaces_grow_with_the_sizes(B):
    """A workspace for more requests or tokens serves fewer of them."""
    a = [B.moe_attn_workspace_bytes(n, 16, 4, 128) for n in (0, 1, 7, 128, 1000)]
    assert a == sorted(a) and a[0] >= 512
    p = [B.moe_lora_workspace_bytes(t, 2048, 16) for t in (0, 1, 7, 128)]
    assert p == sorted(p) and p[0] >= 512


def test_binding_refuses_wrong_tensors(B):
    """CPU tensors, wrong shapes and types never reach the library."""
    x, y = torch.zeros(2, 64), torch.zeros(2, 64)
    with pytest.raises(ValueError):
        B.moe_rmsnorm(x, None, 1e-5, y)
    with pytest.raises(ValueError):
        B.moe_rmsnorm(x, None, 1e-5, torch.zeros(2, 32))
    with pytest.raises(ValueError):
        B.moe_rmsnorm(x, torch.ones(32), 1e-5, y)
    kv = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.KvCache(kv, kv)
    with pytest.raises(ValueError):
        B.KvCache(kv, kv[:1])
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError):
        B.moe_lora_project(x, torch.zeros(32, 48), torch.zeros(2, 32), ws)
    with pytest.raises(ValueError):
        B.moe_lora_project(x, torch.zeros(32, 64), torch.zeros(2, 32), ws, adapter=torch.zeros(2, dtype=torch.int32))

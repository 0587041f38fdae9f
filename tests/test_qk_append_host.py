"""Host-side checks of moe_qk_norm_append (no GPU needed)."""

import ctypes as C

import pytest
import torch

from tests.helpers import ensure_built
from tests.test_block_host import APPEND, BF16, F32, FP8, INVALID, P, UNSUPPORTED, _cache, _call

AXIS = (C.c_uint8 * 32)(*([0, 1, 2, 1] * 8))
QK = {n: APPEND[n] for n in APPEND if n not in ("status", "stream")}
QK.update(qw=P, kw=P, w_dt=BF16, eps=1e-6, ap=P, axes=3, axis=AXIS, status=None, stream=None)


@pytest.fixture(scope="module")
def B():
    return ensure_built()


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=FP8), UNSUPPORTED, "dtype"),
    (dict(T=-1), INVALID, "T"),
    (dict(ld=3), INVALID, "table_ld"),
    (dict(rot=66), INVALID, "rot"),
    (dict(q=None), INVALID, "q_out"),
    (dict(k=None), INVALID, "null"),
    (dict(v=P + 1), INVALID, "aligned"),
    (dict(eps=-1e-6), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(eps=float("inf")), INVALID, "eps"),
    (dict(w_dt=FP8), UNSUPPORTED, "weights"),
    (dict(qw=P + 1), INVALID, "q_weight"),
    (dict(kw=P + 2, w_dt=F32), INVALID, "k_weight"),
    (dict(axes=-1), INVALID, "axes"),
    (dict(axes=256), INVALID, "axes"),
    (dict(axes=0), INVALID, "axes"),
    (dict(axis=None), INVALID, "axes"),
    (dict(ap=None), INVALID, "axes"),
    (dict(axes=2), INVALID, "axis[2]=2"),
    (dict(rot=0, cs=None, max_pos=0), INVALID, "axes"),
])
def test_qk_append_refusals(B, over, code, text):
    assert _call(B.lib().moe_qk_norm_append, dict(QK, cache=_cache(B)), over) == code
    assert text in B.lib().moe_last_error().decode()


def test_qk_append_no_tokens(B):
    """Nothing is launched, and pointers of an empty batch are not asked for."""
    assert _call(B.lib().moe_qk_norm_append, dict(QK, cache=_cache(B)),
                 dict(T=0, k=None, v=None, pos=None, ap=None, q=None, qo=None, qw=None, kw=None, w_dt=7)) == 0


def test_binding_refuses_host_tensors(B):
    x = torch.zeros(1, 2, 64)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="KvCache"):
        B.moe_qk_norm_append(x, x, x, None, None, 1e-6, None, i, i[0], x)
    with pytest.raises(TypeError, match="q_out"):
        B.moe_qk_norm_append(x, x, x, None, None, 1e-6, None, i, i[0])

"""What the binding of the decode-block calls does with sizes beyond 32 bits and with tensors of more than
one layout, on the GPU."""

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import assert_within, cos_sin_table, gen, make_cache, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def test_sizes_beyond_32_bits_are_refused(B):
    """2^32 tokens or requests (views of one; their positions or lengths never written) are no empty batch."""
    n = 1 << 32
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    _, _, _, _, cache = make_cache(B, gen(0), 2, 16, 2, 64, "bf16")
    row = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda").expand(n, 2, 64)
    numbers = torch.empty(n, dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="32 bits"):
        B.moe_kv_append(row, row, cache, table, numbers, req=numbers)
    with pytest.raises(ValueError, match="32 bits"):
        B.moe_attn_decode(row, cache, table.expand(n, 2), numbers, 0.125, row, B.new_attn_workspace(1, 2, 2, 64))


def test_append_views_with_a_size_of_one(B):
    """One token, or one head, whose meaningless stride is no multiple of 8."""
    g = gen(2)
    for shape, strides in (((1, 2, 64), (133, 64, 1)), ((3, 1, 64), (64, 9, 1))):
        T, hkv, D = shape
        k, v, _, _, cache = make_cache(B, g, 6, 4, hkv, D, "bf16", fill=0)
        kn, vn, q, qo = (normal(g, T * hkv * D, dtype=torch.bfloat16).as_strided(shape, strides) for _ in range(4))
        table = torch.arange(6, dtype=torch.int32, device="cuda")[:2 * T].view(T, 2)
        pos = torch.tensor([5, 0, 7][:T], dtype=torch.int32, device="cuda")
        B.moe_kv_append(kn, vn, cache, table, pos, cos_sin=cos_sin_table(8, 64), q=q, q_out=qo)
        want = O.rotate(q, pos, cos_sin_table(8, 64))
        assert_within(qo, want, 1e-5 + 1.01 * 2.0 ** -8 * want.abs(), "q")
        for t in range(T):
            p, i = O.slot_of(table, t, int(pos[t]), 4)
            assert torch.equal(v[p, i], vn[t])


def test_a_cache_of_another_device_is_refused(B):
    """What a call reads is on the current device, whose stream it takes."""
    _, _, _, _, cache = make_cache(B, gen(0), 2, 16, 2, 64, "bf16")
    x, i = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    B.moe_kv_append(x, x, cache, i, i[0])
    cache.handle.device += 1          # as of a cache on the next GPU
    with pytest.raises(ValueError, match="device"):
        B.moe_kv_append(x, x, cache, i, i[0])
    with pytest.raises(ValueError, match="device"):
        B.moe_attn_decode(x, cache, i, i[0], 1.0, x, B.new_attn_workspace(1, 2, 2, 64))

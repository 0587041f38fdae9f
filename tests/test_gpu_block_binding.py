"""What the binding of the decode-block calls does with sizes beyond 32 bits, on the GPU."""

import pytest
import torch

from tests.helpers import ensure_built
from tests.test_gpu_block import gen, make_cache

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

"""moe_qk_norm_append gives equal calls equal bits, with calls on other tokens and caches between them that nothing waits for."""

import pytest
import torch

from tests.helpers import ensure_built
from tests.test_gpu_block import DT, cos_sin_table, gen, make_cache, normal
from tests.test_gpu_pages_shared import bits
from tests.test_gpu_qk_append import axes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


@pytest.mark.parametrize("T,hq,hkv,D,rot,x,A", [(5000, 56, 8, 128, 64, "bf16", 3), (3001, 8, 2, 64, 64, "bf16", 0), (97, 16, 4, 128, 128, "f32", 3),
                                                (1, 16, 4, 128, 128, "bf16", 0), (700, 6, 2, 80, 24, "f32", 2), (500, 5, 1, 80, 6, "bf16", 2)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_qk_append_equal_calls_give_equal_bits(B, T, hq, hkv, D, rot, x, A, dtype):
    page, calls = 16, []
    for seed in (1, 2):
        g = gen(seed)
        cols = T // page + 1
        k, v, _, _, cache = make_cache(B, g, cols, page, hkv, D, dtype)
        qkv = normal(g, T, hq + 2 * hkv, D, std=2.0, dtype=DT[x])
        w = [1 + 0.2 * normal(g, D) for _ in range(2)]
        table = torch.randperm(cols, generator=g, device="cuda").to(torch.int32).view(1, cols)
        pos = torch.randperm(T, generator=g, device="cuda").to(torch.int32)
        req = torch.zeros(T, dtype=torch.int32, device="cuda")
        at, axis = axes_of(T, A, rot // 2, seed) if A else (None, None)
        cs = cos_sin_table(64 if A else T, rot)
        out = torch.empty(T, hq, D, dtype=DT[x], device="cuda")

        def call(qkv=qkv, w=w, cache=cache, table=table, pos=pos, out=out, req=req, cs=cs, at=at, axis=axis):
            B.moe_qk_norm_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *w, 1e-6, cache, table, pos, out, req=req,
                                 cos_sin=cs, axis_positions=at, axis=axis)

        seen = torch.zeros(cols, page, dtype=torch.bool, device="cuda")
        seen[table[0].long()[pos.long() // page], pos.long() % page] = True
        calls.append((call, (out, k, v), seen))
    (call, tensors, seen), (other, _, _) = calls
    call()
    torch.cuda.synchronize()
    want = [bits(t).clone() for t in tensors]
    for _ in range(5):
        for t in tensors:
            bits(t)[...] = 17
        call()
        other()
        call()
        torch.cuda.synchronize()
        for t, w in zip(tensors, want):
            got = bits(t)
            if t is tensors[0]:
                assert torch.equal(got, w)
            else:
                assert torch.equal(got[seen], w[seen]) and (got[~seen] == 17).all()

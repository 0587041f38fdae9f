"""The projection with adapters: infinite weights, scales written right before the call, against the fp64
oracle (tolerance: 64 u of sum |w x|, u = 2^-24, as in test_gpu_block.py)."""

import math

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import DT, U, assert_within, e4m3, gen, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def check(y, want, size, at):
    """y equals the oracle's infinities at `at` and is near it elsewhere."""
    got = O.f64(y)
    assert torch.isinf(want[at]).all() and torch.equal(got[at], want[at]), "infinities"
    zero = torch.zeros_like(want)
    assert_within(torch.where(at, zero, got), torch.where(at, zero, want), torch.where(at, zero, 64 * U * size), "the others")


@pytest.mark.parametrize("T", [1, 2, 5, 33, 128])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_lora_infinite_weights(B, T, x):
    """A row of W with an infinity gives infinities of x's sign, whatever bits x has."""
    g, d, N = gen(T), 1024, 264
    xt = normal(g, T, d, dtype=DT[x])
    xt[0] = xt[0].to(torch.bfloat16).to(DT[x])      # nothing beyond a bf16
    w = normal(g, N, d, std=0.02, dtype=torch.bfloat16)
    w[7, 300], w[200, 1000] = math.inf, -math.inf
    y = torch.empty(T, N, device="cuda")
    B.moe_lora_project(xt, w, y, B.new_lora_workspace(T, d))
    fin = w.clone()
    fin[7, 300], fin[200, 1000] = 0, 0
    want, size = O.lora_project(xt, fin)
    want[:, 7], want[:, 200] = torch.sign(O.f64(xt)[:, 300]) * math.inf, torch.sign(O.f64(xt)[:, 1000]) * -math.inf
    at = torch.zeros(T, N, dtype=torch.bool)
    at[:, [7, 200]] = True
    check(y, want, size, at)


@pytest.mark.parametrize("T,r,na", [(1, 16, 2), (2, 128, 2), (6, 16, 4), (6, 72, 4), (100, 16, 3), (100, 128, 3), (64, 24, 40)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_lora_infinite_adapter_weights(B, T, r, na, x):
    """An infinity in B_a gives the adapter's tokens one of v's sign."""
    g, d, N = gen(T + r), 512, 264
    xt, w = normal(g, T, d, dtype=DT[x]), normal(g, N, d, std=0.02, dtype=torch.bfloat16)
    la, lb = normal(g, na, r, d, std=0.05, dtype=torch.bfloat16), normal(g, na, N, r, std=0.05, dtype=torch.bfloat16)
    la[1, 3] = 0.0
    la[1, 3, 8] = 0.5                               # v = x[8] / 2 exactly: x's bits alone
    scale = torch.ones(na, device="cuda")
    ad = torch.tensor([t % na if T > 2 else 1 for t in range(T)], dtype=torch.int32, device="cuda")
    fin = lb.clone()
    lb[1, 5, 3], lb[1, 250, 3] = math.inf, -math.inf
    fin[1, 5, 3], fin[1, 250, 3] = 0, 0
    y = torch.empty(T, N, device="cuda")
    B.moe_lora_project(xt, w, y, B.new_lora_workspace(T, d, r), lora=(la, lb, scale), adapter=ad)
    want, size = O.lora_project(xt, w, (la, fin, scale), ad)
    mine = (ad == 1).cpu()
    sign = torch.sign(O.f64(xt)[mine, 8])
    at = torch.zeros(T, N, dtype=torch.bool)
    at[mine, 5], at[mine, 250] = True, True
    want[mine, 5], want[mine, 250] = sign * math.inf, -sign * math.inf
    check(y, want, size, at)


@pytest.mark.parametrize("T", [3, 128])
def test_lora_weight_scales_of_the_kernel_before(B, T):
    """w_scale (and lora's own) written by a copy right before the call, with adapters: what an earlier call
    left in a cache must not be seen."""
    g, d, N, r, na = gen(T), 1024, 768, 32, 6
    x, xs = e4m3(normal(g, T, d, std=100.0)), torch.full((T,), 0.01, device="cuda")
    w = e4m3(normal(g, N, d, std=100.0))
    scales = [0.0002 * (1 + torch.rand(N, generator=g, device="cuda")) for _ in range(2)]
    lscales = [torch.rand(na, generator=g, device="cuda") for _ in range(2)]
    a, b = normal(g, na, r, d, std=0.05, dtype=torch.bfloat16), normal(g, na, N, r, std=0.05, dtype=torch.bfloat16)
    ad = torch.randint(-1, na, (T,), generator=g, device="cuda", dtype=torch.int32)
    ws_, ls = torch.empty(N + 1, device="cuda")[1:], torch.empty(na, device="cuda")     # 4-byte aligned
    y, ws = torch.empty(T, N, device="cuda"), B.new_lora_workspace(T, d, r)

    def step(i):
        ws_.copy_(scales[i])
        ls.copy_(lscales[i])
        B.moe_lora_project(x, w, y, ws, lora=(a, b, ls), adapter=ad, x_scale=xs, w_scale=ws_)

    want = []
    for i in range(2):
        step(i)
        torch.cuda.synchronize()
        ref, size = O.lora_project(x, w, (a, b, ls), ad, xs, ws_)
        assert_within(y, ref, 64 * U * size, "y")
        want.append(y.clone())
    got = []
    for k in range(60):
        step(k % 2)
        got.append(y.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k % 2]) for k in range(60))

"""The decode block of examples/decode_block.py, every stage against the fp64
oracle on the inputs that the stage got on the GPU, over several steps; and the
same steps replayed from a CUDA graph.

Tolerances as in test_gpu_block.py (u = 2^-24; a bf16 result adds 2^-8 of
itself) and, for the MoE layer, its own 1e-4 of the largest output."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from moe_decode_layer_fp32_gb300 import synth
from oracle import block_oracle as O
from oracle import moe_oracle as M
from tests import helpers as H

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 1.01 * 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.ensure_built()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_block.py")
    spec = importlib.util.spec_from_file_location("decode_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def within(got, want, bound, what):
    off = (O.f64(got) - want).abs()
    assert torch.isfinite(O.f64(got)).all(), what
    assert ((off - bound) <= 0).all(), f"{what}: off by {off.max().item():.3g}"


@pytest.mark.parametrize("shape,cache", [(synth.TINY_VANILLA, "bf16"), (synth.TINY_DEAMOE, "bf16"),
                                         (synth.TINY_DEAMOE, "e4m3")])
def test_block_steps(example, shape, cache):
    T, D, hq, hkv = 5, 64, 4, 2
    blk = example.DecodeBlock(shape, T, 48, hq, hkv, D, page=8, adapters=3, rank=8, cache=cache, seed=3)
    x = torch.zeros(T, shape.d, device="cuda")
    start = torch.tensor([0, 3, 7, 8, 20], dtype=torch.int32, device="cuda")
    adapter = torch.tensor([0, -1, 2, 2, 1], dtype=torch.int32, device="cuda")
    k_cache, v_cache, ks, vs = blk.cache.tensors
    for i in range(3):
        positions = start + i
        seq = positions + 1
        delta = synth.hidden(T, shape.d, 10 + i, "cuda")
        x0 = x.clone()
        y = blk.step(delta, x, positions, seq, adapter)
        torch.cuda.synchronize()
        assert blk.status() == 0
        h1, z1 = O.rms_norm(delta, blk.norm1, example.EPS, x0)
        within(blk.h1, h1, 40 * U * h1.abs() + BF * h1.abs(), "h1")
        # the projection's output was rotated in place: k, v are in the cache, q is
        qkv, size = O.lora_project(blk.h1, blk.w_qkv, blk.lora_qkv, adapter)
        heads, hsize = qkv.view(T, -1, D), size.view(T, -1, D)
        # a bf16 value before the rotation and one after it
        near = 2 * BF * heads.abs().amax(2, keepdim=True) + 64 * U * hsize.amax(2, keepdim=True)
        q = blk.qkv.view(T, -1, D)[:, :hq]
        within(q, O.rotate(heads[:, :hq], positions, blk.cos_sin), 2 * near[:, :hq], "q")
        want_k, want_v = O.rotate(heads[:, hq:hq + hkv], positions, blk.cos_sin), heads[:, hq + hkv:]
        for t in range(T):
            n = int(seq[t])
            rk = O.cached_rows(k_cache, ks, blk.block_table[t], 0, n)
            rv = O.cached_rows(v_cache, vs, blk.block_table[t], 0, n)
            for row, want, nr in ((rk[n - 1], want_k[t], near[t, hq:hq + hkv]), (rv[n - 1], want_v[t], near[t, hq + hkv:])):
                step = 0.0 if ks is None else 2.0 ** -4 * want.abs() + O.f64(ks)[:, None] * 2.0 ** -10
                within(row, want, 2 * nr + 1.1 * step, "cache row")
            o, _ = O.decode_attention(q[t], (rk, rv), D ** -0.5)
            within(blk.attn[t], o, 1e-4 * rv.abs().max() + BF * o.abs(), f"attention of request {t}")
        o, size = O.lora_project(blk.attn.view(T, -1), blk.w_o, blk.lora_o, adapter)
        within(blk.o, o, 64 * U * size, "o")
        h2, z2 = O.rms_norm(blk.o, blk.norm2, example.EPS, z1)
        within(x, z2, 4 * U * (z2.abs() + z1.abs()), "residual stream")
        within(blk.h2, h2, 80 * U * (h2.abs() + 1), "h2")
        L = blk.layer
        idx, p, _ = M.route(blk.h2, L["router"], shape.k)
        assert np.array_equal(blk.topk_idx.cpu().numpy(), idx)
        if shape.I_sh:
            ref = M.deamoe_layer_c(blk.h2, idx, p, shape.g, L["dgate"], L["dup"], L["ddown"], L["pgate"], L["pup"], L["pdown"])
        else:
            ref = M.vanilla_layer(blk.h2, idx, p, L["gate"], L["up"], L["down"])
        assert H.rel_err(y.cpu().numpy(), ref) <= 1e-4


def test_block_graph_replays_equal_eager_steps(example):
    T, D = 4, 64
    runs = []
    for captured in (False, True):
        blk = example.DecodeBlock(synth.TINY_VANILLA, T, 40, 4, 2, D, page=8, adapters=2, rank=8, seed=5)
        x, delta = torch.zeros(T, 256, device="cuda"), synth.hidden(T, 256, 2, "cuda")
        positions = torch.tensor([0, 1, 9, 17], dtype=torch.int32, device="cuda")
        seq = positions + 1
        adapter = torch.tensor([1, -1, 0, 1], dtype=torch.int32, device="cuda")

        def one():
            blk.step(delta, x, positions, seq, adapter)
            positions.add_(1)
            seq.add_(1)

        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
            step = graph.replay
        else:
            step = one
        for _ in range(6):
            step()
        torch.cuda.synchronize()
        assert blk.status() == 0
        # the layer adds its experts' outputs with atomics: compare what comes before it
        runs.append((blk.attn.clone(), blk.h2.clone(), x.clone(), blk.y.clone()))
    for a, b in zip(runs[0][:3], runs[1][:3]):
        assert torch.equal(a, b)
    assert H.rel_err(runs[1][3].cpu().numpy(), runs[0][3].cpu().numpy()) <= 1e-5

"""The norm's E4M3 codes at the ends of fp32's range, and its row-walking form with a scale per 128
columns, against the fp64 oracle.

Bounds (u = 2^-24): a scale is amax / 448 within 40 u, and within half a step of fp32's subnormals
(2^-150) of that; a code times its scale is y within 2^-4 of y (half a step of E4M3), 2^-10 of the scale
(half a step of its subnormals), and what a product z w that is subnormal loses before the row's factor."""

import pytest
import torch

from oracle import block_oracle as O
from tests.helpers import ensure_built
from tests.test_gpu_block import DT, U, assert_within, gen, normal, run_norm

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ensure_built()


def check_codes(B, x, w, group):
    T, d = x.shape
    y = torch.empty(T, d, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty((T, d // group) if group else (T,), device="cuda")
    B.moe_rmsnorm(x, w, EPS, y, y_scale=sc)
    yr, zr = O.rms_norm(x, w, EPS)
    sr = O.e4m3_scales(yr, group)
    assert_within(sc, sr, 40 * U * sr + 2.0 ** -149, "scale")
    s = O.f64(sc).repeat_interleave(group, 1) if group else O.f64(sc)[:, None]
    rstd = 1 / torch.sqrt((zr * zr).mean(1, keepdim=True) + EPS)
    bound = yr.abs() * 2.0 ** -4 * 1.0001 + s * 2.0 ** -10 * 1.0001 + rstd * 2.0 ** -149
    codes = O.f64(y)
    assert torch.isfinite(codes).all(), "codes are not finite"
    assert (codes[(yr == 0)] == 0).all(), "zeros"
    assert_within(codes * s, yr, bound, "codes")


@pytest.mark.parametrize("T", [3, 400])          # a block per row, and blocks that walk over rows
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("tiny", [1e-34, 1e-37, 1e-40])
def test_norm_codes_of_tiny_rows(B, T, x, group, tiny):
    """Zeros and a few tiny values: the whole row, and 128 columns of an ordinary one."""
    g = gen(T)
    v = torch.zeros(T, 512, device="cuda")
    v[:, 128] = tiny
    v[:, 200] = -0.5 * tiny
    v[:, 255] = 0.15 * tiny
    v[1, 256:] = normal(g, 256)
    for w in (None, (1 + 0.1 * normal(g, 512)).to(torch.bfloat16)):
        check_codes(B, v.to(DT[x]), w, group)


@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_codes_of_huge_weights(B, T, group):
    x = torch.ones(T, 256, device="cuda")
    x[:, ::2] = -1.0
    w = torch.ones(256, device="cuda")
    w[5], w[6], w[7] = 2.0 ** 127, 2.0 ** 126, -1.5 * 2.0 ** 120
    check_codes(B, x, w, group)


def test_norm_codes_below_the_smallest_scale(B):
    """amax / 448 that fp32 rounds to zero: scale 1, codes 0; NaN stays in its own row and 128 columns."""
    x = torch.zeros(3, 256, device="cuda")
    x[0, 3] = 1e-44
    x[1, 3], x[1, 200] = 1.0, 1e-44
    x[2, 5], x[2, 6] = float("nan"), 1.0
    y, sc = torch.empty(3, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(3, 2, device="cuda")
    B.moe_rmsnorm(x, None, 1.0, y, y_scale=sc)
    assert sc[0].tolist() == [1.0, 1.0] and sc[1, 1].item() == 1.0
    c = O.f64(y)
    assert (c[0] == 0).all() and (c[1, 128:] == 0).all() and c[1, 3] == 448
    assert torch.isnan(c[2]).all()


@pytest.mark.parametrize("T,d", [(1000, 128), (700, 1152), (400, 4224), (461, 7168), (331, 8320), (310, 16384)])
@pytest.mark.parametrize("x,res", [("bf16", "bf16"), ("f32", None), ("bf16", None), ("f32", "f32")])
def test_norm_walk_with_a_scale_per_128_columns(B, T, d, x, res):
    run_norm(B, T, d, x=x, res=res, y="e4m3", group=128, seed=T + d)

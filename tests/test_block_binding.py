"""The binding of the decode-block calls on the host (no GPU needed): what it takes for a cache."""

import ctypes as C

import pytest
import torch

from tests.helpers import ensure_built


@pytest.fixture(scope="module")
def B():
    return ensure_built()


def test_only_a_cache_is_taken_for_one(B):
    """An object that has an ``address`` of its own is no cache, wherever that points."""
    class Other:
        args = B.KvCacheArgs(heads=2, head_dim=64)
        address = C.addressof(args)

    x = torch.zeros(1, 2, 64)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for other in (Other(), Other, None, 7):
        with pytest.raises(ValueError, match="KvCache"):
            B.moe_kv_append(x, x, other, i, i[0])
        with pytest.raises(ValueError, match="KvCache"):
            B.moe_attn_decode(x, other, i, i[0], 1.0, x, i)


def test_functions_stay_the_modules_own(B, monkeypatch):
    """A call leaves the module's functions, their signatures and a caller's patch of one as they are."""
    import inspect

    names = ("moe_rmsnorm", "moe_kv_append", "moe_attn_decode", "moe_lora_project")
    before = {n: getattr(B, n) for n in names}
    def patch(*args, **kw):
        return "patched"

    monkeypatch.setattr(B, "moe_kv_append", patch)
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        B.moe_rmsnorm(x, None, 1e-5, x)
    assert B.moe_kv_append() == "patched"
    monkeypatch.undo()
    for n in names:
        assert getattr(B, n) is before[n] and getattr(B, n).__doc__
        assert list(inspect.signature(getattr(B, n)).parameters)
    assert "residual_out" in inspect.signature(B.moe_rmsnorm).parameters


def test_import_without_cuda_in_torch(B):
    """The binding imports, and calls that need no stream work, on a torch without CUDA's private names."""
    import subprocess
    import sys

    code = ("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "from moe_decode_layer_fp32_gb300 import binding as B\n"
            "print(B.moe_lora_workspace_bytes(2, 64, 16))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert int(r.stdout) == B.moe_lora_workspace_bytes(2, 64, 16)

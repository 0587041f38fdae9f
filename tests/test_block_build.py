"""What the build makes when parts of the machine are missing or change (no compiler runs here)."""

import os

import pytest

from moe_decode_layer_fp32_gb300 import build_native as N


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """A build into an empty folder whose commands only write their output file; they are listed."""
    ran = []

    def run(cmd):
        ran.append(cmd)
        if fake.fails and cmd[0] == fake.fails:
            raise RuntimeError("command failed")
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return ""

    fake.fails = None
    monkeypatch.setattr(N, "_run", run)
    monkeypatch.setattr(N, "nvcc_path", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(N, "OBJDIR", str(tmp_path / "obj"))
    monkeypatch.setattr(N, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(N, "BIND", str(tmp_path / "bind.so"))
    fake.ran = ran
    return fake


@pytest.mark.parametrize("missing", ["torch", "g++", "Python's headers"])
def test_the_library_needs_no_torch(fake, monkeypatch, capsys, missing):
    """Without what the extension module needs, the C library is built all the same and the rest is named."""
    if missing == "torch":
        find = N.importlib.util.find_spec
        monkeypatch.setattr(N.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    elif missing == "g++":
        which = N.shutil.which
        monkeypatch.setattr(N.shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    else:
        monkeypatch.setattr(N.sysconfig, "get_paths", lambda *a, **k: {"include": "/nowhere"})
    assert N.build() == N.LIB
    assert os.path.exists(N.LIB) and not os.path.exists(N.BIND)
    assert missing in capsys.readouterr().err


def test_a_failing_extension_leaves_the_library(fake):
    fake.fails = "g++"
    with pytest.raises(RuntimeError, match="command failed"):
        N.build()
    assert os.path.exists(N.LIB)


def test_another_torch_rebuilds_the_extension(fake, monkeypatch, tmp_path):
    """Only the extension, and only when torch's version, its place or the command changed."""
    torch = tmp_path / "torch"
    for f in ("include/c10/cuda/CUDAStream.h", "__init__.py", "version.py"):
        (torch / f).parent.mkdir(parents=True, exist_ok=True)
        (torch / f).write_text("__version__ = '1'")
    find = N.importlib.util.find_spec
    spec = type("Spec", (), {"origin": str(torch / "__init__.py")})
    monkeypatch.setattr(N.importlib.util, "find_spec", lambda n, *a: spec if n == "torch" else find(n, *a))
    N.build()
    fake.ran.clear()
    N.build()
    assert fake.ran == []
    (torch / "version.py").write_text("__version__ = '2'")
    os.utime(torch / "version.py", (0, 0))          # installed files may be older than the build
    N.build()
    assert [c[0] for c in fake.ran] == ["g++"]
    fake.ran.clear()
    N.build()
    assert fake.ran == []

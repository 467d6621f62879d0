"""What the build compiles and links, with the compilers replaced by a fake that only writes the
files they would write."""

import os
import subprocess
import sys

import pytest


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """The build module over an empty folder; ``ran`` lists (program, output) of each command."""
    from state_space_model_ssd_gb300 import build
    ran, fails = [], []

    def run(cmd, check=False, **_):
        out = cmd[cmd.index("-o") + 1]
        name = os.path.basename(out).split(".so.")[0]
        ran.append((os.path.basename(cmd[0]), name + (".so" if ".so." in out else "")))
        bad = any(f in ran[-1] for f in fails)
        if not bad:
            with open(out, "w") as f:
                f.write(" ".join(cmd))
        if bad and check:
            raise subprocess.CalledProcessError(1, cmd)
        return subprocess.CompletedProcess(cmd, int(bad), "", "")

    monkeypatch.setattr(build, "OBJDIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libssd.so"))
    monkeypatch.setattr(build, "EXT", str(tmp_path / "_layer_ext.so"))
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    build.ran, build.fails = ran, fails
    yield build
    del build.ran, build.fails


def test_library_builds_without_torch(fake, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert fake.build() == fake.LIB and os.path.exists(fake.LIB)
    assert not os.path.exists(fake.EXT) and all(p == "nvcc" for p, _ in fake.ran)
    assert "torch" in capsys.readouterr().err
    n = len(fake.ran)
    fake.build()
    assert len(fake.ran) == n  # nothing is stale


def test_library_is_linked_where_the_binding_fails(fake):
    """A machine without Python's or torch's headers still gets the C library, and the error."""
    import torch
    fake.fails.append("g++")
    with pytest.raises(RuntimeError, match="g"):
        fake.build()
    assert os.path.exists(fake.LIB) and not os.path.exists(fake.EXT)
    fake.fails.clear()
    fake.build()
    assert os.path.exists(fake.EXT) and [p for p, _ in fake.ran].count("nvcc") == len(fake.sources()) + 1
    assert torch.__version__ in open(fake.EXT).read()


def test_a_kernel_that_does_not_compile_fails_the_build(fake):
    fake.fails.append("ssd_norm.o")
    with pytest.raises(RuntimeError, match="ssd_norm"):
        fake.build()
    assert not os.path.exists(fake.LIB)


def test_binding_follows_the_torch_that_is_installed(fake, monkeypatch):
    """Back to an earlier torch, whose object is older than the module that was linked since."""
    import torch
    linked = lambda: open(fake.EXT).read()  # noqa: E731
    for version in ("2.9.1", "2.11.0", "2.9.1", "2.9.1", "2.11.0"):
        monkeypatch.setattr(torch, "__version__", version)
        n = len(fake.ran)
        same = os.path.exists(fake.EXT) and "torch" + version in linked()
        fake.build()
        assert "torch" + version in linked()
        assert not same or len(fake.ran) == n

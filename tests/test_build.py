"""What the build does, with a compiler and a linker that only write their output files (no GPU)."""
import os
import subprocess

import pytest

from tiled_attention_08_gb300 import build as fa_build


class Tools:
    """Stands in for subprocess.run: every command writes its -o file; those whose output's name
    contains one of `failing` fail, leaving a torn file behind as an interrupted one does."""

    def __init__(self):
        self.made, self.failing = [], ()

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("torn")
        if any(x in os.path.basename(out) for x in self.failing):
            return subprocess.CompletedProcess(cmd, 1, "", "it failed")
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        self.made.append(os.path.basename(out).split(".tmp")[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def since(self):
        made, self.made = self.made, []
        return made


@pytest.fixture
def tools(tmp_path, monkeypatch):
    """The build in an empty folder, with a torch of its own."""
    t = Tools()
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1.0'\n")
    monkeypatch.setattr(fa_build.subprocess, "run", t)
    monkeypatch.setattr(fa_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(fa_build, "LIB", str(tmp_path / "_build" / "libfa.so"))
    monkeypatch.setattr(fa_build, "TORCH_LIB", str(tmp_path / "_build" / "fa_torch.so"))
    spec = type("Spec", (), {"submodule_search_locations": [str(torch_dir)]})
    monkeypatch.setattr(fa_build.importlib.util, "find_spec", lambda name, *a: t.spec if name == "torch" else None)
    t.spec, t.dir, t.torch = spec, tmp_path / "_build", torch_dir
    return t


def test_library_without_torch(tools, capsys):
    """libfa.so needs nvcc alone; the binding is left out, with a word about it."""
    tools.spec = None
    assert fa_build.build() == fa_build.LIB and os.path.exists(fa_build.LIB)
    made = tools.since()
    assert "libfa.so" in made and "fa_fwd.o" in made and not any("torch" in m for m in made)
    assert "torch is not installed" in capsys.readouterr().err
    fa_build.build()
    assert tools.since() == []
    tools.spec = type("Spec", (), {"submodule_search_locations": [str(tools.torch)]})  # torch comes later
    fa_build.build()
    assert tools.since() == ["fa_torch.o", "fa_torch.so"]
    fa_build.build()
    assert tools.since() == []


def test_binding_follows_the_installed_torch(tools):
    """Another torch is noticed by its version, however old its files are."""
    fa_build.build()
    assert "fa_torch.so" in tools.since()
    version = tools.torch / "version.py"
    version.write_text("__version__ = '1.1'\n")
    os.utime(version, (1, 1))
    fa_build.build()
    assert tools.since() == ["fa_torch.o", "fa_torch.so"]
    os.utime(version)  # touched, but the same
    fa_build.build()
    assert tools.since() == []


@pytest.mark.parametrize("broken", ["fa_fwd.o", "libfa.so", "fa_torch.o", "fa_torch.so"])
def test_a_build_that_failed_half_way_is_taken_up_again(tools, broken):
    """Whatever step fails, nothing torn is left in its place, and the next build ends with libraries that
    are newer than all objects."""
    fa_build.build()
    tools.since()
    before = {name: (tools.dir / name).read_text() for name in os.listdir(tools.dir)}
    for name in os.listdir(tools.dir):  # everything is older than the sources
        os.utime(tools.dir / name, (1, 1))
    tools.failing = (broken,)
    with pytest.raises(RuntimeError):
        fa_build.build()
    assert (tools.dir / broken).read_text() == before[broken]
    assert all("torn" not in (tools.dir / name).read_text() for name in os.listdir(tools.dir))
    tools.failing = ()
    tools.since()
    fa_build.build()
    assert broken in tools.since()
    for lib in ("libfa.so", "fa_torch.so"):
        t = os.path.getmtime(tools.dir / lib)
        objs = [n for n in os.listdir(tools.dir) if n.endswith(".o") and (n == "fa_torch.o") == (lib == "fa_torch.so")]
        assert t > 1 and all(os.path.getmtime(tools.dir / n) <= t for n in objs)
    fa_build.build()
    assert tools.since() == []

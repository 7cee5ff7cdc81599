"""CPU checks of the build: what is compiled for which torch. Nothing is compiled here: the commands are recorded."""
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The build module with its outputs in an empty folder, and the list of what its commands made."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "tiled_tensor_core_tcgen05_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    for name in ("LIB", "BINDING", "OBJDIR", "LIB_DEBUG", "OBJDIR_DEBUG", "BINDING_FOR"):
        monkeypatch.setattr(b, name, str(tmp_path / name), raising=False)
    out = []

    def run(cmd, **kw):
        to = cmd[cmd.index("-o") + 1]
        with open(to, "w"):
            pass
        out.append(os.path.basename(to).split(".tmp")[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    real = importlib.util.find_spec
    torch_at = {"dir": None}

    def find(name, *a):
        if name != "torch":
            return real(name, *a)
        if torch_at["dir"] is None:
            return None
        return importlib.util.spec_from_file_location("torch", os.path.join(torch_at["dir"], "__init__.py"))

    monkeypatch.setattr(importlib.util, "find_spec", find)

    def install(name, version):
        d = tmp_path / name
        os.makedirs(d / "lib", exist_ok=True)
        (d / "__init__.py").write_text("")
        (d / "version.py").write_text(f"__version__ = {version!r}")
        (d / "lib" / "libc10_cuda.so").write_text("")
        torch_at["dir"] = str(d)

    def built():
        out.clear()
        b.build()
        return out[:]

    return built, install


def test_without_torch_the_library_alone_is_built(made):
    built, install = made
    first = built()
    assert "LIB" in first and "tg_api.o" in first and "tg_torch.o" not in first
    assert built() == []


def test_another_torch_builds_the_module_again(made):
    built, install = made
    install("one", "2.11")
    first = built()
    assert "LIB" in first and first[-1] == "BINDING"
    assert built() == []
    install("one", "2.12")
    assert built() == ["tg_torch.o", "BINDING"]
    install("two", "2.12")
    assert built() == ["tg_torch.o", "BINDING"]
    assert built() == []


def test_the_package_keeps_to_public_torch():
    package = os.path.join(ROOT, "tiled_tensor_core_tcgen05_gb300")
    for name in os.listdir(package):
        if name.endswith(".py"):
            with open(os.path.join(package, name)) as f:
                assert "torch._C" not in f.read(), name

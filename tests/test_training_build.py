"""What building the library and the training operators' binding needs, with the compilers replaced by stand-ins."""

import os
import subprocess
import sys
import types

import pytest

from powersgd_rank_gradient_gb300 import build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """build() in an empty directory; ``commands`` lists the compilers' calls, sources in ``broken`` fail."""
    state = types.SimpleNamespace(commands=[], broken=set())
    for name, file in (("BUILD", "_build"), ("LIB", "libpsgd.so"), ("BIND", "_bind.so"), ("PTXAS_LOG", "_build/ptxas.log")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    monkeypatch.setattr(build.library_hash, "__defaults__", (build.LIB, build.HASH_MARKER))

    def run(cmd, **kw):
        if "--version" in cmd:
            return subprocess.CompletedProcess(cmd, 0, "a compiler", "")
        state.commands.append(cmd)
        target = cmd[cmd.index("-o") + 1]
        if "-c" in cmd:
            if os.path.basename(cmd[cmd.index("-c") + 1]) in state.broken:
                return subprocess.CompletedProcess(cmd, 1, "", "no such header")
            content = b""
        else:
            machine = build._ELF_MACHINE[build.platform.machine()].to_bytes(2, "little")
            content = b"\x7fELF" + bytes(14) + machine + bytes(44)
            if "libpsgd.so" in os.path.basename(target):
                content += build.HASH_MARKER + build.source_hash().encode()
            else:
                content += build.BIND_MARKER + build.bind_hash().encode()
        with open(target, "wb") as fh:
            fh.write(content)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    return state


def built():
    return os.path.exists(build.LIB), os.path.exists(build.BIND)


def test_both_are_built_once(fake):
    pytest.importorskip("torch")
    assert build.build() == build.LIB and built() == (True, True)
    n = len(fake.commands)
    assert n == len(build.SOURCES) + 3
    build.build()
    assert len(fake.commands) == n
    build.build(force=True)
    assert len(fake.commands) == 2 * n


def without_torch(monkeypatch, tmp_path):
    monkeypatch.setitem(sys.modules, "torch", None)


def with_a_cpu_torch(monkeypatch, tmp_path):
    module = types.ModuleType("torch")
    module.__file__, module.__version__ = str(tmp_path / "torch" / "__init__.py"), "2.9.1+cpu"
    monkeypatch.setitem(sys.modules, "torch", module)


def without_python_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})


def without_a_host_compiler(monkeypatch, tmp_path):
    which = build.shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name, *a, **kw: None if name == "g++" else which(name, *a, **kw))


@pytest.mark.parametrize("missing", [without_torch, with_a_cpu_torch, without_python_headers, without_a_host_compiler])
def test_the_library_needs_nvcc_alone(fake, monkeypatch, tmp_path, capsys, missing):
    missing(monkeypatch, tmp_path)
    assert build.build() == build.LIB and built() == (True, False)
    assert not any("g++" in cmd[0] for cmd in fake.commands)
    assert "not built" in capsys.readouterr().err


def test_a_binding_that_does_not_compile_leaves_the_library(fake):
    pytest.importorskip("torch")
    fake.broken.add(build.BIND_SOURCE)
    with pytest.raises(RuntimeError, match="psgd_bind"):
        build.build()
    assert built() == (True, False)
    fake.broken.clear()
    build.build()
    assert built() == (True, True)


def test_a_kernel_that_does_not_compile_links_nothing(fake):
    fake.broken.add("psgd_misc.cu")
    with pytest.raises(RuntimeError, match="psgd_misc"):
        build.build()
    assert built() == (False, False)

"""The library is built whether or not the Python extension can be, and an extension built for
another torch is neither kept nor used."""

import os
import subprocess
import types

import pytest

import exact_io_aware_46_b200 as attn
from exact_io_aware_46_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Built files in an empty folder; compilers that write their output, or fail."""
    monkeypatch.setattr(build, "SO", str(tmp_path / "libattn.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    ran, broken = [], set()

    def compile(cmd):
        name = "nvcc" if "nvcc" in cmd[0] else "c++"
        ran.append(name)
        if name in broken:
            raise subprocess.CalledProcessError(1, cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(" ".join(cmd).encode())

    monkeypatch.setattr(build.subprocess, "check_call", compile)
    return types.SimpleNamespace(ran=ran, broken=broken)


def test_the_library_does_not_need_the_extension(tree):
    tree.broken.add("c++")
    with pytest.warns(RuntimeWarning, match="exit status 1"):
        assert build.build() == build.SO
    assert os.path.exists(build.SO) and not os.path.exists(build.BINDING)
    tree.broken.clear()
    build.build()
    assert tree.ran == ["nvcc", "c++", "c++"] and os.path.exists(build.BINDING)
    build.build()
    assert len(tree.ran) == 3
    tree.broken.add("nvcc")  # that one is needed
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)


def test_an_extension_for_another_torch_is_built_again(tree, monkeypatch):
    build.build()
    assert build.binding_up_to_date()
    monkeypatch.setattr(attn, "BINDING_TAG", attn.BINDING_TAG.replace("torch ", "torch 9."))
    assert not build.binding_up_to_date()
    tree.broken.add("c++")
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not os.path.exists(build.BINDING)  # not left for the import to find


def test_an_extension_for_another_torch_is_not_used():
    assert attn._binding.BUILT_FOR == attn.BINDING_TAG

    def other():
        return types.SimpleNamespace(BUILT_FOR=attn.BINDING_TAG + "x")

    def missing():
        raise ImportError("undefined symbol: f")

    for load, word in ((other, "built for"), (missing, "undefined symbol"),
                       (types.SimpleNamespace, "something else")):
        with pytest.warns(RuntimeWarning, match=word):
            assert attn._load_binding(load) is None
    same = types.SimpleNamespace(BUILT_FOR=attn.BINDING_TAG)
    assert attn._load_binding(lambda: same) is same


def test_without_a_library_there_is_nothing_to_warn_of(monkeypatch, recwarn):
    monkeypatch.setattr(attn, "LIB_PATH", "/nonexistent/libattn.so")

    def missing():
        raise ImportError("no module")

    assert attn._load_binding(missing) is None and not recwarn.list

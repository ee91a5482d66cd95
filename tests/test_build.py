"""What the build makes, with compilers that only write their output file (CPU only)."""

import sys

import pytest

from sparse_attention_top_ds_b200 import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """Build into a folder of its own; the names of what the compilers were asked for."""
    names = []

    class Popen:
        returncode = 0

        def __init__(self, cmd, **kw):
            out = cmd[cmd.index("-o") + 1]
            names.append(out.split("/")[-1].replace(".tmp", ""))
            open(out, "w").close()

        def communicate(self):
            return "", ""

    for name in ("LIB", "LIB_DEBUG", "FRONT"):
        monkeypatch.setattr(build, name, str(tmp_path / getattr(build, name).split("/")[-1]))
    monkeypatch.setattr(build, "stale", lambda lib=None: True)
    monkeypatch.setattr(build.subprocess, "Popen", Popen)
    return names


LIBS = ["libdstopk.so", "libdstopk_debug.so"]


def test_builds_all_three(compiled):
    assert build.build() == build.LIB
    assert sorted(compiled) == ["_front.so", *LIBS]


def test_the_c_libraries_need_no_torch(compiled, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert build.build() == build.LIB
    assert sorted(compiled) == LIBS
    assert "_front.so is not built" in capsys.readouterr().err


def test_the_c_libraries_are_built_where_the_extension_cannot_be(compiled, monkeypatch):
    def fails(out):
        raise RuntimeError("g++ not found")

    monkeypatch.setattr(build, "front_command", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ not found"):
        build.build()
    assert sorted(compiled) == LIBS


def test_an_extension_for_another_torch_is_built_again(compiled, monkeypatch):
    build.build()
    assert not build.front_stale()
    here = build.front_tag()
    monkeypatch.setattr(build, "front_tag", lambda: here + "1")
    assert build.front_stale()
    build.build()
    assert compiled.count("_front.so") == 2 and not build.front_stale()


def test_an_extension_for_another_torch_is_not_loaded(compiled, monkeypatch):
    from sparse_attention_top_ds_b200 import _native
    build.build()
    with open(build.FRONT + ".tag", "w") as f:
        f.write("cpython-999, torch 0.1")
    monkeypatch.setattr(_native, "_front", None)
    monkeypatch.setattr(_native, "load", lambda: None)
    with pytest.raises(RuntimeError, match="built for cpython-999, torch 0.1, not for .*build it with"):
        _native._load_front()

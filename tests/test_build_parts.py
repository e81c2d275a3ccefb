"""The C library needs hipcc alone: it is linked whatever becomes of the Python
binding, which needs torch's headers and libraries. (Nothing is compiled here.)"""

import sys

import pytest

from agent_handoff_amd import build


@pytest.fixture
def made(monkeypatch):
    """Outputs in the order in which they were finished."""
    out = []

    def hipcc(srcs, target, *_, **__):
        out.append(target)
        return target

    monkeypatch.setattr(build, "_hipcc", hipcc)
    return out


def test_without_torch_the_library_is_linked_and_the_binding_left_out(made, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)   # importing it raises ImportError
    assert build.build() == build.LIB_PATH
    assert build.LIB_PATH in made and build.PROBE_LIB in made and build.BINDING_LIB not in made
    assert "torch" in capsys.readouterr().out


def test_a_binding_that_does_not_compile_fails_the_build_after_the_library(made, monkeypatch):
    def broken(*_):
        raise RuntimeError("binding")

    monkeypatch.setattr(build, "_binding", broken)
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert build.LIB_PATH in made and build.PROBE_LIB in made


def test_a_source_that_does_not_compile_fails_the_build(made, monkeypatch):
    def hipcc(srcs, target, *_, **__):
        if str(srcs[0]).endswith("page_kernels.hip"):
            raise RuntimeError("source")
        made.append(target)

    monkeypatch.setattr(build, "_hipcc", hipcc)
    with pytest.raises(RuntimeError, match="source"):
        build.build()
    assert build.LIB_PATH not in made

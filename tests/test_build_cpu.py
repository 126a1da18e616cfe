"""What the build does where torch is missing, or is another one than before."""
import os

import pytest

from paged_kv_gqa_append_gb300 import build as B

B.build()  # no-op when everything is up to date


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build of one host source into a folder of its own."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(B, "BINDING_LIB", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(B, "sources", lambda: [os.path.join(B.CSRC, "rope_scaling.cpp")])
    return tmp_path


def test_the_library_needs_no_torch(small, monkeypatch):
    find = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.is_stale()
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING_LIB)
    assert not B.is_stale()


def test_a_binding_that_does_not_compile_leaves_the_library(small, monkeypatch):
    def fails():
        raise RuntimeError("no Python.h")
    monkeypatch.setattr(B, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="no Python.h"):
        B.build()
    assert os.path.exists(B.LIB)


def test_another_torch_makes_the_binding_stale(small, monkeypatch):
    made = []
    monkeypatch.setattr(B, "_compile_binding", lambda: made.append(1) or "calls.o")

    def link(obj):
        for path, text in ((B.BINDING_LIB, ""), (B._stamp_path(), B._torch_stamp())):
            with open(path, "w") as f:
                f.write(text)
    monkeypatch.setattr(B, "_link_binding", link)
    B.build()
    assert len(made) == 1 and not B.is_stale()
    library = os.stat(B.LIB).st_mtime_ns
    monkeypatch.setattr(B.importlib.metadata, "version", lambda name: "0.0.1")
    assert B.is_stale()
    B.build()
    assert len(made) == 2 and os.stat(B.LIB).st_mtime_ns == library and not B.is_stale()


def test_the_loaded_binding_names_its_torch(monkeypatch):
    import paged_kv_gqa_append_gb300 as pkv
    module = pkv._load_calls()
    assert pkv.torch.__version__.startswith(module.torch_version)
    monkeypatch.setattr(pkv.torch, "__version__", "1.2.3+other")
    with pytest.raises(RuntimeError, match="torch 1.2.3|this is 1.2.3"):
        pkv._load_calls()

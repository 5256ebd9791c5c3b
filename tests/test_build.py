"""What the build makes without torch, without a compiler that takes the binding's module, and
after torch changed."""
import os

import pytest

from paged_kv_attention_21_gb300 import build as libbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A source tree of one small kernel and its build folder."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" __global__ void one(float* x) { x[threadIdx.x] = 1.f; }\n')
    (src / "marshal.cpp").write_text("int marshal() { return 0; }\n")
    out = tmp_path / "_build"
    monkeypatch.setattr(libbuild, "CSRC", str(src))
    monkeypatch.setattr(libbuild, "OUT_DIR", str(out))
    for name, file in (("LIB_PATH", "libpkv.so"), ("MARSHAL_PATH", "_marshal.so"), ("STAMP_PATH", "_marshal.for")):
        monkeypatch.setattr(libbuild, name, str(out / file), raising=False)
    return tmp_path


def test_the_library_is_built_without_torch(tree, monkeypatch):
    find = libbuild.importlib.util.find_spec
    monkeypatch.setattr(libbuild.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    assert not libbuild.up_to_date()
    assert libbuild.build() == libbuild.LIB_PATH
    assert os.path.exists(libbuild.LIB_PATH) and not os.path.exists(libbuild.MARSHAL_PATH)
    assert libbuild.up_to_date()


def test_the_library_is_linked_where_the_binding_does_not_compile(tree, monkeypatch):
    (tree / "csrc" / "marshal.cpp").write_text("#error not here\n")
    with pytest.raises(RuntimeError, match="not here"):
        libbuild.build()
    assert os.path.exists(libbuild.LIB_PATH)
    assert not libbuild.up_to_date()
    with pytest.raises(RuntimeError, match="not here"):
        libbuild.build()  # said again, not taken as done
    made = os.path.getmtime(libbuild.LIB_PATH)
    (tree / "csrc" / "marshal.cpp").write_text("int marshal() { return 0; }\n")
    libbuild.build()
    assert os.path.exists(libbuild.MARSHAL_PATH) and os.path.getmtime(libbuild.LIB_PATH) == made
    assert libbuild.up_to_date()


def test_another_torch_rebuilds_the_binding_alone(tree, monkeypatch):
    libbuild.build()
    assert libbuild.up_to_date()
    made = os.path.getmtime(libbuild.LIB_PATH)
    monkeypatch.setattr(libbuild.importlib.metadata, "version", lambda name: "0.0.1")
    assert not libbuild.up_to_date()
    os.utime(libbuild.MARSHAL_PATH, (1, 1))
    libbuild.build()
    assert libbuild.up_to_date() and os.path.getmtime(libbuild.LIB_PATH) == made
    assert os.path.getmtime(libbuild.MARSHAL_PATH) > 1

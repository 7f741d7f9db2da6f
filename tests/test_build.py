"""The build's optional part must not stand in the library's way."""
import os
import types

import pytest
import torch

from two_tower_block_b200 import build as b
from two_tower_block_b200 import ops


@pytest.mark.parametrize("why", ["no compiler", "no headers"])
def test_the_library_is_built_without_the_compiled_marshalling(why, monkeypatch, tmp_path):
    made = tmp_path / "marshal.so"
    monkeypatch.setattr(b, "MARSHAL", str(made))
    cmd = [str(tmp_path / "no-such-compiler")] if why == "no compiler" else ["false"]
    monkeypatch.setattr(b, "_marshal_cmd", lambda src: cmd)
    with pytest.warns(UserWarning, match="marshalling"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not made.exists()


def test_a_marshalling_of_another_torch_is_not_used():
    def module(**kw):
        return types.SimpleNamespace(addresses=len, **kw)
    assert ops._pick_quick(module(built_for=torch.__version__)) is len
    for other in (module(built_for="1.0"), module(), None):
        assert ops._pick_quick(other) is ops._quick_py


def test_it_is_built_again_for_another_torch_or_python(monkeypatch, tmp_path):
    src = os.path.join(b.CSRC, "marshal.cpp")
    b.build()
    assert b._marshal_is_current(src)
    assert ops._marshal.built_for == torch.__version__
    monkeypatch.setattr(b, "_torch_version", lambda: "1.0")
    assert not b._marshal_is_current(src)
    monkeypatch.undo()
    monkeypatch.setattr(b, "MARSHAL_FOR", str(tmp_path / "none"))
    assert not b._marshal_is_current(src)
    assert os.path.basename(b.MARSHAL).startswith("_marshal.") and b.MARSHAL != os.path.join(b.HERE, "_marshal.so")

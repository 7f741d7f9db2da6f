"""The build's optional part must not stand in the library's way."""
import os

import pytest

from two_tower_block_b200 import build as b


@pytest.mark.parametrize("why", ["no compiler", "no headers"])
def test_the_library_is_built_without_the_compiled_marshalling(why, monkeypatch, tmp_path):
    made = tmp_path / "marshal.so"
    monkeypatch.setattr(b, "MARSHAL", str(made))
    cmd = [str(tmp_path / "no-such-compiler")] if why == "no compiler" else ["false"]
    monkeypatch.setattr(b, "_marshal_cmd", lambda src: cmd)
    with pytest.warns(UserWarning, match="marshalling"):
        assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and not made.exists()

"""CPU checks of the build: what the packed cache does not need may be missing."""
import os
import sysconfig

import pytest

from packed_decode_attention_b200 import build as pkg_build


@pytest.mark.parametrize("what", ["headers", "compiler"])
def test_the_library_is_built_without_the_compiled_binding(monkeypatch, tmp_path, capsys, what):
    pkg_build.build()
    monkeypatch.setattr(pkg_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    if what == "headers":
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(sysconfig, "get_paths", lambda: paths)
    else:
        monkeypatch.setenv("CC", "no-such-compiler")
    assert pkg_build.build() == pkg_build.LIB
    assert not os.path.exists(pkg_build.MARSHAL)
    assert "_marshal.so not built" in capsys.readouterr().err


def test_the_compiled_binding_is_built(monkeypatch, tmp_path):
    pkg_build.build()
    monkeypatch.setattr(pkg_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    assert pkg_build.build_marshal() == pkg_build.MARSHAL and os.path.exists(pkg_build.MARSHAL)

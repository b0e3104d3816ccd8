"""The C library is built where the native binding cannot be (no host compiler,
or no torch or Python headers)."""
import os

import pytest

from gated_delta_rule_51_amd import build


def test_library_without_binding(tmp_path, monkeypatch):
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.hip").write_text('extern "C" int one() { return 1; }\n')

    def none():
        raise RuntimeError("no headers")

    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "OUT", str(tmp_path / "libone.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "_compile_binding", none)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert os.path.exists(build.OUT) and not os.path.exists(build.BINDING)

"""When the native libraries are built again: sources newer than they are, and another torch or Python than
the binding was compiled against."""
import os

import pytest


@pytest.fixture
def b(tmp_path, monkeypatch):
    from decode_attention_value_gb300 import _build

    _build.build()
    # a stand-in for the built files: the real ones stay as they are
    for name in ("LIB", "BINDING", "STAMP"):
        copy = tmp_path / os.path.basename(getattr(_build, name))
        copy.write_bytes(b"")
        monkeypatch.setattr(_build, name, str(copy))
    (tmp_path / os.path.basename(_build.STAMP)).write_text(_build._against())
    return _build


def test_the_real_build_is_up_to_date():
    from decode_attention_value_gb300 import _build

    _build.build()
    assert _build.up_to_date()


def test_another_torch_or_python_builds_again(b, monkeypatch):
    assert b.up_to_date()
    import torch

    known = b._against()
    assert torch.__version__ in known
    monkeypatch.setattr(b, "_against", lambda: known.replace(torch.__version__, "9.9.9+cu130"))
    assert not b.up_to_date()
    ran = []
    monkeypatch.setattr(b, "_nvcc", lambda: ran.append(1) or (_ for _ in ()).throw(RuntimeError("asked to compile")))
    with pytest.raises(RuntimeError, match="asked to compile"):
        b.build()
    assert ran


def test_unknown_origin_and_newer_sources_build_again(b):
    assert b.up_to_date()
    os.remove(b.STAMP)
    assert not b.up_to_date()
    with open(b.STAMP, "w") as f:
        f.write(b._against())
    assert b.up_to_date()
    os.utime(b.LIB, (1, 1))
    assert not b.up_to_date()

"""What the build step takes as up to date (CPU)."""
import os

import pytest

from fp8_block_scaled_scales_b200 import build


@pytest.fixture
def ext(tmp_path, monkeypatch):
    """An extension just built, its sources older."""
    for name in ("EXT", "EXT_SRC", "EXT_FOR"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
        (tmp_path / name).write_text("this torch")
    monkeypatch.setattr(build, "ROOT", str(tmp_path))
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "dg.h").write_text("")
    for path in (build.EXT_SRC, str(tmp_path / "include" / "dg.h")):
        os.utime(path, (1, 1))
    return tmp_path


def test_extension_is_kept_while_nothing_changes(ext):
    assert not build._ext_stale("this torch")


def test_extension_is_rebuilt_for_another_torch(ext):
    assert build._ext_stale("another torch")


@pytest.mark.parametrize("gone", ["EXT", "EXT_FOR"])
def test_extension_is_rebuilt_when_a_file_is_missing(ext, gone):
    (ext / gone).unlink()
    assert build._ext_stale("this torch")


@pytest.mark.parametrize("newer", ["EXT_SRC", "include/dg.h"])
def test_extension_is_rebuilt_after_its_sources(ext, newer):
    later = os.path.getmtime(build.EXT) + 10
    os.utime(ext / newer, (later, later))
    assert build._ext_stale("this torch")


def test_the_build_records_what_it_was_built_against():
    import torch

    build.build()
    with open(build.EXT_FOR) as f:
        text = f.read()
    assert torch.__version__ in text and not build._ext_stale(text)

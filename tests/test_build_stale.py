"""When the libraries are built again (CPU only: nothing is compiled here)."""

import os

import pytest

from sparse_attention_indexer_score_gb300 import build as B


@pytest.fixture
def built(tmp_path, monkeypatch):
    """Libraries newer than every source, built with this torch and Python."""
    for name in ("LIB", "BINDING", "BUILT_WITH"):
        path = tmp_path / name
        path.write_text("")
        monkeypatch.setattr(B, name, str(path))
    (tmp_path / "BUILT_WITH").write_text(B._tools())
    return tmp_path


def test_a_fresh_build_is_kept(built):
    assert not B._stale()


def test_another_torch_or_python(built, monkeypatch):
    import torch

    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert B._stale()


def test_another_place_of_torch(built):
    (built / "BUILT_WITH").write_text(B._tools().replace(os.sep, os.sep + "else"))
    assert B._stale()


@pytest.mark.parametrize("name", ["LIB", "BINDING", "BUILT_WITH"])
def test_anything_missing(built, name):
    (built / name).unlink()
    assert B._stale()


@pytest.mark.parametrize("name", ["LIB", "BINDING"])
def test_a_source_newer_than_a_library(built, name):
    os.utime(built / name, (1, 1))
    assert B._stale()

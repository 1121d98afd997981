"""The build: the C library needs neither PyTorch nor a C++ compiler for it, and a
binding made for another PyTorch is neither kept nor loaded."""

import os
import warnings

import pytest
import torch

from token_indexed_sparse_b200 import build, qsa


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _fails(*args, **kw):
    raise RuntimeError("no C++ compiler here")


@pytest.mark.parametrize("error", [RuntimeError, ImportError, OSError])
def test_the_library_is_built_without_the_binding(monkeypatch, error):
    def fails(force=False):
        raise error("not here")
    monkeypatch.setattr(build, "build_binding", fails)
    with pytest.warns(RuntimeWarning, match="binding is not"):
        assert build.build() == build.LIB and os.path.exists(build.LIB)


def test_the_library_comes_first(monkeypatch):
    order = []
    monkeypatch.setattr(build, "build_library", lambda force, verbose: order.append("library"))
    monkeypatch.setattr(build, "build_binding", lambda force: order.append("binding"))
    build.build()
    assert order == ["library", "binding"]


def test_another_pytorch_is_another_file(monkeypatch):
    here = build.binding_path()
    assert os.path.exists(here) and os.path.basename(here).startswith("_qsa_torch.")
    monkeypatch.setattr(torch, "__version__", "2.99.0")
    there = build.binding_path()
    assert there != here and not os.path.exists(there)
    # so it is built, not taken for up to date
    monkeypatch.setattr(build.subprocess, "run", _fails)
    with pytest.raises(RuntimeError, match="no C\\+\\+ compiler"):
        build.build_binding()
    monkeypatch.undo()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert build.build_binding() == here


@pytest.mark.parametrize("content", [None, b"not a shared object"])
def test_without_a_binding_the_calls_go_the_long_way(monkeypatch, tmp_path, content):
    path = tmp_path / "_qsa_torch.other.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(build, "binding_path", lambda: str(path))
    monkeypatch.setattr(qsa, "_short", None)
    x, i = torch.zeros(2, 12, 256, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="does not load"):
        with pytest.raises(ValueError, match="CUDA"):   # the long way's own refusal
            qsa.rope(x, None, i, torch.ones(8, dtype=torch.float64))
    with warnings.catch_warnings():                     # said once
        warnings.simplefilter("error")
        pages = torch.zeros(1, 16, 1, 256, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="CUDA"):
            qsa.paged_causal(x, pages, pages, i[None], i[:1], i)
        for name in ("rope", "cache_append", "paged_forward", "paged_causal"):
            assert getattr(qsa._short_way(), name)(1, 2) is NotImplemented

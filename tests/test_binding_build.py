"""The compiled binding is built for one torch and one Python, and is neither
taken for up to date nor loaded under another."""
import os
import sysconfig

import pytest
import torch

import exact_attention_109_b200 as fa
from exact_attention_109_b200 import build


@pytest.fixture
def other_torch(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    monkeypatch.setattr(fa.api, "_binding", None)


def test_the_file_names_what_it_is_built_for():
    build.build()
    path = build.binding_path()
    assert torch.__version__ in path and path.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert os.path.samefile(fa.api._native().__file__, path)


def test_another_torch_finds_no_binding(other_torch):
    with pytest.raises(fa.FaError, match="not built"):
        fa.paged_append(*[None] * 8)


def test_another_torch_builds_its_own(other_torch, monkeypatch):
    ran = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, check: ran.append(cmd))
    monkeypatch.setattr(build, "up_to_date", lambda out=build.OUT, sources=None:
                        os.path.exists(out))
    build.build()
    assert len(ran) == 1 and ran[0][0] == "g++"
    assert ran[0][ran[0].index("-o") + 1] == build.binding_path()
    assert "9.9.9+other" in build.binding_path()


def test_a_file_that_does_not_load_is_an_error(monkeypatch, tmp_path):
    bad = tmp_path / "_fa_binding.so"
    bad.write_bytes(b"not a library")
    monkeypatch.setattr(build, "binding_path", lambda: str(bad))
    monkeypatch.setattr(fa.api, "_binding", None)
    with pytest.raises(fa.FaError, match="does not load"):
        fa.paged_append(*[None] * 8)

"""Building the Python calls of the paged KV cache (build.build_binding): no need of them for the codec, and rebuilt for another torch."""
import os

import pytest

from entropy_coded_lossless_b200 import build as shn_build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The binding and its record in another folder, so that the tree's own stay."""
    shn_build.build()
    monkeypatch.setattr(shn_build, "BINDING", str(tmp_path / "_kv.so"))
    monkeypatch.setattr(shn_build, "BINDING_TORCH", str(tmp_path / "torch"))
    return tmp_path


@pytest.mark.parametrize("old", [False, True])
def test_the_codec_builds_without_what_the_binding_needs(elsewhere, monkeypatch, old):
    monkeypatch.setenv("CXX", str(elsewhere / "no-such-compiler"))
    if old:  # one of other sources or another torch, which would not fit
        (elsewhere / "_kv.so").write_bytes(b"")
    with pytest.warns(RuntimeWarning, match="_kv.so"):
        assert shn_build.build() == shn_build.LIB
    assert os.path.exists(shn_build.LIB) and not os.path.exists(shn_build.BINDING)
    with pytest.raises(OSError):
        shn_build.build_binding()


def test_the_binding_is_rebuilt_for_another_torch(elsewhere, monkeypatch):
    runs = []

    def compile(cmd):
        runs.append(cmd)
        (elsewhere / "_kv.so").write_bytes(b"")

    monkeypatch.setattr(shn_build.subprocess, "check_call", compile)
    shn_build.build_binding()
    shn_build.build_binding()
    assert len(runs) == 1
    monkeypatch.setattr(shn_build, "_torch_version", lambda: "another")
    shn_build.build_binding()
    shn_build.build_binding()
    assert len(runs) == 2

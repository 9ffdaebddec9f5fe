"""When the binding's short way is built again."""
import os

import pytest
import torch

from attn_fwd_04_b200 import build as fa_build


def test_calls_are_built_again_for_another_torch(monkeypatch, tmp_path):
    runs = []

    def run(cmd, check):
        runs.append(cmd)
        with open(fa_build.CALLS, "w") as f:
            f.write("x")

    monkeypatch.setattr(fa_build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(fa_build, "CALLS_TORCH", str(tmp_path / "notes" / "calls.torch"))
    monkeypatch.setattr(fa_build.subprocess, "run", run)
    fa_build._build_calls(False, False)
    assert len(runs) == 1  # there was none
    fa_build._build_calls(False, False)
    assert len(runs) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    fa_build._build_calls(False, False)
    assert len(runs) == 2  # one of another torch
    fa_build._build_calls(False, False)
    assert len(runs) == 2
    os.remove(fa_build.CALLS_TORCH)
    fa_build._build_calls(False, False)
    assert len(runs) == 3  # one that nothing is known of
    fa_build._build_calls(True, False)
    assert len(runs) == 4


def test_calls_of_another_torch_are_refused(monkeypatch):
    from attn_fwd_04_b200 import fa as binding

    fa_build.build()
    monkeypatch.setattr(binding, "_short_calls", None)
    binding._short()  # of this one
    monkeypatch.setattr(binding, "_short_calls", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0+cu1")
    with pytest.raises(ImportError, match="another torch"):
        binding._short()

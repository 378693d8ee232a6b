"""Build steps, with the compilers replaced: the CUDA libraries need neither torch
nor a working host compiler step."""
import importlib.util
import os
import subprocess

import pytest


@pytest.fixture
def steps(monkeypatch, tmp_path):
    from nvfp4_weight_only_router_b200 import build
    for name, file in (("LIB", "libnvfp4moe.so"), ("DENSE_LIB", "libnvfp4dense.so"), ("DENSE_CALLS", "_dense_calls.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")

    def run(cmd, verbose):
        if cmd[0] in run.missing:
            raise subprocess.CalledProcessError(1, cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    run.missing = ()
    monkeypatch.setattr(build, "_run", run)
    return build, run, tmp_path


def _built(tmp_path):
    return sorted(f for f in os.listdir(tmp_path) if f.endswith(".so"))


def test_all_is_built(steps):
    build, _, out = steps
    assert build.build() == build.LIB
    assert _built(out) == ["_dense_calls.so", "libnvfp4dense.so", "libnvfp4moe.so"]


def test_without_torch_the_c_libraries_are_built(steps, monkeypatch):
    build, run, out = steps
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    run.missing = ("g++",)
    assert build.build() == build.LIB
    assert _built(out) == ["libnvfp4dense.so", "libnvfp4moe.so"]


def test_a_failed_host_compiler_is_reported_behind_the_c_libraries(steps):
    build, run, out = steps
    run.missing = ("g++",)
    with pytest.raises(subprocess.CalledProcessError):
        build.build()
    assert _built(out) == ["libnvfp4dense.so", "libnvfp4moe.so"]
    # and the next call tries again
    run.missing = ()
    build.build()
    assert "_dense_calls.so" in _built(out)

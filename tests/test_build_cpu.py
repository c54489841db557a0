"""What a build makes, and when it makes it again (no compiler runs here)."""

import importlib.util
import os

import pytest

from paged_kv_cache_209_gb300 import build


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """A tree whose outputs are all there; what a build would compile and link is collected instead."""
    done = []
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_pkv_calls.so"))

    def write(path):
        os.makedirs(os.path.dirname(path), exist_ok=True)
        with open(path, "w"):
            pass

    def compile_(src, obj, extra):
        done.append(os.path.basename(src))
        write(obj)
        return src, 0, ""

    class Run:
        returncode, stdout, stderr = 0, "", ""

        def __init__(self, cmd, **kw):
            out = cmd[cmd.index("-o") + 1]
            done.append(os.path.basename(out))
            write(out)
    monkeypatch.setattr(build, "_compile", compile_)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build.subprocess, "run", Run)
    return done


def test_everything_once(compiled):
    build.build()
    assert {"pkv_q4.cu", "pkv_pool.cpp", "libpkv.so", "_pkv_calls.so"} <= set(compiled)
    compiled.clear()
    build.build()
    assert compiled == []


def test_without_torch_the_library_is_built_alone(compiled, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    build.build()
    assert "libpkv.so" in compiled and "_pkv_calls.so" not in compiled


def test_other_flags_build_everything_again(compiled, monkeypatch):
    build.build()
    compiled.clear()
    at = os.path.getmtime
    monkeypatch.setattr(build.os.path, "getmtime", lambda p: at(p) + (1e6 if p == os.path.abspath(build.__file__) else 0))
    build.build()
    assert {"pkv_q4.cu", "_pkv_calls.so"} <= set(compiled)

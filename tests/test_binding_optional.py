"""The library without its C++ binding: a host whose torch has no headers, or another
torch than the one that the binding was built for, keeps every call."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

import prep_token_gb300 as dp
from prep_token_gb300 import _build


@pytest.fixture(scope="module")
def alone(tmp_path_factory):
    """A copy of the package with its library and no binding."""
    _build.build_library()
    at = tmp_path_factory.mktemp("alone")
    shutil.copytree(_build.PKG, at / "prep_token_gb300",
                    ignore=lambda _, names: [n for n in names if n.startswith("_binding")
                                             or n in ("csrc", "__pycache__")])
    return at


CALLS = """
import warnings, torch
import prep_token_gb300 as dp
with warnings.catch_warnings():
    warnings.simplefilter("error")
    lib = dp.library()
    assert dp.dsa_status_string(0) and dp.dsa_paged_attention_max_workspace_bytes(128) > 0
    assert lib.dsa_cache_free(0, *[None] * 2, 0, 0, None, 0, 0, None, 0, 0, 0, 0, None, None) == 3
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    for _ in range(2):
        for name in ("rms_norm", "kv_append", "tree_attention", "cache_keep"):
            assert getattr(dp._marshal(), name)() is NotImplemented
        try:
            dp.dsa_rms_norm(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(64), 1e-6)
        except ValueError as e:
            assert "CUDA" in str(e)
        else:
            raise AssertionError
assert [w.category for w in seen] == [RuntimeWarning] and "ctypes" in str(seen[0].message)
print("done")
"""


def run(at):
    got = subprocess.run([sys.executable, "-c", CALLS], cwd=at, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(at)})
    assert got.returncode == 0 and got.stdout.strip() == "done", got.stderr


def test_every_call_without_it(alone):
    run(alone)


@pytest.mark.parametrize("content", [b"", b"not a shared library"])
def test_one_that_does_not_load(alone, content):
    # under its name and under one without versions
    for path in {os.path.basename(getattr(_build, "binding_path", lambda: "_binding.so")()),
                 "_binding.so"}:
        (alone / "prep_token_gb300" / path).write_bytes(content)
    run(alone)


def test_another_torch_has_another_binding(monkeypatch):
    here = _build.binding_path()
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    assert _build.binding_path() != here and "1.2.3" in _build.binding_path()


def test_built_without_headers(monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(_build, "PKG", str(tmp_path))  # where the binding goes
    monkeypatch.setattr(_build, "_torch_include", lambda: str(tmp_path / "none"))
    assert _build.build_library() == _build.LIB_PATH
    assert os.listdir(tmp_path) == []
    assert "is not built" in capsys.readouterr().err


@pytest.mark.parametrize("ends", ["library", "binding"])
def test_a_build_that_fails_leaves_no_file(monkeypatch, tmp_path, ends):
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    code = 0 if ends == "library" else 3
    monkeypatch.setattr(_build, "_binding_command", lambda out: [
        sys.executable, "-c", f"open({out!r}, 'w').close(); raise SystemExit({code})"])
    monkeypatch.setattr(_build, "_stale", lambda: ends == "library")

    def fail(*_):
        raise subprocess.CalledProcessError(1, "nvcc")
    monkeypatch.setattr(_build, "_build_cuda", fail)
    with pytest.raises(subprocess.CalledProcessError):
        _build.build_library()
    assert os.listdir(tmp_path) == []


def test_the_one_that_was_built():
    """It loads, and has the calls that are marshalled through it."""
    _build.build_library()
    if not os.path.exists(_build.binding_path()):
        pytest.skip("torch's headers are not installed")
    for name in ("rms_norm", "kv_append", "tree_attention", "cache_keep"):
        assert getattr(dp._load_binding(), name)() is NotImplemented

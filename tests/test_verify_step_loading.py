"""The verify step's native module is no part of the other calls: the library loads and builds without it."""
import os
import subprocess
import sys

import pytest

from nvfp4_speculative_draft_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def run(code):
    """In a process of its own: the module and what it is bound to live as long as the process."""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_library_loads_without_the_binding():
    run("""
import ctypes, torch
import nvfp4_speculative_draft_gb300 as nd
from nvfp4_speculative_draft_gb300 import build
real = build.binding_path
build.binding_path = lambda: "/nonexistent/_binding.so"
L = nd.load()
ex = nd._Exec(None, None, 0, None)
assert L.nvfp4_quantize(None, 4, 64, None, None, None, None, ctypes.byref(ex)) == 1
assert L.fp8b_quantize(None, 4, 64, 64, None, None, ctypes.byref(ex)) == 1
w = torch.zeros((4, 64), dtype=torch.bfloat16)
try:
    nd.nvfp4_quantize(w)
except ValueError as e:  # its own check
    assert "CUDA" in str(e)
for call in (lambda: nd.fp8b_quantize(w), lambda: nd.fp8b_rmsnorm(w, None), lambda: nd.fp8b_gemm(None, None),
             lambda: nd.spec_verify(w, w, w, w)):
    try:
        call()
        raise SystemExit("not refused")
    except ImportError as e:
        assert "binding not built" in str(e)
build.binding_path = real  # built meanwhile: the next call finds it
try:
    nd.fp8b_quantize(w)
    raise SystemExit("not refused")
except ValueError as e:
    assert "CUDA" in str(e)
""")


def test_calls_before_bind_are_refused():
    run("""
import nvfp4_speculative_draft_gb300 as nd
native = nd._load_binding()
for f, n in ((native.quantize, 5), (native.rmsnorm, 8), (native.gemm, 6), (native.verify, 10)):
    try:
        f(*[None] * n)
        raise SystemExit("not refused")
    except TypeError as e:
        assert "bind" in str(e)
nd._native()
for f, n in ((native.quantize, 5), (native.rmsnorm, 8), (native.verify, 10)):
    try:
        f(*[None] * n)
        raise SystemExit("not refused")
    except ValueError as e:
        assert "CUDA" in str(e)
""")


def test_build_warns_where_the_binding_does_not_compile(monkeypatch):
    def fails(force=False):
        raise RuntimeError("no headers")
    monkeypatch.setattr(build, "build_binding", fails)
    with pytest.warns(RuntimeWarning, match="no headers"):
        assert build.build() == build.LIB


def test_build_without_a_compiler_leaves_no_old_binding(monkeypatch, tmp_path):
    target = tmp_path / "_binding.so"
    target.write_bytes(b"old")
    monkeypatch.setattr(build, "binding_path", lambda: str(target))
    monkeypatch.setenv("PATH", str(tmp_path))
    with pytest.raises(RuntimeError, match=r"g\+\+"):
        build.build_binding(force=True)
    assert not target.exists()

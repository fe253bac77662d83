"""The C entries of the grouped router, the 8-bit products and the gradient norm when the host runs out of memory: a
status, not an exception that leaves a C function. A small library whose operator new fails on demand is loaded in
front of the C++ one, in a process of its own; nothing is launched."""
import os
import shutil
import subprocess
import sys

import pytest

from test_exceptions_host import FAILING_NEW, ROOT

CHILD = r"""
import ctypes, struct, sys
import pack_virtual_rank_gb300 as rv
L, fail = rv.lib(), ctypes.CDLL(sys.argv[1]).fail_new
words = bytes(200)
one = ctypes.c_void_p(1 << 40)
ptr, count, dtype = (ctypes.c_void_p * 1)(1 << 40), (ctypes.c_size_t * 1)(8), (ctypes.c_int32 * 1)(0)
g = rv.RelayGrads(1, ptr, count, dtype)
bad = rv.RelayGrads(-1, ptr, count, dtype)
how = struct.pack("7if", 7, 1, 1, 1, 1, 1, 1, 1.0)
prod = struct.pack("12q4i", 1 << 40, 128, 1 << 41, 1 << 42, 128, 1 << 43, 1 << 40, 128, 8, 8, 128, 0, 0, 0, 0, 0)
calls = {
    "grouped forward": lambda: L.relay_packed_grouped_forward(how, words),
    "grouped backward": lambda: L.relay_packed_grouped_backward(how, words),
    "bias": lambda: L.relay_router_bias_update(None, None, 0, 0.0, None, None),
    "depth": lambda: L.relay_fp8_depth(-1, 0),
    "quantize": lambda: L.relay_quantize_fp8(words, None),
    "matmul": lambda: L.relay_matmul_fp8(prod, None),
    "wait": lambda: L.relay_test_fp8_wait(words, -1, None),
    "grad workspace": lambda: L.relay_grad_workspace_size(ctypes.byref(bad)),
    "norm": lambda: L.relay_grad_norm(ctypes.byref(g), one, one, 1 << 20, None),
    "clip": lambda: L.relay_grad_clip(ctypes.byref(g), None, one, 1.0, None),
}
for name, call in calls.items():
    assert call() != 0, name
    before = L.relay_last_error()
    fail(1)
    st = call()
    fail(0)
    assert st in (-1, rv.ERR_CUDA), (name, st)
    assert L.relay_last_error() != before, name     # not the text of another error
    assert call() != 0 and L.relay_last_error() == before, name
    print("ok", name, flush=True)
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_no_exception_leaves_a_c_entry(relay_lib, tmp_path):
    src, lib = tmp_path / "failing_new.cpp", tmp_path / "failing_new.so"
    src.write_text(FAILING_NEW)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    env = dict(os.environ, LD_PRELOAD=str(lib), PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD, str(lib)], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.count("ok ") == 10

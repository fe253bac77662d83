"""The C entries of the losses and the router when the host runs out of memory: a status, not an exception that
leaves a C function (which ends the process). A small library whose operator new fails on demand is loaded in front of
the C++ one, in a process of its own; nothing is launched."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAILING_NEW = r"""
#include <cstdlib>
#include <new>
static thread_local bool failing = false;
extern "C" void fail_new(int on) { failing = on != 0; }
static void* take(std::size_t n) {
  void* p = failing ? nullptr : std::malloc(n ? n : 1);
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void* operator new(std::size_t n) { return take(n); }
void* operator new[](std::size_t n) { return take(n); }
void operator delete(void* p) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t) noexcept { std::free(p); }
"""

CHILD = r"""
import ctypes, sys
import pack_virtual_rank_gb300 as rv
L, fail = rv.lib(), ctypes.CDLL(sys.argv[1]).fail_new
words = (ctypes.c_int64 * 16)()
calls = {
    "xent": lambda: L.relay_linear_xent(None, None, None, None, None, 0, None),
    "distill": lambda: L.relay_linear_distill(None, None, 0, None, 1, 1.0, None, None, None, 0, None),
    "distill top": lambda: L.relay_linear_distill(None, None, 0, None, 0, 1.0, None, None, None, 0, None),
    "workspace": lambda: L.relay_head_workspace_size(None, 0),
    "wait": lambda: L.relay_test_head_wait(None, None, None, None, 0, -1, None),
    "forward": lambda: L.relay_router_forward(None, 0, 7, 0, 1, 1, 0, None, None, None, None, None, None, 0, None),
    "balance": lambda: L.relay_balance_loss(None, None, 0, 1, 1.0, None, None, None),
    "backward": lambda: L.relay_router_backward(None, 0, 7, 0, 1, 1, 0, None, None, None, None, 0, None),
    "router workspace": lambda: L.relay_router_workspace_size(-1, 1),
    "packed": lambda: L.relay_packed_router_balance(bytes(words)),
}
for name, call in calls.items():
    assert call() != 0
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

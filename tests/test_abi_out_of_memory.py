"""No C++ exception crosses the C ABI when host memory runs out: psgd.h says so, and an
exception that left an entry point would end the process.

A child process preloads an operator new that fails on request.  Every entry point is then
called in ways that end before any HIP call, with the n-th allocation and all later ones
failing, for every n until the call gets along: it has to return PSGD_ERR_NO_MEMORY until
then.  CPU only."""

import os
import shutil
import subprocess
import sys

import pytest

pytestmark = pytest.mark.usefixtures("built_library")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAILING_NEW = r"""
#include <cstdlib>
#include <new>
static thread_local long left = -1;  // allocations that still succeed; -1: all
extern "C" void new_fails_after(long n) { left = n; }
static void* get(std::size_t n) {
  if (left == 0) throw std::bad_alloc();
  if (left > 0) --left;
  void* p = std::malloc(n ? n : 1);
  if (p == nullptr) throw std::bad_alloc();
  return p;
}
void* operator new(std::size_t n) { return get(n); }
void* operator new[](std::size_t n) { return get(n); }
void* operator new(std::size_t n, const std::nothrow_t&) noexcept {
  try { return get(n); } catch (...) { return nullptr; }
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete[](void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }
void operator delete[](void* p, std::size_t) noexcept { std::free(p); }
"""

CHILD = r"""
import ctypes, sys
from distributed_sgd_gradient_ef_amd import psgd
fails = ctypes.CDLL(sys.argv[1]).new_fails_after
fails.argtypes = [ctypes.c_long]
fails.restype = None
lib = psgd.load_library()
OK, INVALID, UNSUPPORTED, NO_MEMORY = 0, psgd.PSGD_ERR_INVALID_ARG, psgd.PSGD_ERR_UNSUPPORTED, psgd.PSGD_ERR_NO_MEMORY
h = ctypes.c_void_p()
out = ctypes.byref(h)
i64 = lambda *v: (ctypes.c_int64 * len(v))(*v)
layers = lambda *s: (psgd._Layer * len(s))(*[psgd._Layer(r, c) for r, c in s])
good, bad = layers((40, 30), (1, 9), (300, 70)), layers((40, 30), (0, 9))
tops, keeps, none = i64(50, 9, 100), i64(20, 3, 10), i64(20, 0, 10)
long_matrix = layers((2000, 1100))

CREATE = {
    "psgd_plan": lambda l, n: lib.psgd_plan_create(l, n, 2, 3, 0, 0, out),
    "psgd_rtopk_plan": lambda l, n: lib.psgd_rtopk_plan_create(l, n, tops, keeps, 3, 0, 0, out),
    "psgd_atomo_plan": lambda l, n: lib.psgd_atomo_plan_create(l, n, 1.5, 3, 0, out),
    "psgd_clip_plan": lambda l, n: lib.psgd_clip_plan_create(l, n, 3, 0, 0, out),
}

def sweep(name, call, want):
    for n in range(10000):
        h.value = None
        fails(n)
        try:
            status = call()
        finally:
            fails(-1)
        if status != NO_MEMORY:
            assert status == want, (name, n, status)
            print(name, n, flush=True)
            return
        assert not h.value, (name, n)
        assert lib.psgd_last_error()
    raise AssertionError(name)

plans = {}
for kind, create in CREATE.items():
    sweep(kind + "_create", lambda: create(good, 3), OK)
    plans[kind] = h.value
    sweep(kind + "_create: refused layer", lambda: create(bad, 2), INVALID)
    sweep(kind + "_create: no layers", lambda: create(good, 0), INVALID)
    sweep(kind + "_create: NULL", lambda: create(None, 3), INVALID)
    sweep(kind + "_sizes", lambda: getattr(lib, kind + "_sizes")(None, None), INVALID)
    sweep(kind + "_layer_info", lambda: getattr(lib, kind + "_layer_info")(plans[kind], 0, None), INVALID)
    sweep(kind + "_set_timing", lambda: getattr(lib, kind + "_set_timing")(None, 1), INVALID)
    sweep(kind + "_kernel_stats", lambda: getattr(lib, kind + "_kernel_stats")(plans[kind], None, 3, None, 0), INVALID)
    sweep(kind + "_kernel_stats: none", lambda: getattr(lib, kind + "_kernel_stats")(plans[kind], None, 0, None, 0), OK)
sweep("psgd_plan_create: rank", lambda: lib.psgd_plan_create(good, 3, 9, 3, 0, 0, out), UNSUPPORTED)
sweep("psgd_rtopk_plan_create: keep", lambda: lib.psgd_rtopk_plan_create(good, 3, tops, none, 3, 0, 0, out), INVALID)
sweep("psgd_atomo_plan_create: k", lambda: lib.psgd_atomo_plan_create(long_matrix, 1, 1.5, 3, 0, out), UNSUPPORTED)

p, r, a, c = (plans[k] for k in CREATE)
A = [0x10000000 * (i + 1) for i in range(12)]
cfg = ctypes.byref(psgd.AdamwConfig(max_norm=-1.0))
for name, call in {
    "psgd_plan_set_power_iterations": lambda: lib.psgd_plan_set_power_iterations(p, 99),
    "psgd_plan_reset_carry": lambda: lib.psgd_plan_reset_carry(None),
    "psgd_plan_reset_carry_stream": lambda: lib.psgd_plan_reset_carry_stream(p, None, None),
    "psgd_errors_materialize": lambda: lib.psgd_errors_materialize(p, A[0], A[0] + 16, A[1], None),
    "psgd_stream_copy": lambda: lib.psgd_stream_copy(A[0], A[0] + 16, 64, None),
    "psgd_compress_step": lambda: lib.psgd_compress_step(p, A[0], A[1], A[2], A[3], A[4], A[4] + 16, None),
    "psgd_compress_step: NULL": lambda: lib.psgd_compress_step(p, None, A[1], A[2], A[3], A[4], A[5], None),
    "psgd_compress_step_noalloc": lambda: lib.psgd_compress_step_noalloc(None, *A[:5], None),
    "psgd_ef_momentum_apply": lambda: lib.psgd_ef_momentum_apply(p, *A[:6], 1e999, 0.9, A[7], A[8], None),
    "psgd_rtopk_step": lambda: lib.psgd_rtopk_step(r, A[0], A[0], *A[2:7], None),
    "psgd_rtopk_step: NULL": lambda: lib.psgd_rtopk_step(r, A[0], None, *A[2:7], None),
    "psgd_rtopk_errors_materialize": lambda: lib.psgd_rtopk_errors_materialize(r, A[0], A[0] + 16, A[1], None),
    "psgd_rtopk_plan_reset_state": lambda: lib.psgd_rtopk_plan_reset_state(r, 8, None),
    "psgd_atomo_step": lambda: lib.psgd_atomo_step(a, A[0], A[0], *A[2:9], None),
    "psgd_atomo_step: NULL": lambda: lib.psgd_atomo_step(a, A[0], None, *A[2:9], None),
    "psgd_grad_norm": lambda: lib.psgd_grad_norm(c, A[0], 0, A[0], None, A[1], None),
    "psgd_grad_clip": lambda: lib.psgd_grad_clip(c, A[0], A[1], 0, -1.0, A[2], A[3], A[4], None),
    "psgd_adamw_apply": lambda: lib.psgd_adamw_apply(c, cfg, *A[:8], None),
}.items():
    sweep(name, call, INVALID)
for kind, handle in plans.items():
    assert getattr(lib, kind + "_destroy")(handle) == OK
print("done")
"""


def test_no_exception_leaves_an_entry_point(tmp_path):
    gxx = shutil.which("g++")
    assert gxx, "g++ is part of the toolchain"
    src, lib = tmp_path / "failing_new.cpp", tmp_path / "failing_new.so"
    src.write_text(FAILING_NEW)
    subprocess.run([gxx, "-O1", "-shared", "-fPIC", str(src), "-o", str(lib)], check=True)
    preload = ":".join(p for p in (str(lib), os.environ.get("LD_PRELOAD")) if p)
    env = {**os.environ, "LD_PRELOAD": preload, "PYTHONPATH": ROOT}
    res = subprocess.run([sys.executable, "-c", CHILD, str(lib)], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=120)
    assert res.returncode == 0 and res.stdout.endswith("done\n"), (res.returncode, res.stdout[-1500:], res.stderr[-2000:])

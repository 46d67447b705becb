"""The language-model part of the C ABI without a GPU: plan validation, the packed layout, and
argument checks that happen before any device call (the fake addresses below are never
dereferenced); no exception leaves an entry point when host memory runs out."""

import ctypes
import math
import os
import shutil
import subprocess
import sys

import pytest

from distributed_sgd_gradient_ef_amd import psgd
from tests.test_abi_out_of_memory import FAILING_NEW, ROOT

pytestmark = pytest.mark.usefixtures("built_library")

SHAPES = [(7, 9), (501, 40), (1, 40)]
INVALID, UNSUPPORTED = psgd.PSGD_ERR_INVALID_ARG, psgd.PSGD_ERR_UNSUPPORTED
A = {name: 0x100000000 * (i + 1) for i, name in enumerate(
    ["x", "params", "rows", "losses", "lse", "mean", "scale", "dx", "grads", "workspace", "out", "step"])}


def _status(fn, *args, **kw):
    with pytest.raises(psgd.PsgdError) as e:
        fn(*args, **kw)
    assert str(e.value)
    return e.value.status


@pytest.mark.parametrize("args,expect", [
    (([], 0, 1, 1), INVALID), ((SHAPES, -1, 1, 1), INVALID), ((SHAPES, 3, 1, 1), INVALID), ((SHAPES, 1, 0, 1), INVALID),
    ((SHAPES, 1, 65536, 1), INVALID), ((SHAPES, 1, 1, 0), INVALID), ((SHAPES, 1, 1, (1 << 23) + 1), INVALID),
    ((SHAPES, 1, 4, (1 << 21) + 1), INVALID), (([(0, 5)], 0, 1, 1), INVALID), (([(5, -1)], 0, 1, 1), INVALID),
    (([(65536, 32768)], 0, 1, 1), INVALID), (([(1 << 40, 1 << 40)], 0, 1, 1), INVALID),
    (([((1 << 31) - 1, 1)], 0, 1, 1), INVALID),           # over 2^23 blocks of the table
    (([(1, 1 << 20)], 0, 1, 1 << 20), INVALID),           # ... and of the rows
    (([(1, (1 << 23) + 1)], 0, 1, 1), INVALID),
    ((SHAPES, 1, 1, 1, 7), UNSUPPORTED), ((SHAPES, 1, 1, 1, 0, 7), UNSUPPORTED), ((SHAPES, 1, 1, 1, 0, 0, 1), UNSUPPORTED),
])
def test_plan_create_refuses(args, expect):
    assert _status(psgd.psgd_lm_plan_create, *args) == expect


def test_null_arguments():
    lib = psgd.load_library()
    h = ctypes.c_void_p()
    arr = (psgd._Layer * 1)(psgd._Layer(4, 4))
    assert lib.psgd_lm_plan_create(arr, 1, 0, 1, 1, 0, 0, 0, None) == INVALID
    assert lib.psgd_lm_plan_create(None, 1, 0, 1, 1, 0, 0, 0, ctypes.byref(h)) == INVALID
    assert lib.psgd_lm_plan_sizes(None, None) == INVALID
    assert lib.psgd_lm_plan_set_timing(None, 1) == INVALID
    assert lib.psgd_lm_plan_kernel_stats(None, None, 0, None, 0) == INVALID
    assert lib.psgd_lm_plan_destroy(None) == psgd.PSGD_OK
    plan = psgd.psgd_lm_plan_create(SHAPES, 1, 2, 3)
    assert psgd.psgd_lm_plan_kernel_stats(plan) == {}
    assert lib.psgd_lm_plan_kernel_stats(plan.handle, None, 4, None, 0) == INVALID


@pytest.mark.parametrize("table", [0, 1, 2])
@pytest.mark.parametrize("act,grad", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_layout_is_that_of_the_compressors(table, act, grad):
    plan = psgd.psgd_lm_plan_create(SHAPES, table, 3, 50, act, grad)
    clip = psgd.psgd_clip_plan_create(SHAPES, 3)
    s = plan.sizes
    assert s["worker_stride"] == clip.sizes["worker_stride"] and s["table_offset"] == clip.layers[table].offset
    assert (s["vocab"], s["dim"]) == SHAPES[table] and (s["n_workers"], s["rows"], s["table"]) == (3, 50, table)
    assert (s["act_dtype"], s["grad_dtype"], s["n_layers"]) == (act, grad, 3) and s["workspace_bytes"] % 256 == 0


def test_workspace_holds_a_piece_of_the_gradient_at_most():
    """The gradient by the scores of 8192 rows of a 131,072-word vocabulary is 2 GiB in bfloat16."""
    plan = psgd.psgd_lm_plan_create([(131072, 64)], 0, 1, 8192, psgd.PSGD_BF16, psgd.PSGD_BF16)
    assert plan.sizes["workspace_bytes"] < 600 << 20


CALLS = {
    "embed": (["params", "rows", "drop", "out"], lambda lib: lib.psgd_lm_embed),
    "embed_grad": (["rows", "x", "drop", "grads", "flags", "workspace"], lambda lib: lib.psgd_lm_embed_grad),
    "loss": (["x", "params", "rows", "drop", "losses", "lse", "mean", "workspace"], lambda lib: lib.psgd_lm_loss),
    "loss_grad": (["x", "params", "rows", "lse", "scale", "drop", "dx", "grads", "flags", "workspace"],
                  lambda lib: lib.psgd_lm_loss_grad),
}


def _call(which, plan, **bad):
    names, fn = CALLS[which]
    lib = psgd.load_library()
    a = {**A, "drop": None, "flags": 0, **bad}
    return fn(lib)(None if plan is None else plan.handle, *[a[n] for n in names], None)


@pytest.mark.parametrize("which", sorted(CALLS))
def test_calls_refuse_bad_pointers(which):
    plan = psgd.psgd_lm_plan_create(SHAPES, 1, 2, 33)
    names = [n for n in CALLS[which][0] if n not in ("drop", "flags")]
    assert _call(which, None) == INVALID
    for n in names:
        if n not in ("scale", "dx", "grads") or which == "embed_grad" and n == "grads":
            assert _call(which, plan, **{n: None}) == INVALID, n
        assert _call(which, plan, **{n: A[n] + (2 if n in ("x", "lse", "dx", "out", "losses", "mean", "scale") else 4)}) == INVALID, n
        for m in names:
            if m != n:
                assert _call(which, plan, **{n: A[m]}) == INVALID, (n, m)
    assert psgd.load_library().psgd_last_error()


def test_loss_grad_needs_an_output():
    plan = psgd.psgd_lm_plan_create(SHAPES, 1, 2, 33)
    assert _call("loss_grad", plan, dx=None, grads=None) == INVALID


@pytest.mark.parametrize("which", ["embed_grad", "loss_grad"])
def test_unknown_flags(which):
    assert _call(which, psgd.psgd_lm_plan_create(SHAPES, 1, 2, 33), flags=2) == UNSUPPORTED


@pytest.mark.parametrize("which", sorted(CALLS))
def test_bad_dropout(which):
    plan = psgd.psgd_lm_plan_create(SHAPES, 1, 2, 33)
    for p in (-0.1, 1.0000001, math.nan, math.inf):
        assert _call(which, plan, drop=ctypes.byref(psgd.DropoutConfig(p))) == INVALID
    c = psgd.DropoutConfig(0.5)
    c.step = A["step"] + 4
    assert _call(which, plan, drop=ctypes.byref(c)) == INVALID
    out = [n for n in CALLS[which][0] if n in ("out", "grads", "losses")][0]
    c.step = A[out] + 8  # inside an output
    assert _call(which, plan, drop=ctypes.byref(c)) == INVALID


def _dropout(x=A["x"], xs=8, residual=None, rs=0, out=A["out"], os=8, rows=4, cols=8, dtype=0, p=0.5, config=True):
    c = psgd.DropoutConfig(p)
    return psgd.load_library().psgd_dropout(x, xs, residual, rs, out, os, rows, cols, dtype,
                                            ctypes.byref(c) if config else None, None)


@pytest.mark.parametrize("bad,expect", [
    (dict(config=False), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(rows=-1), INVALID), (dict(cols=-1), INVALID),
    (dict(xs=7), INVALID), (dict(os=7), INVALID), (dict(residual=A["dx"], rs=7), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(x=A["x"] + 2), INVALID), (dict(out=A["x"] + 16), INVALID), (dict(out=A["x"], os=9), INVALID),
    (dict(residual=A["out"] + 4, rs=8), INVALID), (dict(p=-1.0), INVALID), (dict(p=math.nan), INVALID),
    (dict(rows=1 << 40, cols=1 << 30), INVALID), (dict(rows=1 << 32, cols=1 << 10, xs=1 << 10, os=1 << 10), INVALID),
    (dict(rows=1 << 20, xs=1 << 42), INVALID), (dict(residual=A["x"], rs=8, out=A["x"], os=9), INVALID),
])
def test_dropout_refuses(bad, expect):
    assert _dropout(**bad) == expect


def test_dropout_of_nothing():
    assert _dropout(rows=0) == psgd.PSGD_OK and _dropout(cols=0, xs=0, os=0) == psgd.PSGD_OK
    assert _dropout(rows=0, x=None, out=None) == psgd.PSGD_OK


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    plan = psgd.psgd_lm_plan_create(SHAPES, 1, 2, 3)
    s = plan.sizes
    x, t = torch.zeros((2, 3, 40)), torch.zeros((2, 3), dtype=torch.int64)
    p, g = torch.zeros(s["worker_stride"]), torch.zeros((2, s["worker_stride"]))
    f, ws = torch.zeros((2, 3)), torch.zeros(s["workspace_bytes"], dtype=torch.uint8)
    assert _status(psgd.psgd_lm_embed, plan, p, t, None, x) == INVALID
    assert _status(psgd.psgd_lm_embed_grad, plan, t, x, None, g, 0, ws) == INVALID
    assert _status(psgd.psgd_lm_loss, plan, x, p, t, None, f, f, f, ws) == INVALID
    assert _status(psgd.psgd_lm_loss_grad, plan, x, p, t, f, None, None, x, g, 0, ws) == INVALID
    assert _status(psgd.psgd_dropout, x[0], None, x[0], psgd.DropoutConfig(0.5)) == INVALID
    assert _status(psgd.DropoutConfig, 0.5, 1, torch.zeros(1, dtype=torch.int64)) == INVALID


CHILD = r"""
import ctypes, sys
from distributed_sgd_gradient_ef_amd import psgd
fails = ctypes.CDLL(sys.argv[1]).new_fails_after
fails.argtypes = [ctypes.c_long]
fails.restype = None
lib = psgd.load_library()
h = ctypes.c_void_p()
layers = lambda *s: (psgd._Layer * len(s))(*[psgd._Layer(r, c) for r, c in s])
good, bad, wide = layers((40, 30), (501, 9)), layers((40, 30), (0, 9)), layers(((1 << 31) - 1, 1))

def sweep(name, call, want):
    for n in range(10000):
        h.value = None
        fails(n)
        try:
            status = call()
        finally:
            fails(-1)
        if status != psgd.PSGD_ERR_NO_MEMORY:
            assert status == want, (name, n, status)
            print(name, n, flush=True)
            return
        assert not h.value, (name, n)
        assert lib.psgd_last_error()
    raise AssertionError(name)

create = lambda l, n: lib.psgd_lm_plan_create(l, n, n - 1, 3, 5, 0, 0, 0, ctypes.byref(h))
sweep("create", lambda: create(good, 2), 0)
plan = h.value
sweep("create: refused layer", lambda: create(bad, 2), 1)
sweep("create: blocks", lambda: create(wide, 1), 1)
sweep("create: NULL", lambda: create(None, 2), 1)
sweep("sizes", lambda: lib.psgd_lm_plan_sizes(None, None), 1)
sweep("set_timing", lambda: lib.psgd_lm_plan_set_timing(None, 1), 1)
sweep("kernel_stats", lambda: lib.psgd_lm_plan_kernel_stats(plan, None, 3, None, 0), 1)
sweep("kernel_stats: none", lambda: lib.psgd_lm_plan_kernel_stats(plan, None, 0, None, 0), 0)
A = [0x10000000 * (i + 1) for i in range(12)]
drop = ctypes.byref(psgd.DropoutConfig(2.0))
sweep("embed", lambda: lib.psgd_lm_embed(plan, A[0], A[0], None, A[1], None), 1)
sweep("embed_grad", lambda: lib.psgd_lm_embed_grad(plan, A[0], A[1], drop, A[2], 0, A[3], None), 1)
sweep("embed_grad: flags", lambda: lib.psgd_lm_embed_grad(plan, A[0], A[1], None, A[2], 8, A[3], None), 2)
sweep("loss", lambda: lib.psgd_lm_loss(plan, A[0], None, A[1], None, *A[2:6], None), 1)
sweep("loss_grad", lambda: lib.psgd_lm_loss_grad(plan, *A[:4], None, None, None, None, 0, A[5], None), 1)
sweep("dropout", lambda: lib.psgd_dropout(A[0], 8, None, 0, A[0] + 16, 8, 4, 8, 0, ctypes.byref(psgd.DropoutConfig(0.5)), None), 1)
sweep("dropout: p", lambda: lib.psgd_dropout(A[0], 8, None, 0, A[1], 8, 4, 8, 0, drop, None), 1)
assert lib.psgd_lm_plan_destroy(plan) == 0
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

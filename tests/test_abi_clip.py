"""The clipping and AdamW part of the C ABI without a GPU: plan validation, the packed
layout, byte accounting, and argument checks that happen before any device call (the
fake addresses below are never dereferenced)."""

import ctypes
import math

import numpy as np
import pytest

from distributed_sgd_gradient_ef_amd import psgd

pytestmark = pytest.mark.usefixtures("built_library")

SHAPES = [(64, 27), (1, 64), (10, 512), (3, 5)]
INVALID, UNSUPPORTED = psgd.PSGD_ERR_INVALID_ARG, psgd.PSGD_ERR_UNSUPPORTED


def _status(fn, *args, **kw):
    with pytest.raises(psgd.PsgdError) as e:
        fn(*args, **kw)
    assert str(e.value)
    return e.value.status


def test_plan_create_rejects_bad_arguments():
    create = psgd.psgd_clip_plan_create
    assert _status(create, SHAPES, 0) == INVALID
    assert _status(create, SHAPES, 65536) == INVALID
    assert _status(create, [], 1) == INVALID
    assert _status(create, [(0, 5)], 1) == INVALID
    assert _status(create, [(5, -1)], 1) == INVALID
    assert _status(create, [(65536, 32768)], 1) == INVALID      # 2^31 elements
    assert _status(create, [(1 << 40, 1 << 40)], 1) == INVALID  # a product past 64 bits
    assert _status(create, SHAPES, 1, 7) == UNSUPPORTED
    assert _status(create, SHAPES, 1, psgd.PSGD_F32, 1) == UNSUPPORTED
    lib = psgd.load_library()
    arr = (psgd._Layer * 1)(psgd._Layer(4, 4))
    h = ctypes.c_void_p()
    assert lib.psgd_clip_plan_create(arr, 1, 1, 0, 0, None) == INVALID
    assert lib.psgd_clip_plan_create(None, 1, 1, 0, 0, ctypes.byref(h)) == INVALID
    assert lib.psgd_clip_plan_sizes(None, None) == INVALID
    assert lib.psgd_clip_plan_destroy(None) == psgd.PSGD_OK


@pytest.mark.parametrize("shapes", [SHAPES, [(1, 1)], [(46341, 46340)], [(33, 35), (1, 10), (130, 1030), (5000, 22)]])
def test_layout_is_that_of_the_compressors(shapes):
    clip = psgd.psgd_clip_plan_create(shapes, 3)
    others = [psgd.psgd_plan_create(shapes, 2, 3),
              psgd.psgd_rtopk_plan_create(shapes, [1] * len(shapes), [1] * len(shapes), 3)]
    if max(min(s) for s in shapes) <= psgd.PSGD_ATOMO_MAX_K:
        others.append(psgd.psgd_atomo_plan_create(shapes, 1.0, 3))
    for other in others:
        assert clip.sizes["worker_stride"] == other.sizes["worker_stride"]
        assert clip.sizes["numel"] == other.sizes["numel"]
        assert [L.offset for L in clip.layers] == [L.offset for L in other.layers]
    assert [(L.rows, L.cols, L.numel) for L in clip.layers] == [(r, c, r * c) for r, c in shapes]


@pytest.mark.parametrize("dtype,gb", [(psgd.PSGD_F32, 4), (psgd.PSGD_BF16, 2)])
def test_byte_accounting(dtype, gb):
    s = psgd.psgd_clip_plan_create(SHAPES, 5, dtype).sizes
    n = sum(r * c for r, c in SHAPES)
    assert (s["n_layers"], s["n_slices"], s["grad_dtype"], s["numel"]) == (4, 5, dtype, n)
    assert s["norm_bytes"] == 5 * n * gb and s["clip_bytes"] == 10 * n * gb and s["adamw_bytes"] == n * (gb + 24)
    assert s["worker_stride"] % 64 == 0 and s["workspace_bytes"] > 0


def test_layer_info_range():
    plan = psgd.psgd_clip_plan_create(SHAPES, 1)
    for li in (-1, 4):
        assert _status(psgd.psgd_clip_plan_layer_info, plan, li) == INVALID


A = {name: 0x10000000 * (i + 1) for i, name in enumerate(
    ["grads", "out", "norms", "tensor_norms", "coefs", "workspace", "params", "exp_avg", "exp_avg_sq", "copy", "step"])}


@pytest.mark.parametrize("bad", [
    dict(grads=None), dict(norms=None), dict(workspace=None), dict(grads=A["grads"] + 4), dict(norms=A["norms"] + 2),
    dict(tensor_norms=A["tensor_norms"] + 1), dict(workspace=A["workspace"] + 8), dict(norms=A["grads"] + 64),
    dict(tensor_norms=A["norms"]), dict(norms=A["workspace"]),
])
def test_norm_rejects_bad_pointers(bad):
    a = {**A, **bad}
    plan = psgd.psgd_clip_plan_create(SHAPES, 4)
    lib = psgd.load_library()
    assert lib.psgd_grad_norm(plan.handle, a["grads"], 0, a["norms"], a["tensor_norms"], a["workspace"], None) == INVALID
    assert lib.psgd_last_error()


def test_norm_rejects_null_plan_and_unknown_kind():
    lib = psgd.load_library()
    plan = psgd.psgd_clip_plan_create(SHAPES, 4)
    assert lib.psgd_grad_norm(None, A["grads"], 0, A["norms"], None, A["workspace"], None) == INVALID
    for kind in (-1, 2):
        assert lib.psgd_grad_norm(plan.handle, A["grads"], kind, A["norms"], None, A["workspace"], None) == UNSUPPORTED
        assert lib.psgd_grad_clip(plan.handle, A["grads"], A["out"], kind, 1.0, A["norms"], A["coefs"], A["workspace"],
                                  None) == UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(grads=None), dict(out=None), dict(norms=None), dict(coefs=None), dict(workspace=None),
    dict(out=A["out"] + 8), dict(coefs=A["coefs"] + 1), dict(out=A["grads"] + 256), dict(coefs=A["norms"]),
    dict(norms=A["out"] + 16), dict(out=A["workspace"]),
])
def test_clip_rejects_bad_pointers(bad):
    a = {**A, **bad}
    plan = psgd.psgd_clip_plan_create(SHAPES, 4)
    assert psgd.load_library().psgd_grad_clip(plan.handle, a["grads"], a["out"], 0, 1.0, a["norms"], a["coefs"],
                                              a["workspace"], None) == INVALID


@pytest.mark.parametrize("max_norm", [0.0, -1.0, math.nan, -math.inf])
def test_clip_rejects_bad_bounds(max_norm):
    plan = psgd.psgd_clip_plan_create(SHAPES, 4)
    lib = psgd.load_library()
    assert lib.psgd_grad_clip(plan.handle, A["grads"], A["out"], 0, max_norm, A["norms"], A["coefs"], A["workspace"],
                              None) == INVALID
    assert lib.psgd_grad_clip(None, A["grads"], A["out"], 0, 1.0, A["norms"], A["coefs"], A["workspace"],
                              None) == INVALID


def _adamw(plan, cfg, **bad):
    a = {**A, **bad}
    return psgd.load_library().psgd_adamw_apply(plan.handle, ctypes.byref(cfg), a["grads"], a["params"], a["exp_avg"],
                                                a["exp_avg_sq"], a["copy"], a["step"], a["norms"], a["workspace"], None)


@pytest.mark.parametrize("bad", [
    dict(grads=None), dict(params=None), dict(exp_avg=None), dict(exp_avg_sq=None), dict(step=None), dict(norms=None),
    dict(workspace=None), dict(step=A["step"] + 4), dict(copy=A["copy"] + 2), dict(params=A["grads"]),
    dict(exp_avg=A["exp_avg_sq"] + 128), dict(copy=A["params"]), dict(norms=A["step"]),
])
def test_adamw_rejects_bad_pointers(bad):
    plan = psgd.psgd_clip_plan_create(SHAPES, 1)
    assert _adamw(plan, psgd.AdamwConfig(max_norm=1.0), **bad) == INVALID


@pytest.mark.parametrize("cfg,expect", [
    (dict(lr=-1.0), INVALID), (dict(lr=math.nan), INVALID), (dict(lr=math.inf), INVALID), (dict(lr=1e39), INVALID),
    (dict(beta1=1.0), INVALID), (dict(beta1=-0.1), INVALID), (dict(beta2=1.0), INVALID), (dict(beta2=math.nan), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=1e-60), INVALID), (dict(eps=math.inf), INVALID),
    (dict(weight_decay=-0.1), INVALID), (dict(weight_decay=math.inf), INVALID), (dict(max_norm=-1.0), INVALID),
    (dict(max_norm=math.nan), INVALID), (dict(norm_kind=9), UNSUPPORTED), (dict(flags=4), UNSUPPORTED),
])
def test_adamw_rejects_bad_configs(cfg, expect):
    plan = psgd.psgd_clip_plan_create(SHAPES, 1)
    assert _adamw(plan, psgd.AdamwConfig(**{"max_norm": 1.0, **cfg})) == expect


def test_adamw_rejects_contradictions():
    plan = psgd.psgd_clip_plan_create(SHAPES, 1)
    assert _adamw(psgd.psgd_clip_plan_create(SHAPES, 2), psgd.AdamwConfig(max_norm=1.0)) == INVALID
    assert _adamw(plan, psgd.AdamwConfig(max_norm=0.0)) == INVALID  # a norm output without a norm
    assert _adamw(plan, psgd.AdamwConfig(max_norm=0.0, flags=psgd.PSGD_ADAMW_SKIP_NONFINITE), norms=None) == INVALID
    lib = psgd.load_library()
    assert lib.psgd_adamw_apply(plan.handle, None, *[0x1000] * 9) == INVALID


def test_pack_roundtrip():
    plan = psgd.psgd_clip_plan_create(SHAPES, 3)
    rng = np.random.default_rng(1)
    per = [rng.standard_normal((3,) + s).astype(np.float32) for s in SHAPES]
    flat = psgd.pack(plan, per)
    assert flat.shape == (3, plan.sizes["worker_stride"])
    for li, a in enumerate(per):
        assert np.array_equal(psgd.unpack(plan, flat, li), a)
    one = psgd.pack(plan, [a[0] for a in per], workers=0)
    assert np.array_equal(one, flat[0])


def test_timing_calls_without_gpu():
    plan = psgd.psgd_clip_plan_create(SHAPES, 1)
    psgd.psgd_clip_plan_set_timing(plan, True)
    assert psgd.psgd_clip_plan_kernel_stats(plan) == {}
    psgd.psgd_clip_plan_set_timing(plan, False)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    plan = psgd.psgd_clip_plan_create(SHAPES, 2)
    n = plan.sizes["worker_stride"]
    g, f = torch.zeros((2, n)), torch.zeros(2)
    ws = torch.zeros(plan.sizes["workspace_bytes"], dtype=torch.uint8)
    assert _status(psgd.psgd_grad_norm, plan, g, 0, f, None, ws) == INVALID
    assert _status(psgd.psgd_grad_clip, plan, g, g, 0, 1.0, f, f, ws) == INVALID

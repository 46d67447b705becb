"""Gradient norms, clipping and AdamW on the GPU against the float64 oracle
(oracle/clip_adamw.py).

Tolerances, with u = 2^-24 (half a float32 step):
* a norm is a float64 sum rounded once: u relative.  Up to 2^31 float64 additions of
  positive terms add at most 2^-22 u each in relative size only if summed one after the
  other; the tests' largest chains are thousands long, so 1.001 u covers them;
* a coefficient is one float64 division rounded once: 1.001 u;
* out is the single float32 product of the coefficient the GPU reports and g, rounded to
  the gradient type: compared bit for bit with the same two roundings in numpy;
* g' = c U: 2 u.  m: beta1, the products, the sum and g' add at most 5 u of
  |beta1 m| + |(1 - beta1) g'|.  v: g'^2 (4 u + u), 1 - beta2, product, sum: 8 u of v.
  The step's fraction m / (sqrt(v) / sqrt(bc2) + eps) * rate: sqrt(v) carries 4 u of v's
  and 2 u for a square root within one ulp, its factor and product 2 u, eps and the sum
  2 u; the division 5 u (2.5 ulp), rate and its product 2 u: 17 u, plus m's error.
  x - d x: 2 u of |x| (d << 1), the final difference u of |x| + |fraction|;
* the bfloat16 copy is the GPU's own new params rounded to nearest even: bit for bit.
"""

import math

import numpy as np
import pytest

from distributed_sgd_gradient_ef_amd import psgd
from oracle import clip_adamw as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
U = 2.0 ** -24
KINDS = {"l2": psgd.PSGD_NORM_L2, "max": psgd.PSGD_NORM_MAX}
DTYPES = {"f32": (psgd.PSGD_F32, torch.float32), "bf16": (psgd.PSGD_BF16, torch.bfloat16)}

SHAPE_SETS = {
    "one": [(1, 1)],
    "ends": [(1, 1), (1, 3), (1, 4), (1, 5), (1, 63), (1, 64), (1, 65), (7, 129), (1, 1023), (1, 1025)],
    "tiles": [(1, 4095), (64, 64), (1, 4097), (1, 8191), (8, 1025), (1, 16383), (128, 128), (5, 3277), (257, 129)],
    "mixed": [(64, 27), (1, 64), (3, 5), (10, 512), (1, 70001), (333, 257), (1, 2), (65537, 1)],
    "many": [(1 + i % 5, 1 + (i * 37) % 211) for i in range(300)],
    "large": [(1500, 1700), (1, 31), (2049, 1023)],
}


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    return psgd.load_library()


def _grads(plan, dtype, seed, scales=None):
    """Packed random gradients with NaN in the padding (which must not matter)."""
    rng = np.random.default_rng(seed)
    W, ld = plan.sizes["n_slices"], plan.sizes["worker_stride"]
    a = np.full((W, ld), np.nan, dtype=np.float32)
    for L in plan.layers:
        a[:, L.offset:L.offset + L.numel] = rng.standard_normal((W, L.numel)) * math.exp(rng.normal())
    if scales is not None:
        a *= np.asarray(scales, dtype=np.float32)[:, None]
    return torch.from_numpy(a).to(dtype).to(DEV)


def _values(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tensors(plan, row):
    return [row[L.offset:L.offset + L.numel] for L in plan.layers]


def _workspace(plan):
    return torch.full((plan.sizes["workspace_bytes"],), 0xFF, dtype=torch.uint8, device=DEV)


def _padding(plan):
    keep = np.ones(plan.sizes["worker_stride"], dtype=bool)
    for L in plan.layers:
        keep[L.offset:L.offset + L.numel] = False
    return keep


def _near(got, want, rel):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
    assert np.all(np.abs(got[fin] - want[fin]) <= rel * np.abs(want[fin])), (got, want)


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


# ------------------------------------------------------------------ norms
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", SHAPE_SETS)
def test_norms(name, kind, dtype):
    code, td = DTYPES[dtype]
    W = 3
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], W, code)
    g = _grads(plan, td, seed=1)
    norms = torch.full((W,), -1.0, device=DEV)
    per = torch.full((W, len(plan.layers)), -1.0, device=DEV)
    psgd.psgd_grad_norm(plan, g, KINDS[kind], norms, per, _workspace(plan))
    alone = torch.full((W,), -1.0, device=DEV)
    psgd.psgd_grad_norm(plan, g, KINDS[kind], alone, None, _workspace(plan))
    torch.cuda.synchronize()
    assert torch.equal(norms, alone)
    rows = _values(g)
    _near(norms.cpu(), [O.norm_of_tensors(_tensors(plan, r), kind) for r in rows], 1.001 * U)
    _near(per.cpu(), [[O.norm(t, kind) for t in _tensors(plan, r)] for r in rows], 1.001 * U)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e25, 1e37])
@pytest.mark.parametrize("kind", KINDS)
def test_norms_at_the_ends_of_the_range(kind, scale):
    """Squares outside float32's range do not matter."""
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["ends"], 2)
    g = (_grads(plan, torch.float32, seed=2).clamp(-3, 3) * scale)
    norms = torch.zeros(2, device=DEV)
    psgd.psgd_grad_norm(plan, g, KINDS[kind], norms, None, _workspace(plan))
    want = np.array([O.norm_of_tensors(_tensors(plan, r), kind) for r in _values(g)])
    got = norms.cpu().numpy()
    # at 1e37 the L2 norms are 6.7e38 and 6.6e38: past float32's largest number (3.4e38) by
    # more than half a step, so they round to infinity
    past = want > 2.0 ** 128
    assert np.all(got[past] == np.inf)
    # results near the smallest normal number may be a subnormal's half step off
    assert np.all(np.abs(got - want)[~past] <= (1.001 * U * want + 2.0 ** -150)[~past])


@pytest.mark.parametrize("kind", KINDS)
def test_norms_of_zeros_and_non_finite_entries(kind):
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["mixed"], 5)
    g = _grads(plan, torch.float32, seed=3)
    at = plan.layers[5].offset + 77_000
    g[0] = 0.0
    g[1, at] = math.inf
    g[2, at] = math.nan
    g[3, plan.layers[6].offset] = -math.inf
    g[3, plan.layers[0].offset] = math.nan
    norms, per = torch.zeros(5, device=DEV), torch.zeros((5, len(plan.layers)), device=DEV)
    psgd.psgd_grad_norm(plan, g, KINDS[kind], norms, per, _workspace(plan))
    rows = _values(g)
    _near(norms.cpu(), [O.norm_of_tensors(_tensors(plan, r), kind) for r in rows], 1.001 * U)
    _near(per.cpu(), [[O.norm(t, kind) for t in _tensors(plan, r)] for r in rows], 1.001 * U)


# ------------------------------------------------------------------ clipping
def _check_clip(plan, g, out, norms, coefs, kind, max_norm):
    rows = _values(g)
    want = [O.norm_of_tensors(_tensors(plan, r), kind) for r in rows]
    _near(norms.cpu(), want, 1.001 * U)
    bound = float(np.float32(max_norm))
    _near(coefs.cpu(), [O.coefficient(n, bound) for n in want], 1.001 * U)
    # the single product, in the same two roundings
    prod = torch.from_numpy(g.float().cpu().numpy() * coefs.cpu().numpy()[:, None]).to(g.dtype)
    inside = torch.from_numpy(~_padding(plan))
    a, b = out.cpu()[:, inside], prod[:, inside]
    nan = torch.isnan(b.float())
    assert torch.equal(torch.isnan(a.float()), nan)
    assert torch.equal(_bits(a)[~nan], _bits(b)[~nan])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", SHAPE_SETS)
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(name, kind, dtype, in_place):
    code, td = DTYPES[dtype]
    W = 5
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], W, code)
    g = _grads(plan, td, seed=4, scales=[1e-3, 1.0, 300.0, 0.0, 0.05])
    given = g.clone()
    out = g if in_place else torch.full_like(g, 7.0)
    norms, coefs = torch.zeros(W, device=DEV), torch.zeros(W, device=DEV)
    max_norm = 0.5
    psgd.psgd_grad_clip(plan, g, out, KINDS[kind], max_norm, norms, coefs, _workspace(plan))
    torch.cuda.synchronize()
    _check_clip(plan, given, out, norms, coefs, kind, max_norm)
    assert (coefs[3] == 1) and (name == "one" or coefs[2] < 1)
    pad = torch.from_numpy(_padding(plan)).to(DEV)
    if in_place:
        assert torch.isnan(out[:, pad].float()).all()
    else:
        assert torch.equal(_bits(g), _bits(given)) and (out[:, pad] == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_clip_of_non_finite_gradients(kind, in_place):
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["mixed"], 4)
    g = _grads(plan, torch.float32, seed=5)
    g[1, plan.layers[4].offset + 9] = -math.inf
    g[2, plan.layers[7].offset + 65_536] = math.nan
    given = g.clone()
    out = g if in_place else torch.zeros_like(g)
    norms, coefs = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    psgd.psgd_grad_clip(plan, g, out, KINDS[kind], 0.1, norms, coefs, _workspace(plan))
    _check_clip(plan, given, out, norms, coefs, kind, 0.1)
    assert coefs[1] == 0 and torch.isnan(coefs[2]) and torch.isfinite(coefs[0]) and torch.isfinite(coefs[3])


def test_clip_with_an_infinite_bound_copies():
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["mixed"], 2)
    g = _grads(plan, torch.float32, seed=6)
    g[1, 3] = math.inf
    out, norms, coefs = torch.zeros_like(g), torch.zeros(2, device=DEV), torch.zeros(2, device=DEV)
    psgd.psgd_grad_clip(plan, g, out, psgd.PSGD_NORM_L2, math.inf, norms, coefs, _workspace(plan))
    inside = torch.from_numpy(~_padding(plan)).to(DEV)
    assert torch.equal(out[:, inside], g[:, inside]) and (coefs == 1).all() and norms[1] == math.inf


def test_clipped_norm_is_the_bound():
    """The norm of what comes out is the bound up to rounding: every entry is within 2 u."""
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["large"], 2)
    g = _grads(plan, torch.float32, seed=7)
    norms, coefs = torch.zeros(2, device=DEV), torch.zeros(2, device=DEV)
    ws = _workspace(plan)
    psgd.psgd_grad_clip(plan, g, g, psgd.PSGD_NORM_L2, 0.75, norms, coefs, ws)
    psgd.psgd_grad_norm(plan, g, psgd.PSGD_NORM_L2, norms, None, ws)
    _near(norms.cpu(), [0.75, 0.75], 3.01 * U)


# ------------------------------------------------------------------ AdamW
def _adamw_state(plan, seed, step):
    rng = np.random.default_rng(seed)
    n = plan.sizes["worker_stride"]
    x = rng.standard_normal(n).astype(np.float32)
    m = (0.1 * rng.standard_normal(n) * (step > 0)).astype(np.float32)
    v = ((rng.random(n) ** 4 + 1e-12) * (step > 0)).astype(np.float32)
    pad = _padding(plan)
    for a in (x, m, v):
        a[pad] = np.nan
    dev = [torch.from_numpy(a).to(DEV) for a in (x, m, v)]
    return dev + [torch.full((1,), step, dtype=torch.int64, device=DEV)]


def _check_adamw(plan, cfg, g, before, after, t, kind, copy=None):
    inside = ~_padding(plan)
    gv = _values(g)
    c = 1.0
    if cfg.max_norm > 0:
        c = O.coefficient(O.norm_of_tensors(_tensors(plan, gv), kind), cfg.max_norm)
    gv = (gv * c)[inside]
    x0, m0, v0 = (_values(a)[inside] for a in before)
    x1, m1, v1 = (_values(a)[inside] for a in after)
    decay = np.full(plan.sizes["worker_stride"], cfg.weight_decay)
    if cfg.flags & psgd.PSGD_ADAMW_DECAY_MATRICES_ONLY:
        for L in plan.layers:
            if L.rows == 1 or L.cols == 1:
                decay[L.offset:L.offset + L.numel] = 0.0
    r = O.adamw(x0, m0, v0, gv, t, cfg.lr, cfg.beta1, cfg.beta2, cfg.eps, decay[inside])
    tiny = 2.0 ** -148  # subnormal results
    m_err = 5 * U * (np.abs(cfg.beta1 * m0) + np.abs((1 - cfg.beta1) * gv)) * 1.01 + tiny
    assert np.all(np.abs(m1 - r.m) <= m_err)
    assert np.all(np.abs(v1 - r.v) <= 8 * U * 1.01 * r.v + tiny)
    rate = cfg.lr / (1 - cfg.beta1 ** t) / (np.sqrt(r.v / (1 - cfg.beta2 ** t)) + cfg.eps)
    frac = np.abs(rate * r.m)
    x_err = (3 * U * np.abs(x0) + 18 * U * frac + rate * m_err) * 1.01 + tiny
    assert np.all(np.abs(x1 - r.params) <= x_err)
    pad = torch.from_numpy(~inside).to(DEV)
    assert all(torch.isnan(a[pad]).all() for a in after)
    if copy is not None:
        ins = torch.from_numpy(inside).to(DEV)
        assert torch.equal(_bits(copy[ins]), _bits(after[0][ins].to(torch.bfloat16)))
        assert (copy[pad] == 5.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", SHAPE_SETS)
@pytest.mark.parametrize("max_norm,kind", [(0.0, "l2"), (0.3, "l2"), (0.01, "max"), (math.inf, "l2")])
def test_adamw(name, dtype, max_norm, kind):
    code, td = DTYPES[dtype]
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], 1, code)
    ws = _workspace(plan)
    for step, flags, want_copy in ((0, 0, True), (37, psgd.PSGD_ADAMW_DECAY_MATRICES_ONLY, False), (10 ** 7, 0, False)):
        g = _grads(plan, td, seed=8 + step % 5)[0]
        cfg = psgd.AdamwConfig(lr=3e-3, beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.1, max_norm=max_norm,
                               norm_kind=KINDS[kind], flags=flags)
        x, m, v, t = _adamw_state(plan, seed=9, step=step)
        before = [a.clone() for a in (x, m, v)]
        copy = torch.full_like(x, 5.0, dtype=torch.bfloat16) if want_copy else None
        norm = torch.zeros(1, device=DEV) if max_norm > 0 else None
        psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, copy, t, norm, ws)
        torch.cuda.synchronize()
        assert int(t) == step + 1
        _check_adamw(plan, cfg, g, before, (x, m, v), step + 1, kind, copy)
        if norm is not None:
            _near(norm.cpu(), [O.norm_of_tensors(_tensors(plan, _values(g)), kind)], 1.001 * U)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", ["ends", "mixed", "large"])
def test_adamw_skips_a_non_finite_update(name, kind):
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], 1)
    ws = _workspace(plan)
    cfg = psgd.AdamwConfig(max_norm=1.0, norm_kind=KINDS[kind], flags=psgd.PSGD_ADAMW_SKIP_NONFINITE)
    x, m, v, t = _adamw_state(plan, seed=10, step=3)
    norm = torch.zeros(1, device=DEV)
    copy = torch.full_like(x, 5.0, dtype=torch.bfloat16)
    at = max(plan.layers, key=lambda L: L.numel)
    for bad in (math.nan, math.inf, -math.inf):
        g = _grads(plan, torch.float32, seed=11)[0]
        g[at.offset + at.numel - 1] = bad
        before = [a.clone() for a in (x, m, v, copy)]
        psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, copy, t, norm, ws)
        assert int(t) == 3 and not torch.isfinite(norm).any()
        assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(before, (x, m, v, copy)))
    g = _grads(plan, torch.float32, seed=12)[0]
    before = [a.clone() for a in (x, m, v)]
    psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, copy, t, norm, ws)
    assert int(t) == 4
    _check_adamw(plan, cfg, g, before, (x, m, v), 4, kind, copy)


@pytest.mark.parametrize("name", ["ends", "mixed", "large"])
@pytest.mark.parametrize("beta1,beta2,weight_decay", [(0.0, 0.0, 0.0), (0.0, 0.99, 0.1), (0.95, 0.0, 0.1)])
def test_adamw_at_the_ends_of_its_ranges(name, beta1, beta2, weight_decay):
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], 1)
    g = _grads(plan, torch.float32, seed=60)[0]
    cfg = psgd.AdamwConfig(lr=1e-2, beta1=beta1, beta2=beta2, weight_decay=weight_decay, max_norm=0.5)
    x, m, v, t = _adamw_state(plan, seed=61, step=1)
    before = [a.clone() for a in (x, m, v)]
    psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, torch.zeros(1, device=DEV), _workspace(plan))
    assert int(t) == 2
    _check_adamw(plan, cfg, g, before, (x, m, v), 2, "l2")
    # a rate of zero moves the moments and the count, not the weights
    cfg = psgd.AdamwConfig(lr=0.0, beta1=beta1, beta2=beta2, weight_decay=weight_decay)
    before = x.clone()
    psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, None, _workspace(plan))
    assert int(t) == 3 and torch.equal(_bits(x), _bits(before))


@pytest.mark.parametrize("name", ["ends", "mixed", "large"])
def test_outputs_need_only_their_types_alignment(name):
    W = 3
    plan, one = psgd.psgd_clip_plan_create(SHAPE_SETS[name], W), psgd.psgd_clip_plan_create(SHAPE_SETS[name], 1)
    n = len(plan.layers)
    g = _grads(plan, torch.float32, seed=62)
    norms, coefs = torch.full((W + 2,), 9.0, device=DEV), torch.full((W + 2,), 9.0, device=DEV)
    per = torch.full((W * n + 2,), 9.0, device=DEV)
    psgd.psgd_grad_norm(plan, g, psgd.PSGD_NORM_L2, norms[1:W + 1], per[1:W * n + 1], _workspace(plan))
    rows = _values(g)
    _near(norms[1:-1].cpu(), [O.norm_of_tensors(_tensors(plan, r), "l2") for r in rows], 1.001 * U)
    _near(per[1:-1].cpu(), [O.norm(t, "l2") for r in rows for t in _tensors(plan, r)], 1.001 * U)
    out = torch.zeros_like(g)
    psgd.psgd_grad_clip(plan, g, out, psgd.PSGD_NORM_L2, 0.5, norms[1:W + 1], coefs[1:W + 1], _workspace(plan))
    _check_clip(plan, g, out, norms[1:-1], coefs[1:-1], "l2", 0.5)
    x, m, v, _ = _adamw_state(one, seed=63, step=0)
    steps = torch.tensor([7, 7, 7], dtype=torch.int64, device=DEV)
    psgd.psgd_adamw_apply(one, psgd.AdamwConfig(max_norm=1.0), g[0], x, m, v, None, steps[1:2], norms[W + 1:],
                          _workspace(one))
    assert steps.tolist() == [7, 8, 7]
    assert all(float(a[0]) == 9.0 for a in (norms, coefs, per)) and float(coefs[-1]) == float(per[-1]) == 9.0


def test_adamw_of_a_non_finite_update_spreads_it_without_the_flag():
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["ends"], 1)
    x, m, v, t = _adamw_state(plan, seed=13, step=3)
    g = _grads(plan, torch.float32, seed=14)[0]
    g[0] = math.nan
    psgd.psgd_adamw_apply(plan, psgd.AdamwConfig(max_norm=1.0), g, x, m, v, None, t, torch.zeros(1, device=DEV),
                          _workspace(plan))
    assert int(t) == 4 and torch.isnan(x).all() and torch.isnan(m).all() and torch.isnan(v).all()


# ------------------------------------------------------------------ streams, graphs, repeats
def _one_of_each(plan, g, ws):
    """Buffers of a clip of 3 slices, and the call."""
    norms, coefs, out = torch.zeros(3, device=DEV), torch.zeros(3, device=DEV), torch.zeros_like(g)
    per = torch.zeros((3, len(plan.layers)), device=DEV)

    def call(stream=None):
        psgd.psgd_grad_clip(plan, g, out, psgd.PSGD_NORM_L2, 0.5, norms, coefs, ws, stream)
        psgd.psgd_grad_norm(plan, out, psgd.PSGD_NORM_MAX, norms, per, ws, stream)

    return call, (norms, coefs, out, per)


@pytest.mark.parametrize("name", ["mixed", "large"])
def test_equal_calls_give_equal_bits(name):
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], 3)
    g = _grads(plan, torch.float32, seed=15)
    a, outs = _one_of_each(plan, g, _workspace(plan))
    b, again = _one_of_each(plan, g, torch.zeros_like(_workspace(plan)))
    a()
    b()
    inside = torch.from_numpy(~_padding(plan)).to(DEV)
    for x, y in zip(outs, again):
        x, y = (x[:, inside], y[:, inside]) if x.shape[-1] == inside.numel() else (x, y)
        assert torch.equal(x, y)


def test_two_streams_at_once():
    """Two plans with workspaces of their own, on streams of their own."""
    sets = []
    for seed in (16, 17):
        plan = psgd.psgd_clip_plan_create(SHAPE_SETS["large"], 3)
        g = torch.nan_to_num(_grads(plan, torch.float32, seed=seed))
        call, outs = _one_of_each(plan, g, _workspace(plan))
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        sets.append((call, outs, want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, _, _, st in sets:
            call(st)
    torch.cuda.synchronize()
    for _, outs, want, _ in sets:
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_capture_needs_an_eager_call_first():
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["ends"], 3)
    g = torch.nan_to_num(_grads(plan, torch.float32, seed=18))
    call, _ = _one_of_each(plan, g, _workspace(plan))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(psgd.PsgdError) as e:
            call()
        g.add_(0.0)
    assert e.value.status == psgd.PSGD_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["ends", "mixed", "large"])
def test_a_captured_training_tail(name):
    """Clip every worker, average, AdamW with clipping, captured once and replayed with new
    gradients; every replay equals the eager run bit for bit."""
    W = 3
    shapes = SHAPE_SETS[name]
    cfg = psgd.AdamwConfig(lr=1e-2, max_norm=0.2, flags=psgd.PSGD_ADAMW_SKIP_NONFINITE)

    def make():
        workers, one = psgd.psgd_clip_plan_create(shapes, W), psgd.psgd_clip_plan_create(shapes, 1)
        n = one.sizes["worker_stride"]
        x, m, v, t = _adamw_state(one, seed=19, step=0)
        return dict(workers=workers, one=one, g=torch.zeros((W, n), device=DEV), u=torch.zeros(n, device=DEV),
                    x=x, m=m, v=v, t=t, wws=_workspace(workers), ows=_workspace(one),
                    norms=torch.zeros(W, device=DEV), coefs=torch.zeros(W, device=DEV), norm=torch.zeros(1, device=DEV),
                    copy=torch.zeros(n, dtype=torch.bfloat16, device=DEV))

    def step(s):
        psgd.psgd_grad_clip(s["workers"], s["g"], s["g"], psgd.PSGD_NORM_L2, 0.5, s["norms"], s["coefs"], s["wws"])
        torch.add(s["g"][0], s["g"][1], out=s["u"])
        psgd.psgd_adamw_apply(s["one"], cfg, s["u"], s["x"], s["m"], s["v"], s["copy"], s["t"], s["norm"], s["ows"])

    a, b = make(), make()

    def load(seed, bad=False):
        g = torch.nan_to_num(_grads(a["workers"], torch.float32, seed=seed))
        if bad:
            g[0, 0] = math.nan
        a["g"].copy_(g)
        b["g"].copy_(g)

    load(20)
    step(a)
    step(b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    scratch = torch.zeros(1 << 20, device=DEV)
    steps = 1
    for i in range(5):
        load(21 + i, bad=i == 2)
        torch.cuda.synchronize()
        graph.replay()
        scratch.add_(1.0)
        torch.cuda.synchronize()
        step(b)
        torch.cuda.synchronize()
        steps += i != 2
        assert int(a["t"]) == steps == int(b["t"])
        inside = torch.from_numpy(~_padding(a["one"])).to(DEV)
        for k in ("x", "m", "v", "copy"):
            assert torch.equal(_bits(a[k][inside]), _bits(b[k][inside])), (i, k)
        for k in ("norms", "coefs", "norm"):
            assert torch.equal(_bits(a[k]), _bits(b[k])), (i, k)


def test_timing_names():
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["large"], 1)
    g = torch.nan_to_num(_grads(plan, torch.float32, seed=22))
    ws = _workspace(plan)
    norms, coefs = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    psgd.psgd_clip_plan_set_timing(plan, True)
    x, m, v, t = _adamw_state(plan, seed=23, step=0)
    psgd.psgd_grad_clip(plan, g, g, psgd.PSGD_NORM_L2, 1.0, norms, coefs, ws)
    psgd.psgd_adamw_apply(plan, psgd.AdamwConfig(max_norm=1.0), g[0], x, m, v, None, t, norms, ws)
    stats = psgd.psgd_clip_plan_kernel_stats(plan, reset=True)
    assert stats and set(stats) <= {"cl_norm", "cl_final", "cl_scale", "cl_adamw", "cl_small", "cl_small_adamw"}
    assert all(n > 0 and ms > 0 for n, ms in stats.values())
    assert psgd.psgd_clip_plan_kernel_stats(plan) == {}


def test_binding_refuses_wrong_tensors():
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["ends"], 2)
    n = plan.sizes["worker_stride"]
    g, norms, ws = torch.zeros((2, n), device=DEV), torch.zeros(2, device=DEV), _workspace(plan)
    bad = [dict(g=g.to(torch.bfloat16)), dict(g=g[:1]), dict(g=torch.zeros((2, 2 * n), device=DEV)[:, ::2]),
           dict(norms=norms.double()), dict(norms=norms[:1]), dict(norms=norms.cpu()), dict(ws=ws[:8])]
    for b in bad:
        a = dict(g=g, norms=norms, ws=ws, **{}) | b
        with pytest.raises(psgd.PsgdError) as e:
            psgd.psgd_grad_norm(plan, a["g"], 0, a["norms"], None, a["ws"])
        assert e.value.status == psgd.PSGD_ERR_INVALID_ARG


# ------------------------------------------------------------------ long buffers
def test_slices_beyond_32_bit_offsets():
    """Five slices of 2^30 elements: element offsets past 2^32."""
    plan = psgd.psgd_clip_plan_create([(32768, 32768)], 5, psgd.PSGD_BF16)
    g = torch.full((5, 1 << 30), 2.0 ** -10, dtype=torch.bfloat16, device=DEV)
    g[4, 12345] = 64.0
    norms, coefs, ws = torch.zeros(5, device=DEV), torch.zeros(5, device=DEV), _workspace(plan)
    psgd.psgd_grad_clip(plan, g, g, psgd.PSGD_NORM_L2, 16.0, norms, coefs, ws)
    torch.cuda.synchronize()
    # 2^30 entries of 2^-20 sum to 2^10; 64^2 replaces one of them
    want = [32.0] * 4 + [math.sqrt(1024.0 - 2.0 ** -20 + 4096.0)]
    _near(norms.cpu(), want, 1.001 * U)
    _near(coefs.cpu(), [16.0 / n for n in want], 1.001 * U)
    assert all(bool((g[w] == 2.0 ** -11).all()) for w in range(4))
    c = float(coefs[4])
    assert float(g[4, 12345]) == float(torch.tensor(64.0 * c).bfloat16())
    assert float(g[4, -1]) == float(torch.tensor(2.0 ** -10 * c).bfloat16()) == float(g[4, 0])


def test_adamw_beyond_31_bit_offsets():
    shapes = [(32768, 32768), (32768, 32768), (9, 11)]
    plan = psgd.psgd_clip_plan_create(shapes, 1)
    n = plan.sizes["worker_stride"]
    L = plan.layers[2]
    assert L.offset == 1 << 31
    g = torch.zeros(n, device=DEV)
    g[L.offset:L.offset + 99] = torch.linspace(-1, 1, 99, device=DEV)
    x, m, v = torch.ones(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    t, norm = torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, device=DEV)
    cfg = psgd.AdamwConfig(lr=0.25, weight_decay=0.5, eps=1e-6, max_norm=0.5)
    psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, norm, _workspace(plan))
    torch.cuda.synchronize()
    gv = _values(g[L.offset:L.offset + 99])
    n2 = O.norm(gv, "l2")
    _near(norm.cpu(), [n2], 1.001 * U)
    r = O.adamw(np.ones(99), np.zeros(99), np.zeros(99), gv * O.coefficient(n2, 0.5), 1, 0.25, 0.9, 0.999, 1e-6, 0.5)
    got = _values(x[L.offset:L.offset + 99])
    assert np.all(np.abs(got - r.params) <= 40 * U)  # |x|, |fraction| <= 1: 3 u + 18 u + 5 u, doubled for rate's sum
    # where the gradient is zero only the decay acts: 1 - 0.125, exact
    assert bool((x[:1 << 31] == 0.875).all()) and bool((m[:1 << 31] == 0).all())


# ------------------------------------------------------------------ together with the compressors
def test_clip_compress_and_adamw_together():
    """Three training steps: every worker's gradient clipped, compressed with error
    feedback by PowerSGD, and the update applied by AdamW with clipping.  The compressor's
    own parity is tested elsewhere: here its input is what the clipping left, its output is
    what AdamW took."""
    from oracle import powersgd_ef as PO

    shapes = [(64, 27), (1, 64), (130, 96), (10, 512), (1, 10)]
    W, r = 4, 2
    comp = psgd.psgd_plan_create(shapes, r, W)
    workers, one = psgd.psgd_clip_plan_create(shapes, W), psgd.psgd_clip_plan_create(shapes, 1)
    s = comp.sizes
    n = s["worker_stride"]
    q = torch.from_numpy(np.random.default_rng(31).standard_normal(s["q_elems"]).astype(np.float32)).to(DEV)
    p, errors = torch.zeros(s["p_elems"], device=DEV), torch.zeros((W, n), device=DEV)
    u, cws = torch.zeros(n, device=DEV), torch.zeros(s["workspace_bytes"], dtype=torch.uint8, device=DEV)
    x, m, v, t = _adamw_state(one, seed=32, step=0)
    norms, coefs, norm = torch.zeros(W, device=DEV), torch.zeros(W, device=DEV), torch.zeros(1, device=DEV)
    cfg = psgd.AdamwConfig(lr=1e-2, max_norm=0.05, flags=psgd.PSGD_ADAMW_DECAY_MATRICES_ONLY)
    for step in range(3):
        g = torch.nan_to_num(_grads(workers, torch.float32, seed=33 + step))
        given, e0, q0 = g.clone(), errors.clone(), q.clone()
        psgd.psgd_grad_clip(workers, g, g, psgd.PSGD_NORM_L2, 0.5, norms, coefs, _workspace(workers))
        psgd.psgd_compress_step(comp, g, errors, q, p, u, cws)
        before = [a.clone() for a in (x, m, v)]
        psgd.psgd_adamw_apply(one, cfg, u, x, m, v, None, t, norm, _workspace(one))
        torch.cuda.synchronize()
        _check_clip(workers, given, g, norms, coefs, "l2", 0.5)
        for li, L in enumerate(comp.layers):
            cut = slice(L.offset, L.offset + L.rows * L.cols)
            gw = g[:, cut].cpu().numpy().reshape(W, L.rows, L.cols)
            if L.compressed:
                ew = e0[:, cut].cpu().numpy().reshape(W, L.rows, L.cols)
                qw = q0[L.q_offset:L.q_offset + L.cols * r].cpu().numpy().reshape(L.cols, r)
                ref = PO.compress_matrix(gw, ew, qw).update
            else:
                ref = PO.average_tensor(gw)
            got = u[cut].cpu().numpy().reshape(L.rows, L.cols)
            assert np.linalg.norm(got - ref) <= 1e-4 * np.linalg.norm(ref)
        assert int(t) == step + 1
        _check_adamw(one, cfg, u, before, (x, m, v), step + 1, "l2")


# ------------------------------------------------------------------ more calls the header allows
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ["ends", "large"])
def test_clip_into_subnormal_numbers(name, dtype):
    """Products below the smallest normal number keep their subnormal bits."""
    code, td = DTYPES[dtype]
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS[name], 2, code)
    g = _grads(plan, td, seed=40, scales=[1.0, 1e-35])
    given, out = g.clone(), torch.full_like(g, 7.0)
    norms, coefs = torch.zeros(2, device=DEV), torch.zeros(2, device=DEV)
    psgd.psgd_grad_clip(plan, g, out, psgd.PSGD_NORM_MAX, 1e-39, norms, coefs, _workspace(plan))
    bound = float(np.float32(1e-39))  # a subnormal itself: half a step of it is 2^-150
    want = [O.norm_of_tensors(_tensors(plan, r), "max") for r in _values(given)]
    assert np.all(np.abs(_values(coefs) - [bound / n for n in want]) <= 2.0 ** -150 + 1.001 * U * bound / np.array(want))
    inside = torch.from_numpy(~_padding(plan))
    prod = torch.from_numpy(given.float().cpu().numpy() * coefs.cpu().numpy()[:, None]).to(td)
    assert torch.equal(_bits(out.cpu()[:, inside]), _bits(prod[:, inside]))
    assert bool((out.float().abs().nan_to_num(0.0)[:, inside.to(DEV)] > 0).any())


@pytest.mark.parametrize("total", [8191, 8192, 8193, 16384, 16385, 32768, 32769, 65536, 2097152, 2097153])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sizes_around_the_variants_borders(total, dtype):
    """Element counts at which another kernel takes over; one call of each operator."""
    code, td = DTYPES[dtype]
    shapes = [(1, total - 640), (16, 40)]
    plan, one = psgd.psgd_clip_plan_create(shapes, 2, code), psgd.psgd_clip_plan_create(shapes, 1, code)
    g = _grads(plan, td, seed=41)
    ws = _workspace(plan)
    norms, coefs, per = torch.zeros(2, device=DEV), torch.zeros(2, device=DEV), torch.zeros((2, 2), device=DEV)
    psgd.psgd_grad_norm(plan, g, psgd.PSGD_NORM_L2, norms, per, ws)
    first = norms.clone()
    out = torch.full_like(g, 7.0)
    psgd.psgd_grad_clip(plan, g, out, psgd.PSGD_NORM_L2, 0.5, norms, coefs, ws)
    rows = _values(g)
    _near(first.cpu(), [O.norm_of_tensors(_tensors(plan, r), "l2") for r in rows], 1.001 * U)
    _near(per.cpu(), [[O.norm(t, "l2") for t in _tensors(plan, r)] for r in rows], 1.001 * U)
    _check_clip(plan, g, out, norms, coefs, "l2", 0.5)
    for max_norm in (0.0, 0.25):
        cfg = psgd.AdamwConfig(lr=1e-2, max_norm=max_norm, flags=psgd.PSGD_ADAMW_DECAY_MATRICES_ONLY)
        x, m, v, t = _adamw_state(one, seed=42, step=9)
        before = [a.clone() for a in (x, m, v)]
        norm = torch.zeros(1, device=DEV) if max_norm else None
        psgd.psgd_adamw_apply(one, cfg, g[0], x, m, v, None, t, norm, _workspace(one))
        assert int(t) == 10
        _check_adamw(one, cfg, g[0], before, (x, m, v), 10, "l2")


def test_many_slices():
    """The most slices a plan takes, on a small plan and through the two-launch path."""
    plan = psgd.psgd_clip_plan_create([(1, 3), (2, 2)], 65535)
    ld = plan.sizes["worker_stride"]
    g = torch.arange(65535, dtype=torch.float32, device=DEV)[:, None].expand(65535, ld).contiguous()
    norms, coefs = torch.zeros(65535, device=DEV), torch.zeros(65535, device=DEV)
    psgd.psgd_grad_clip(plan, g, g, psgd.PSGD_NORM_L2, 100.0, norms, coefs, _workspace(plan))
    want = np.sqrt(7.0) * np.arange(65535, dtype=np.float64)
    _near(norms.cpu(), want, 1.001 * U)
    scaled = np.float32(np.arange(65535)) * coefs.cpu().numpy()
    assert np.array_equal(g[:, 0].cpu().numpy(), scaled) and np.array_equal(g[:, ld - 61].cpu().numpy(), scaled)
    plan = psgd.psgd_clip_plan_create([(1, 1)] * 200, 700)  # 200 tensors: not a small plan
    g = torch.ones((700, plan.sizes["worker_stride"]), device=DEV)
    norms, per = torch.zeros(700, device=DEV), torch.zeros((700, 200), device=DEV)
    psgd.psgd_grad_norm(plan, g, psgd.PSGD_NORM_L2, norms, per, _workspace(plan))
    _near(norms.cpu(), np.full(700, math.sqrt(200.0)), 1.001 * U)
    assert bool((per == 1).all())


def test_capture_is_refused_with_timing_on():
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["ends"], 3)
    g = torch.nan_to_num(_grads(plan, torch.float32, seed=43))
    call, _ = _one_of_each(plan, g, _workspace(plan))
    call()
    psgd.psgd_clip_plan_set_timing(plan, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(psgd.PsgdError) as e:
            call()
        g.add_(0.0)
    assert e.value.status == psgd.PSGD_ERR_INVALID_ARG


def test_two_graphs_of_one_plan_one_after_the_other():
    """Graphs that share a plan and a workspace, replayed in turn on one stream."""
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["mixed"], 3)
    ws = _workspace(plan)
    sets = []
    for seed in (44, 45):
        g = torch.nan_to_num(_grads(plan, torch.float32, seed=seed))
        call, outs = _one_of_each(plan, g, ws)
        call()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        sets.append((graph, outs, want, g))  # a graph reads g as long as it is replayed
    for _ in range(3):
        for graph, outs, _, _ in sets:
            for o in outs:
                o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, outs, want, _ in sets:
            assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_scaled_update_changes_nothing_but_the_norm():
    """Clipping makes AdamW blind to the size of a large update: U and 2^20 U (both clipped)
    give the same c U up to its roundings, and a power of two changes none of them."""
    plan = psgd.psgd_clip_plan_create(SHAPE_SETS["large"], 1)
    g = torch.nan_to_num(_grads(plan, torch.float32, seed=46))[0]
    cfg = psgd.AdamwConfig(max_norm=0.125)
    results = []
    for scale in (1.0, 2.0 ** 20):
        x, m, v, t = _adamw_state(plan, seed=47, step=5)
        norm = torch.zeros(1, device=DEV)
        psgd.psgd_adamw_apply(plan, cfg, g * scale, x, m, v, None, t, norm, _workspace(plan))
        results.append((x, m, v, norm / scale))
    inside = torch.from_numpy(~_padding(plan)).to(DEV)
    for a, b in zip(*results):
        a, b = (a[inside], b[inside]) if a.numel() > 1 else (a, b)
        assert torch.equal(a, b)


@pytest.mark.parametrize("compressor", ["rtopk", "atomo"])
def test_clip_and_adamw_around_the_other_compressors(compressor):
    """Two steps: worker gradients clipped in place, compressed, AdamW from the update."""
    shapes, W = [(20, 33), (33, 20), (1, 9)], 3
    workers, one = psgd.psgd_clip_plan_create(shapes, W), psgd.psgd_clip_plan_create(shapes, 1)
    n = one.sizes["worker_stride"]
    rng = np.random.default_rng(50)
    u, errors = torch.zeros(n, device=DEV), torch.zeros((W, n), device=DEV)
    if compressor == "rtopk":
        plan = psgd.psgd_rtopk_plan_create(shapes, [60, 70, 5], [30, 20, 5], W)
        s = plan.sizes
        index = torch.zeros((W, s["keep_total"]), dtype=torch.int32, device=DEV)
        value = torch.zeros((W, s["keep_total"]), device=DEV)
    else:
        plan = psgd.psgd_atomo_plan_create(shapes, 1.5, W)
        s = plan.sizes
        sv = [torch.zeros((W, s["sv_total"]), device=DEV) for _ in range(2)]
        index = torch.zeros((W, s["sv_total"]), dtype=torch.int32, device=DEV)
        count = torch.zeros((W, s["n_matrices"]), dtype=torch.int32, device=DEV)
        atoms = torch.zeros((W, s["atom_total"]), device=DEV)
    ws = torch.zeros(s["workspace_bytes"], dtype=torch.uint8, device=DEV)

    def compress(g):
        if compressor == "rtopk":
            ranks = psgd.pack_rows(plan, [np.stack([rng.permutation(t) for _ in range(W)]) for t in (60, 70, 5)], "top",
                                   np.uint32).view(np.int32)
            psgd.psgd_rtopk_step(plan, g, errors, torch.from_numpy(ranks).to(DEV), index, value, u, ws)
        else:
            x = torch.from_numpy(rng.random((W, s["sv_total"])).astype(np.float32)).to(DEV)
            psgd.psgd_atomo_step(plan, g, x, sv[0], sv[1], index, count, atoms, u, ws)
        torch.cuda.synchronize()  # the inputs above end with this call

    x, m, v, t = _adamw_state(one, seed=51, step=0)
    norms, coefs, norm = torch.zeros(W, device=DEV), torch.zeros(W, device=DEV), torch.zeros(1, device=DEV)
    cfg = psgd.AdamwConfig(lr=1e-2, max_norm=0.1)
    for step in range(2):
        g = torch.nan_to_num(_grads(workers, torch.float32, seed=52 + step))
        given = g.clone()
        psgd.psgd_grad_clip(workers, g, g, psgd.PSGD_NORM_L2, 0.5, norms, coefs, _workspace(workers))
        compress(g)
        before = [a.clone() for a in (x, m, v)]
        psgd.psgd_adamw_apply(one, cfg, u, x, m, v, None, t, norm, _workspace(one))
        torch.cuda.synchronize()
        _check_clip(workers, given, g, norms, coefs, "l2", 0.5)
        assert bool((u != 0).any()) and int(t) == step + 1
        _check_adamw(one, cfg, u, before, (x, m, v), step + 1, "l2")

"""AdamW where its numbers get long: averages over many steps, large gradients, betas next
to 1.  Against float64, with u = 2^-24 (half a float32 step); tolerances are derived beside
each test.  The element counts take the single launch, the joined partials and cl_final."""

import math
from decimal import Decimal, localcontext

import numpy as np
import pytest

from distributed_sgd_gradient_ef_amd import psgd
from tests.test_gpu_clip import DEV, DTYPES, U, _adamw_state, _check_adamw, _padding, _workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SIZES = {"single": 8000, "joined": 65536, "final": 2_200_000}


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    return psgd.load_library()


@pytest.mark.parametrize("beta", [0.9999, 0.99999])
@pytest.mark.parametrize("max_norm", [0.0, math.inf])
@pytest.mark.parametrize("size", SIZES)
def test_moments_stay_the_average_of_the_gradients(size, max_norm, beta):
    """2000 steps on random gradients, from moments at their steady state.

    Each step rounds a moment once by at most u of it; on random gradients these roundings
    are independent and have mean zero.  So the mean over n elements is off by at most
    1.5 u sqrt(2 T ln(2e9) / n) but for one case in 1e9 (Hoeffding; 1.5 bounds an element's
    moment against the mean).  One-sided are only the new gradient's weight and products:
    3 u.  A pair of weights that does not add up to 1, or not to the step's beta, drifts by
    up to u / 2 every step: hundreds of u."""
    n, steps = SIZES[size], 2000
    plan = psgd.psgd_clip_plan_create([(1, n)], 1)
    ld = plan.sizes["worker_stride"]
    gen = torch.Generator(device=DEV).manual_seed(71)
    cfg = psgd.AdamwConfig(lr=1e-3, beta1=beta, beta2=beta, max_norm=max_norm)
    x, m, v = torch.zeros(ld, device=DEV), torch.full((ld,), 1.5, device=DEV), torch.full((ld,), 2.5, device=DEV)
    m64, v64 = m[:n].double(), v[:n].double()
    t = torch.full((1,), 10 ** 6, dtype=torch.int64, device=DEV)
    norm, ws = torch.zeros(1, device=DEV) if max_norm else None, _workspace(plan)
    for _ in range(steps):
        g = torch.randn(ld, generator=gen, device=DEV) * 0.5 + 1.5
        psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, norm, ws)
        d = g[:n].double()
        m64.mul_(beta).add_(d, alpha=1.0 - beta)
        v64.mul_(beta).addcmul_(d, d, value=1.0 - beta)
    tol = (3.0 + 1.5 * math.sqrt(2 * steps * math.log(2e9) / n)) * U
    for got, want in ((m, m64), (v, v64)):
        mean = float(want.mean())
        assert float(want.max()) <= 1.5 * mean
        off = float((got[:n].double() - want).mean()) / mean
        assert abs(off) <= tol, (off / U, tol / U)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("max_norm,flags", [(0.0, 0), (math.inf, psgd.PSGD_ADAMW_SKIP_NONFINITE)])
@pytest.mark.parametrize("size", SIZES)
def test_second_moment_of_large_gradients(size, max_norm, flags, dtype):
    """g^2 is past float32's range, (1 - beta2) g^2 is not (to _check_adamw's tolerances)."""
    code, td = DTYPES[dtype]
    n = SIZES[size]
    plan = psgd.psgd_clip_plan_create([(1, n)], 1, code)
    rng = np.random.default_rng(72)
    a = 1e20 * (1.0 + rng.random(plan.sizes["worker_stride"])) * rng.choice([-1.0, 1.0], plan.sizes["worker_stride"])
    g = torch.from_numpy(a.astype(np.float32)).to(td).to(DEV)
    cfg = psgd.AdamwConfig(lr=1e-2, max_norm=max_norm, flags=flags)
    for step in (0, 3):
        x, m, v, t = _adamw_state(plan, seed=73, step=step)
        before = [b.clone() for b in (x, m, v)]
        norm = torch.zeros(1, device=DEV) if max_norm else None
        psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, norm, _workspace(plan))
        assert int(t) == step + 1
        inside = torch.from_numpy(~_padding(plan)).to(DEV)
        assert bool(torch.isfinite(v[inside]).all())
        _check_adamw(plan, cfg, g, before, (x, m, v), step + 1, "l2")


@pytest.mark.parametrize("beta2", [0.5, 0.999])
@pytest.mark.parametrize("size", SIZES)
def test_an_infinite_second_moment_stays_infinite(size, beta2):
    """beta2 * inf is inf for every beta2, also one that float32 holds exactly: the weight
    only decays (1 - 2^-4, exact), and its neighbours take their step."""
    n = SIZES[size]
    plan = psgd.psgd_clip_plan_create([(1, n)], 1)
    ld = plan.sizes["worker_stride"]
    g, x = torch.ones(ld, device=DEV), torch.ones(ld, device=DEV)
    m, v = torch.zeros(ld, device=DEV), torch.zeros(ld, device=DEV)
    bad = torch.zeros(ld, dtype=torch.bool, device=DEV)
    bad[[0, 70, n - 1]] = True
    v[bad] = math.inf
    t = torch.zeros(1, dtype=torch.int64, device=DEV)
    cfg = psgd.AdamwConfig(lr=0.125, beta1=0.5, beta2=beta2, weight_decay=0.5)
    psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, None, _workspace(plan))
    assert bool((v[bad] == math.inf).all()) and bool((x[bad] == 0.9375).all()) and bool((m[:n] == 0.5).all())
    rest = ~bad
    rest[n:] = False
    # 1 - 2^-4 - lr / (1 + 1e-8): a step within 17 u of itself and three roundings below 1
    assert bool(((x[rest] - 0.8125).abs() <= 5 * U + 17 * U * 0.125 + 2e-9).all())


@pytest.mark.parametrize("gap", [1e-9, 1e-12])
@pytest.mark.parametrize("max_norm", [0.0, math.inf])
@pytest.mark.parametrize("size", SIZES)
def test_bias_corrections_of_betas_next_to_one(size, max_norm, gap):
    """1 - beta^t without cancellation: the weights' step is right to _check_adamw's 17 u and
    the first moment's 5 u, also where 1 - beta^t is as small as 2e-12."""
    n = SIZES[size]
    beta = 1.0 - gap
    w = 1.0 - beta  # exact
    plan = psgd.psgd_clip_plan_create([(1, n)], 1)
    ld = plan.sizes["worker_stride"]
    g = torch.linspace(0.5, 1.5, ld, device=DEV)
    cfg = psgd.AdamwConfig(lr=0.5, beta1=beta, beta2=beta, eps=1e-8, weight_decay=0.0, max_norm=max_norm)
    for step in (0, 1, 2, 6, 99, 12344):
        x = torch.zeros(ld, device=DEV)
        m, v = (torch.full((ld,), float(np.float32(w * step)), device=DEV) for _ in range(2))
        m0 = float(m[0])
        t = torch.full((1,), step, dtype=torch.int64, device=DEV)
        norm = torch.zeros(1, device=DEV) if max_norm else None
        psgd.psgd_adamw_apply(plan, cfg, g, x, m, v, None, t, norm, _workspace(plan))
        with localcontext() as ctx:
            ctx.prec = 60
            bc = float(1 - Decimal(beta) ** (step + 1))
        d = g[:n].double().cpu().numpy()
        m1 = beta * m0 + w * d
        want = -0.5 * (m1 / bc) / (np.sqrt((beta * m0 + w * d * d) / bc) + 1e-8)
        got = x[:n].double().cpu().numpy()
        off = np.max(np.abs(got - want) / np.abs(want))
        assert off <= 23 * 1.01 * U, (step, off / U)

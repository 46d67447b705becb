"""Language-model ends on the GPU: every variant that sizes and types choose, entry by entry.

The reference is float64 on the GPU, one worker at a time, from the formulas of psgd_lm.h; the
bounds are those of test_gpu_lm_numerics.py, with dropout's factor (the float32 next to
1 / (1 - p), u / 2, and a product's rounding, u: 2 u of a score, 2 u of a gradient)."""

import numpy as np
import pytest

from distributed_sgd_gradient_ef_amd import psgd
from oracle import lm as O
from tests.gpu_harness import log
from tests.test_gpu_lm import HALF, TYPES, U, Case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def torch_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    psgd.load_library()
    return torch


class Worker:
    """One worker's scores in float64 and the bound of their error."""

    def __init__(self, c, w, mask):
        torch = self.torch = c.torch
        self.c, self.T = c, c.params[c.span].double().view(c.s["vocab"], c.s["dim"])
        t = c.words[w]
        self.ok = (t >= 0) & (t < c.s["vocab"])
        self.t = torch.where(self.ok, t, 0)
        self.mask = mask[w] if mask is not None else None
        x = c.x[w].double() * (self.mask if mask is not None else 1.0)
        self.x = torch.where(self.ok[:, None], x, 0.0)
        self.s = self.x @ self.T.t()
        a, A, f32 = self.x.abs(), self.T.abs(), c.act == "f32"
        self.es = (a @ A.t()) * ((2 * c.n_adds(c.s["dim"]) + (20 if f32 else 8) + (2 if mask is not None else 0)) * U)
        if f32:
            self.es += 2.0 ** -49 * (a.amax(1, keepdim=True) * A.sum(1) + A.amax(1) * a.sum(1, keepdim=True))

    def loss(self):
        """((losses, lse), their bounds): sums of 64 terms in a lane, 2 per tile, 16 over the tiles."""
        torch, s = self.torch, self.s
        top = s.amax(1, keepdim=True)
        lse = torch.logsumexp(s, 1)
        rel = (torch.exp(s - lse[:, None]) * (self.es + 2 * U * (top - s + 3))).sum(1) + 2 * U * (86 + 4 * s.shape[1] / 256)
        at = self.t[:, None]
        hit, e_hit = s.gather(1, at)[:, 0], self.es.gather(1, at)[:, 0]
        e_lse = 1.01 * rel + 2 * U * (lse.abs() + 1)
        e_loss = 1.01 * rel + 1.01 * e_hit + 3 * U * (1 + lse - hit)
        zero = torch.zeros_like(lse)
        return [torch.where(self.ok, v, zero) for v in (lse - hit, lse, e_loss, e_lse)]

    def grad(self, lse, scale):
        """((dx, table gradient), their bounds)."""
        torch, c = self.torch, self.c
        f32, f32g = c.act == "f32", c.grad == "f32"
        coef = float(scale) / max(1, int(self.ok.sum()))
        away = torch.where(self.ok[:, None], self.s - lse.double()[:, None], -torch.inf)
        p = torch.exp(away)
        away = torch.where(self.ok[:, None], away, 0.0)
        eg = p * (torch.expm1(self.es) + 2 * U * (away.abs() + 3))
        p.scatter_add_(1, self.t[:, None], torch.where(self.ok, -1.0, 0.0).double()[:, None])
        g = p.mul_(coef)
        eg = eg.mul_(abs(coef)) + 4 * U * g.abs()
        n_x, n_w = c.n_adds(c.s["vocab"]) + 20, 3 * (-(-c.s["rows"] // 16) + 4)
        rest_x = 2.1 * U if f32 else HALF["bf16"]
        rest_w = 2.1 * U if f32g else 3.1 * 2.0 ** -16 if f32 else HALF["bf16"]
        A, a, G = self.T.abs(), self.x.abs(), g.abs()
        dx, e_dx = g @ self.T, eg @ A + (G @ A) * ((2 * n_x + 8) * U + rest_x)
        gw, e_gw = g.t() @ self.x, eg.t() @ a + (G.t() @ a) * ((2 * n_w + 8) * U + rest_w)
        if self.mask is not None:
            dx, e_dx, e_gw = dx * self.mask, e_dx * self.mask + 2 * U * dx.abs() * self.mask, e_gw + 2 * U * gw.abs()
        return dx, gw, e_dx, e_gw


def off(name, got, want, err, t):
    got = got.double()
    assert got.isfinite().all(), name
    err = 1.01 * err + HALF[t] * (want.abs() + err) + 1e-37
    worst = float(((got - want).abs() / err).max())
    log(f"   {name}: {worst:.3f} of the bound")
    assert worst <= 1, name


def run(torch, vocab, dim, workers, rows, act, grad, drop, add, loss_only=False):
    log(f"[case] {vocab} x {dim}, {workers} workers, {rows} rows, {act} {grad}, drop {drop}, add {add}")
    c = Case(torch, vocab, dim, workers, rows, act, grad, drop=drop, seed=vocab + dim)
    mask = None
    if drop is not None:
        mask = torch.from_numpy(O.kept(tuple(c.x.shape), *drop)).to(DEV).double() / (1 - drop[0])
    psgd.psgd_lm_plan_set_timing(c.plan, True)
    losses, lse, mean = c.loss()
    dx, grads = (None, None) if loss_only else c.loss_grad(lse, True, add)
    stats = psgd.psgd_lm_plan_kernel_stats(c.plan)
    span = slice(c.s["table_offset"], c.s["table_offset"] + vocab * dim)
    for w in range(workers):
        r = Worker(c, w, mask)
        want_loss, want_lse, e_loss, e_lse = r.loss()
        off("losses", losses[w], want_loss, e_loss, "f32")
        off("lse", lse[w], want_lse, e_lse, "f32")
        n = max(1, int(r.ok.sum()))
        assert abs(float(mean[w]) - float(want_loss.sum()) / n) <= 1.01 * float(e_loss.sum()) / n + 2 * U * float(mean[w])
        if loss_only:
            continue
        want_dx, want_g, e_dx, e_g = r.grad(lse[w], c.scale_np[w])
        off("dx", dx[w], want_dx, e_dx, act)
        if add:
            want_g = want_g + c.old[w, span].double().view(vocab, dim)
        off("grads", grads[w, span].view(vocab, dim), want_g, e_g + 2 * U * want_g.abs(), grad)
        rest = torch.ones(c.s["worker_stride"], dtype=torch.bool, device=DEV)
        rest[span] = False
        assert torch.equal(grads[w, rest], c.old[w, rest])
        del r, want_dx, want_g, e_dx, e_g
    return stats


DROP = (0.3, 0x1234567, 2 ** 32 + 9)


@pytest.mark.parametrize("act,grad", TYPES)
@pytest.mark.parametrize("dim", [192, 130, 650])
@pytest.mark.parametrize("drop,add", [(None, False), (DROP, True)])
def test_large_tiles(torch_gpu, dim, act, grad, drop, add):
    """36 x 4 score tiles of 256 x 256, more than the 128 from which on they are the large ones, for
    the loss and the gradients; a bfloat16 table with dim 192 is read as it is.  The products'
    tiles are the large ones too: 4 of dx and 36 of every worker's table gradient, for every 256 columns."""
    run(torch_gpu, 9001, dim, 4 if dim < 256 else 2, 210 if dim < 256 else 420, act, grad, drop, add)


@pytest.mark.parametrize("act,grad", TYPES)
@pytest.mark.parametrize("dim,drop,add", [(64, None, False), (64, DROP, True), (40, DROP, False), (192, None, True)])
def test_several_pieces_of_the_vocabulary(torch_gpu, dim, act, grad, drop, add):
    """g of all words is past the 512 MB that are held at a time: 2 workers' 1000 rows take two pieces in
    bfloat16, four in parts; neither words nor rows are whole blocks."""
    stats = run(torch_gpu, 140001, dim, 2, 1000, act, grad, drop, add)
    assert stats["lm_products"][0] >= 2 and stats["lm_scores"][0] == 1 + stats["lm_products"][0]


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_several_chunks_of_rows(torch_gpu, act):
    """Maxima and sums of 24,000 rows are past the 64 MB that are held at a time."""
    stats = run(torch_gpu, 100001, 64, 1, 24000, act, act, DROP, False, loss_only=True)
    assert stats["lm_scores"][0] >= 2 and stats["lm_rows"][0] == stats["lm_scores"][0]


@pytest.mark.parametrize("act,grad", TYPES)
@pytest.mark.parametrize("drop", [None, DROP])
@pytest.mark.parametrize("vocab,dim,workers,rows", [(130, 37, 3, 70), (1001, 128, 2, 5), (70, 64, 2, 130)])
def test_small_tiles_with_dropout(torch_gpu, vocab, dim, workers, rows, drop, act, grad):
    """bfloat16 activations through dropout are not rounded again: the bounds are those without it."""
    run(torch_gpu, vocab, dim, workers, rows, act, grad, drop, rows % 2 == 1)

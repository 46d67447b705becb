"""Dropout, embedding and cross entropy as a training step uses them: all together and with the
compressors around them, captured and replayed, on other streams, with masked rows that hold
anything, on sizes past 32 bits."""

import numpy as np
import pytest

from distributed_sgd_gradient_ef_amd import psgd
from oracle import lm as O
from tests.gpu_harness import log
from tests.test_gpu_lm import HALF, U, Case, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch_gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no ROCm GPU visible")
    psgd.load_library()
    return torch


DEV = "cuda:0"


class Model:
    """Embedding, one dense tanh layer and the tied output, on every worker's own tokens: what a
    user's program does around the calls is plain torch in float32."""

    def __init__(self, torch, seed=1, vocab=501, dim=40, workers=3, rows=70, p=0.25):
        self.torch = torch
        rng = np.random.default_rng(seed)
        self.shapes = [(dim, dim), (vocab, dim), (1, dim)]
        self.W, self.T, self.V, self.D, self.p = workers, rows, vocab, dim, p
        self.plan = psgd.psgd_lm_plan_create(self.shapes, 1, workers, rows)
        self.off = [0]
        for r, c in self.shapes:
            self.off.append(-(-(self.off[-1] + r * c) // 64) * 64)
        s = self.plan.sizes
        assert s["table_offset"] == self.off[1] and s["worker_stride"] == self.off[3]
        n = s["worker_stride"]
        self.params = torch.zeros(n, device=DEV)
        for i, (r, c) in enumerate(self.shapes):
            self.params[self.off[i]:self.off[i] + r * c] = torch.from_numpy(rng.standard_normal(r * c).astype(np.float32) * 0.3).to(DEV)
        self.tokens = torch.from_numpy(rng.integers(0, vocab, (workers, rows))).to(DEV)
        self.targets = torch.from_numpy(rng.integers(-1, vocab, (workers, rows))).to(DEV)
        self.step = torch.zeros(1, dtype=torch.int64, device=DEV)
        self.grads = torch.zeros((workers, n), device=DEV)
        self.ws = torch.empty(s["workspace_bytes"], dtype=torch.uint8, device=DEV)
        shape = (workers, rows, dim)
        self.h, self.dx = torch.zeros(shape, device=DEV), torch.zeros(shape, device=DEV)
        self.losses, self.lse = torch.zeros(shape[:2], device=DEV), torch.zeros(shape[:2], device=DEV)
        self.mean = torch.zeros(workers, device=DEV)
        # layers are told apart by their seeds, steps by the optimizer's step count
        self.drop_in, self.drop_out = psgd.DropoutConfig(p, 11, self.step), psgd.DropoutConfig(p, 22, self.step)

    def tensor(self, i, flat=None):
        r, c = self.shapes[i]
        flat = self.params if flat is None else flat
        return flat[..., self.off[i]:self.off[i] + r * c].unflatten(-1, (r, c))

    def gradients(self):
        torch = self.torch
        psgd.psgd_lm_embed(self.plan, self.params, self.tokens, self.drop_in, self.h)
        dense, bias = self.tensor(0), self.tensor(2)[0]
        y = torch.tanh(self.h @ dense.t() + bias)
        psgd.psgd_lm_loss(self.plan, y, self.params, self.targets, self.drop_out, self.losses, self.lse, self.mean, self.ws)
        psgd.psgd_lm_loss_grad(self.plan, y, self.params, self.targets, self.lse, None, self.drop_out, self.dx, self.grads, 0,
                               self.ws)
        dy = self.dx * (1 - y * y)
        self.tensor(0, self.grads).copy_(dy.transpose(1, 2).contiguous() @ self.h)
        self.tensor(2, self.grads).copy_(dy.sum(1, keepdim=True))
        psgd.psgd_lm_embed_grad(self.plan, self.tokens, dy @ dense, self.drop_in, self.grads, psgd.PSGD_LM_ACCUMULATE, self.ws)

    def reference(self):
        """(means, [gradient of every tensor]) in float64 from automatic differentiation on the CPU."""
        torch = self.torch
        leaves = [self.tensor(i).double().cpu().requires_grad_() for i in range(3)]
        step = int(self.step[0])
        masks = [torch.from_numpy(O.dropout(np.ones((self.W, self.T, self.D)), (self.p, seed, step))) for seed in (11, 22)]
        h = leaves[1][self.tokens.cpu()] * masks[0]
        x = torch.tanh(h @ leaves[0].t() + leaves[2][0]) * masks[1]
        means, grads = [], [[] for _ in leaves]
        for w in range(self.W):
            t = self.targets[w].cpu()
            mean = torch.nn.functional.cross_entropy(x[w][t >= 0] @ leaves[1].t(), t[t >= 0])
            means.append(float(mean.detach()))
            for g, one in zip(grads, torch.autograd.grad(mean, leaves, retain_graph=True)):
                g.append(one)
        return np.array(means), [torch.stack(g).numpy() for g in grads]


def _off(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def test_training_steps_with_everything_around_them(torch_gpu):
    """Three steps: the model's gradients, clipping, PowerSGD, AdamW.  The forward pass's sums are
    of at most 501 terms in float32, so means and gradients are within 1e-5 of float64 (2^-24 times
    the terms' root, times the depth of the chain, is below 2e-6)."""
    torch = torch_gpu
    m = Model(torch)
    clip, one = psgd.psgd_clip_plan_create(m.shapes, m.W), psgd.psgd_clip_plan_create(m.shapes, 1)
    comp = psgd.psgd_plan_create(m.shapes, 2, m.W)
    n = m.plan.sizes["worker_stride"]
    errors, update = torch.zeros((m.W, n), device=DEV), torch.zeros(n, device=DEV)
    q = torch.randn(comp.sizes["q_elems"], device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    pp = torch.zeros(comp.sizes["p_elems"], device=DEV)
    norms, coefs, norm = (torch.zeros(k, device=DEV) for k in (m.W, m.W, 1))
    exp_avg, exp_avg_sq = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    wss = {p: torch.empty(p.sizes["workspace_bytes"], dtype=torch.uint8, device=DEV) for p in (clip, one, comp)}
    for step in range(3):
        m.gradients()
        means, grads = m.reference()
        log(f"[step {step}] mean losses {means}")
        assert _off(m.mean.double().cpu().numpy(), means) < 1e-5
        for i, g in enumerate(grads):
            assert _off(m.tensor(i, m.grads).double().cpu().numpy(), g) < 1e-5, i
        before = m.params.clone()
        psgd.psgd_grad_clip(clip, m.grads, m.grads, psgd.PSGD_NORM_L2, 0.5, norms, coefs, wss[clip])
        psgd.psgd_compress_step(comp, m.grads, errors, q, pp, update, wss[comp])
        psgd.psgd_adamw_apply(one, psgd.AdamwConfig(lr=0.01, max_norm=1.0), update, m.params, exp_avg, exp_avg_sq, None,
                              m.step, norm, wss[one])
        assert not torch.equal(before, m.params) and int(m.step[0]) == step + 1


def test_step_in_a_graph_draws_new_masks(torch_gpu):
    torch = torch_gpu
    a, b = Model(torch), Model(torch)
    a.gradients()  # torch's own products: their libraries are set up outside of the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.gradients()
        a.step.add_(1)
    torch.cuda.synchronize()
    scratch, seen = torch.zeros(1 << 20, device=DEV), []
    for replay in range(4):
        graph.replay()
        scratch.add_(1.0)
        torch.cuda.synchronize()
        b.gradients()
        b.step.add_(1)
        torch.cuda.synchronize()
        for name in ("h", "losses", "lse", "mean", "dx", "grads", "step"):
            x, y = getattr(a, name), getattr(b, name)
            # the dense layer's products are the library's, which may choose otherwise in a capture
            assert torch.allclose(x, y, rtol=1e-5, atol=1e-6), (replay, name)
        assert torch.equal(a.h, b.h)
        seen.append(a.h.clone())
    assert not any(torch.equal(seen[0], s) for s in seen[1:])


@pytest.mark.parametrize("act,grad", [("f32", "f32"), ("bf16", "bf16")])
def test_own_calls_in_graphs_that_share_a_plan(torch_gpu, act, grad):
    """Two graphs of the same plan with a workspace each, replayed on two streams at once."""
    torch = torch_gpu
    cases = [Case(torch, 3001, 72, 2, 90, act, grad, drop=(0.2, 5, k), seed=k) for k in range(2)]
    plan = cases[0].plan
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.plan = plan
        outs.append(dict(loss=[c.nan(2, 90), c.nan(2, 90), c.nan(2)], dx=c.nan(*c.x.shape, dtype=c.at), grads=c.old.clone(),
                         out=c.nan(*c.x.shape, dtype=c.at)))

    def run(c, o):
        psgd.psgd_lm_embed(plan, c.params, c.words, c.config, o["out"])
        psgd.psgd_lm_loss(plan, c.x, c.params, c.words, c.config, *o["loss"], c.workspace)
        psgd.psgd_lm_loss_grad(plan, c.x, c.params, c.words, o["loss"][1], c.scale, c.config, o["dx"], o["grads"], 0, c.workspace)
        psgd.psgd_lm_embed_grad(plan, c.words, c.x, c.config, o["grads"], psgd.PSGD_LM_ACCUMULATE, c.workspace)
        psgd.psgd_dropout(c.x.view(180, 72), o["dx"].view(180, 72), o["dx"].view(180, 72), c.config)

    want = []
    for c, o in zip(cases, outs):
        run(c, o)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (*o["loss"], o["dx"], o["grads"], o["out"])])
        for t in (*o["loss"], o["dx"], o["grads"][:, c.span], o["out"]):
            t.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(c, o)
        graphs.append(g)
    torch.cuda.synchronize()
    for replay in range(4):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            for x, y in zip((*o["loss"], o["dx"], o["grads"], o["out"]), w):
                assert torch.equal(x, y), replay


def test_timed_plans_are_not_captured(torch_gpu):
    torch = torch_gpu
    c = Case(torch, 65, 8, 1, 4)
    c.loss()
    psgd.psgd_lm_plan_set_timing(c.plan, True)
    c.loss()
    stats = psgd.psgd_lm_plan_kernel_stats(c.plan, reset=True)
    assert {"lm_peak", "lm_pack", "lm_scores", "lm_rows"} <= set(stats) and all(n == 1 and ms > 0 for n, ms in stats.values())
    with pytest.raises(psgd.PsgdError) as e:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            c.loss()
    assert e.value.status == psgd.PSGD_ERR_INVALID_ARG


def test_calls_go_to_the_current_stream(torch_gpu):
    """The inputs become ready on a stream of their own; the calls are made on it, or name it."""
    torch = torch_gpu
    c = Case(torch, 700, 64, 2, 65)
    want = [t.clone() for t in c.loss()]
    x, slow = c.x.clone(), torch.zeros(1 << 26, device=DEV)
    torch.cuda.synchronize()
    for named in (False, True):
        st = torch.cuda.Stream()
        out = c.nan(2, 65), c.nan(2, 65), c.nan(2)
        c.x.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(20):
                slow.add_(1.0)
            c.x.copy_(x)
            if not named:
                psgd.psgd_lm_loss(c.plan, c.x, c.params, c.words, None, *out, c.workspace)
        if named:
            psgd.psgd_lm_loss(c.plan, c.x, c.params, c.words, None, *out, c.workspace, stream=st)
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("act,grad", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("vocab,dim,rows", [(90, 24, 33), (9001, 640, 600)])
def test_rows_that_do_not_count_may_hold_anything(torch_gpu, act, grad, junk, vocab, dim, rows):
    torch = torch_gpu
    c = Case(torch, vocab, dim, 2, rows, act, grad, seed=8, bad=0.4)
    c.words[1] = -1  # a worker without counted rows
    off = (c.words < 0) | (c.words >= vocab)
    c.x[off] = 0
    want = [t.clone() for t in c.loss()]
    want += c.loss_grad(want[1])
    c.x[off] = junk
    got = list(c.loss())
    lse = got[1].clone()
    lse[off] = junk
    got += c.loss_grad(lse)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not got[0][1].any() and float(got[2][1]) == 0 and not got[3][off].any()
    assert not got[4][1, c.span].any()


def test_one_bad_word_reaches_every_counted_row_and_no_other(torch_gpu):
    torch = torch_gpu
    for act in ("f32", "bf16"):
        c = Case(torch, 200, 16, 2, 40, act, act, seed=3)
        c.words[1] = -100
        off = c.s["table_offset"]
        c.params[off + 77 * 16] = float("nan")
        losses, lse, mean = c.loss()
        counted = (c.words >= 0) & (c.words < 200)
        assert torch.equal(torch.isnan(losses), counted) and torch.isnan(mean[0]) and mean[1] == 0
        dx, grads = c.loss_grad(lse)
        assert torch.equal(torch.isnan(dx).all(-1), counted) and not dx[~counted].any()
        assert torch.isnan(grads[0, c.span]).any() and not grads[1, c.span].any()


@pytest.mark.parametrize("act,grad", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_equal_calls_give_equal_bits(torch_gpu, act, grad):
    torch = torch_gpu
    c = Case(torch, 12001, 200, 2, 333, act, grad, seed=5)
    first = list(c.loss())
    first += c.loss_grad(first[1])
    for _ in range(3):
        c.workspace.fill_(255)
        again = list(c.loss())
        again += c.loss_grad(first[1])
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_slopes_of_the_loss(torch_gpu):
    """The gradients against differences of the losses, along the gradient.  Along a direction that
    changes no score by more than 1 per unit, the third derivative of a mean of log sum exp is a
    mean of third central moments of values in [-1, 1], below 8: a difference over 2h is off by
    8 h^2 / 6, and by the two means' own errors, 2^-20 each, over 2h; moved entries are rounded
    to float32, which is taken into account."""
    torch = torch_gpu
    c = Case(torch, 300, 32, 1, 50, seed=9, bad=0.0)
    lse = c.loss()[1]
    dx, grads = c.loss_grad(lse)
    h = 2.0 ** -5
    for which in ("x", "table"):
        target, g = (c.x, dx) if which == "x" else (c.params[c.span], grads[0, c.span])
        other = c.params[c.span] if which == "x" else c.x
        base = target.clone()
        d = g.reshape(-1, 32) / g.reshape(-1, 32).norm(dim=1, keepdim=True).clamp(min=1e-30)
        d = (d / other.reshape(-1, 32).norm(dim=1).max()).view(base.shape)
        sides = []
        for sign in (1, -1):
            target.copy_(base + sign * h * d)
            sides.append((float(c.loss()[2]), target.double().clone()))
        target.copy_(base)
        slope, moved = sides[0][0] - sides[1][0], sides[0][1] - sides[1][1]
        want = float((g.double() * moved).sum())
        tol = 2 * h * (8 * h * h / 6) + 2 ** -19
        log(f"   {which}: difference {slope:.6f}, gradient {want:.6f}, tolerance {tol:.6f}")
        assert abs(slope - want) <= tol and want > 20 * tol


def test_many_rows_take_several_chunks_and_pieces(torch_gpu):
    """A vocabulary and a number of rows past the chunks of the loss and the pieces of the gradient,
    against float64 on the GPU."""
    torch = torch_gpu
    V, D, T = 100000, 16, 24000
    c = Case(torch, V, D, 1, T, "f32", "f32", seed=2)
    losses, lse, mean = c.loss()
    dx, grads = c.loss_grad(lse)
    x, table, t = c.x[0].double(), c.params[c.span].double().view(V, D), c.words[0]
    ok = (t >= 0) & (t < V)
    gw, worst = torch.zeros((V, D), dtype=torch.float64, device=DEV), 0.0
    for r in range(0, T, 4000):
        s = x[r:r + 4000] @ table.t()
        ref = torch.logsumexp(s, 1)
        part = ok[r:r + 4000]
        worst = max(worst, float((ref - lse[0, r:r + 4000].double())[part].abs().max()))
        p = torch.exp(s - lse[0, r:r + 4000].double()[:, None])
        p[torch.arange(len(s), device=DEV), t[r:r + 4000].clamp(0, V - 1)] -= 1
        p *= (part.double() / ok.sum())[:, None]
        want = p @ table
        assert float((want - dx[0, r:r + 4000].double()).norm() / want.norm()) < 2 ** -17
        gw += p.t() @ x[r:r + 4000]
    assert worst < 2 ** -17  # sums of 1e5 terms, scores below 8
    assert float((gw - grads[0, c.span].double().view(V, D)).norm() / gw.norm()) < 2 ** -17
    assert abs(float(mean) - float(losses.double().sum() / ok.sum())) < 1e-6


def test_slices_past_two_to_the_31_elements(torch_gpu):
    torch = torch_gpu
    V, D, W = 30011, 30000, 3  # 900 million elements per worker
    log("[case] three workers' table gradients of 0.9e9 bfloat16 entries")
    plan = psgd.psgd_lm_plan_create([(V, D)], 0, W, 9, psgd.PSGD_BF16, psgd.PSGD_BF16)
    s = plan.sizes
    grads = torch.empty((W, s["worker_stride"]), dtype=torch.bfloat16, device=DEV).fill_(3.0)
    tokens = torch.tensor([[0, V - 1, 5, 5, V - 1, -1, V, 7, 5]] * W, device=DEV)
    dout = torch.randn((W, 9, D), device=DEV).bfloat16()
    ws = torch.empty(s["workspace_bytes"], dtype=torch.uint8, device=DEV)
    psgd.psgd_lm_embed_grad(plan, tokens, dout, None, grads, 0, ws)
    for w in range(W):
        table = grads[w, :V * D].view(V, D)
        d = dout[w].double()
        for v, rows in ((0, [0]), (V - 1, [1, 4]), (5, [2, 3, 8]), (7, [7])):
            want, size = d[rows].sum(0), d[rows].abs().sum(0)
            assert ((table[v].double() - want).abs() <= HALF["bf16"] * want.abs() + 4 * U * size).all(), (w, v)
        assert not table[1:5].any() and not table[8:V - 1].any() and not table[6].any()
    out = torch.zeros((W, 9, D), dtype=torch.bfloat16, device=DEV)
    psgd.psgd_lm_embed(plan, grads[2], tokens, None, out)
    assert torch.equal(out[1, 1], grads[2, (V - 1) * D:V * D]) and not out[:, 5:7].any()


def test_dropout_past_two_to_the_32_entries(torch_gpu):
    torch = torch_gpu
    log("[case] dropout of 4.4e9 bfloat16 entries, in place")
    for cols in (65536, 65539):
        rows = 66000
        x = torch.ones((rows, cols), dtype=torch.bfloat16, device=DEV)
        psgd.psgd_dropout(x, None, x, psgd.DropoutConfig(0.5, 123))
        for first in (0, (1 << 32) - 4096, (1 << 32), rows * cols // 4 * 4 - 8192):
            n = min(8192, rows * cols - first)
            want = O.kept((n,), 0.5, 123, 0, first) * 2.0
            assert np.array_equal(x.view(-1)[first:first + n].float().cpu().numpy(), want), (cols, first)
        del x
        torch.cuda.empty_cache()


def test_refusals_leave_the_buffers(torch_gpu):
    torch = torch_gpu
    c = Case(torch, 50, 8, 2, 6)
    good = dict(x=c.x, params=c.params, targets=c.words)
    outs = c.nan(2, 6), c.nan(2, 6), c.nan(2)
    for name, bad in {"x": c.x.bfloat16(), "params": c.params[:-1], "targets": c.words.int()}.items():
        with pytest.raises(psgd.PsgdError) as e:
            a = {**good, name: bad}
            psgd.psgd_lm_loss(c.plan, a["x"], a["params"], a["targets"], None, *outs, c.workspace)
        assert e.value.status == psgd.PSGD_ERR_INVALID_ARG
    with pytest.raises(psgd.PsgdError):
        psgd.psgd_lm_loss(c.plan, c.x.transpose(1, 2), c.params, c.words, None, *outs, c.workspace)
    with pytest.raises(psgd.PsgdError):
        psgd.psgd_lm_loss(c.plan, c.x, c.params, c.words, psgd.DropoutConfig(1.5), *outs, c.workspace)
    with pytest.raises(psgd.PsgdError):
        psgd.DropoutConfig(0.5, 0, torch.zeros(1, dtype=torch.int64))  # a step on the host
    x = torch.zeros((4, 8), device=DEV)
    for args in ((x, None, x[:2]), (x, x.bfloat16(), x), (x.t(), None, x.t()), (x[:, :4], None, x[:, 4:]),
                 (x.double(), None, x.double()), (x[0], None, x[0]), (x.expand(3, 4, 8)[0], x[:1].expand(4, 8), x)):
        with pytest.raises(psgd.PsgdError):
            psgd.psgd_dropout(*args, psgd.DropoutConfig(0.5))
    assert torch.isnan(outs[0]).all() and not x.any()
    empty = torch.zeros((0, 8), device=DEV)
    psgd.psgd_dropout(empty, None, empty, psgd.DropoutConfig(0.5))

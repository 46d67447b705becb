"""The gradient-norm, clipping and AdamW operators as measured workloads.

Each case is one call of `psgd_grad_norm`, `psgd_grad_clip` or `psgd_adamw_apply` on a
packed buffer of many tensors.  With `own` false the same results come from elementary
torch operations in 32 bits (64 for the long sums).
"""

import math
import random

import torch

own = False

# CIFAR ResNet-18: convolutions as out_ch x (in_ch*k*k), batch-norm vectors, classifier.
RESNET18 = (
    "64x27 1x64*2 64x576 1x64*2 64x576 1x64*2 64x576 1x64*2 64x576 1x64*2 "
    "128x576 1x128*2 128x1152 1x128*2 128x64 1x128*2 128x1152 1x128*2 128x1152 1x128*2 "
    "256x1152 1x256*2 256x2304 1x256*2 256x128 1x256*2 256x2304 1x256*2 256x2304 1x256*2 "
    "512x2304 1x512*2 512x4608 1x512*2 512x256 1x512*2 512x4608 1x512*2 512x4608 1x512*2 "
    "10x512 1x10"
)
LSTM = "33278x650 2600x650*6"           # a tied embedding and three recurrent layers
SQUARES = "4096x4096*16 8192x8192*2"    # a quarter of the bandwidth-stress set
RAGGED = "1x1*20 1x7*10 1x63*20 7x129*30 33x1025*20 257x511*12 1x65537*4 1999x1001*3"
TINY = "64x27 1x64 10x512 3x5"


def listed():
    def norm(name, shapes, slices, dtype, kind="l2", tensors=False):
        return {"name": name, "op": "norm", "shapes": shapes, "slices": slices, "dtype": dtype, "kind": kind,
                "tensors": tensors}

    def clip(name, shapes, slices, dtype, kind="l2", max_norm=1.0):
        return {"name": name, "op": "clip", "shapes": shapes, "slices": slices, "dtype": dtype, "kind": kind,
                "max_norm": max_norm}

    def adamw(name, shapes, dtype, max_norm=0.0, step=0, copy=False, matrices=False):
        return {"name": name, "op": "adamw", "shapes": shapes, "slices": 1, "dtype": dtype, "kind": "l2",
                "max_norm": max_norm, "step": step, "copy": copy, "matrices": matrices}

    return [
        # A handful of small tensors: what the launches and the call itself cost.
        norm("norm_tiny", TINY, 4, "f32", tensors=True),
        # Every worker's gradient of a small vision model, logged tensor by tensor.
        norm("norm_resnet18_w16", RESNET18, 16, "f32", tensors=True),
        # Largest entry of each worker's bfloat16 gradient of a language model (overflow watch).
        norm("norm_lstm_w8_bf16_max", LSTM, 8, "bf16", kind="max"),
        # Many odd-sized tensors, from one element upwards, in bfloat16.
        norm("norm_ragged_w3_bf16", RAGGED, 3, "bf16", tensors=True),
        # Clipping of a handful of small tensors.
        clip("clip_tiny_bf16", TINY, 4, "bf16"),
        # Each worker's gradient clipped by its own norm before it is compressed.
        clip("clip_resnet18_w16", RESNET18, 16, "f32"),
        # The same for a language model's bfloat16 gradients.
        clip("clip_lstm_w8_bf16", LSTM, 8, "bf16", max_norm=0.25),
        # The one update of a set of large matrices, clipped as a whole.
        clip("clip_squares", SQUARES, 1, "f32"),
        # First step of a tiny model.
        adamw("adamw_tiny", TINY, "f32", max_norm=1.0),
        # Clipped update of the vision model, decay on its matrices only, bfloat16 weights for the next pass.
        adamw("adamw_resnet18", RESNET18, "f32", max_norm=1.0, step=1000, copy=True, matrices=True),
        # Language model, bfloat16 gradient, no clipping.
        adamw("adamw_lstm_bf16", LSTM, "bf16", step=20000),
        # A large model's clipped update.
        adamw("adamw_squares", SQUARES, "f32", max_norm=1.0, step=5000),
    ]


def draw(rng: random.Random):
    op = rng.choice(["norm", "clip", "adamw"])
    slices = 1 if op == "adamw" else rng.choice([1, 2, 3, 4, 5, 8, 16])
    total = math.exp(rng.uniform(math.log(200), math.log((2e8 if op == "adamw" else 3e8) / slices)))
    count = int(math.exp(rng.uniform(0, math.log(120))))
    weights = [rng.expovariate(1.0) ** 2 + 1e-3 for _ in range(count)]
    sizes = [max(1, int(total * w / sum(weights))) for w in weights]
    rows = [1 if rng.random() < 0.4 else int(math.exp(rng.uniform(0, math.log(n)))) for n in sizes]
    case = {"op": op, "slices": slices, "dtype": rng.choice(["f32", "bf16"]), "kind": rng.choice(["l2", "l2", "max"]),
            "shapes": " ".join(f"{r}x{n // r}" for r, n in zip(rows, sizes))}
    if op == "norm":
        return {**case, "tensors": rng.random() < 0.5}
    if op == "clip":
        return {**case, "max_norm": round(rng.uniform(0.1, 5.0), 3)}
    return {**case, "max_norm": rng.choice([0.0, round(rng.uniform(0.1, 5.0), 3)]),
            "step": rng.choice([0, rng.randrange(1, 100000)]), "copy": rng.random() < 0.5,
            "matrices": rng.random() < 0.5}


LR, BETA1, BETA2, EPS, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01


def _shapes(case):
    parts = [p.partition("*") for p in case["shapes"].split()]
    return [tuple(int(v) for v in p.split("x")) for p, _, n in parts for _ in range(int(n or 1))]


def _parts(case):
    """Elements of each tensor followed by those of its padding, in packed order."""
    sizes = [r * c for r, c in _shapes(case)]
    return [k for n in sizes for k in (n, -n % 64)]


def _spread(values, parts, device):
    """values[i] at every element of tensor i, zero in the padding."""
    v = torch.tensor([x for t in values for x in (t, 0.0)], device=device)
    return torch.repeat_interleave(v, torch.tensor(parts, device=device), output_size=sum(parts))


def prepare(case, seed):
    dev = torch.device("cuda:0")
    rng = random.Random(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    shapes, parts, slices = _shapes(case), _parts(case), case["slices"]
    stride = sum(parts)
    f32 = {"dtype": torch.float32, "device": dev}
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # each tensor has a scale of its own; slice w's norm is about reach[w] times the bound
    scale = [math.exp(rng.gauss(0.0, 1.0)) for _ in shapes]
    whole = math.sqrt(sum(s * s * r * c for s, (r, c) in zip(scale, shapes)))
    reach = [math.exp(rng.uniform(-0.7, 1.0)) * (case.get("max_norm") or 1.0) for _ in range(slices)]
    sigma = _spread([s / whole for s in scale], parts, dev)
    grads = torch.stack([(torch.randn(stride, generator=gen, **f32) * sigma * f).to(dtype) for f in reach])
    s = {"case": case, "parts": parts, "grads": grads, "norms": torch.zeros(slices, **f32)}
    if case["op"] == "norm":
        s["tensor_norms"] = torch.zeros((slices, len(shapes)), **f32) if case["tensors"] else None
    elif case["op"] == "clip":
        s["out"] = torch.zeros_like(grads)
        s["coefs"] = torch.zeros(slices, **f32)
    else:
        s["params"] = torch.randn(stride, generator=gen, **f32) * 0.02 * (sigma > 0)
        seen = 1.0 if case["step"] else 0.0
        s["m"] = torch.randn(stride, generator=gen, **f32) * sigma * (0.3 * seen)
        s["v"] = (torch.rand(stride, generator=gen, **f32) + 0.1) * sigma * sigma * seen
        s["step"] = torch.full((1,), case["step"], dtype=torch.int64, device=dev)
        s["copy"] = torch.zeros(stride, dtype=torch.bfloat16, device=dev) if case["copy"] else None
        s["decay"] = _spread([float(min(sh) > 1 or not case["matrices"]) for sh in shapes], parts, dev)
    if own:
        from distributed_sgd_gradient_ef_amd import psgd

        s["plan"] = psgd.psgd_clip_plan_create(shapes, slices, psgd.PSGD_BF16 if case["dtype"] == "bf16" else psgd.PSGD_F32)
        s["workspace"] = torch.empty(s["plan"].sizes["workspace_bytes"], dtype=torch.uint8, device=dev)
        s["kind"] = psgd.PSGD_NORM_MAX if case["kind"] == "max" else psgd.PSGD_NORM_L2
        if case["op"] == "adamw":
            s["config"] = psgd.AdamwConfig(
                lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, max_norm=case["max_norm"],
                norm_kind=s["kind"], flags=psgd.PSGD_ADAMW_DECAY_MATRICES_ONLY if case["matrices"] else 0)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "clip": _own_clip, "adamw": _own_adamw}[op](state)
    return {"norm": _plain_norm, "clip": _plain_clip, "adamw": _plain_adamw}[op](state)


# ------------------------------------------------------------------ the framework's calls
def _own_norm(s):
    from distributed_sgd_gradient_ef_amd import psgd

    psgd.psgd_grad_norm(s["plan"], s["grads"], s["kind"], s["norms"], s["tensor_norms"], s["workspace"])
    return [s["norms"]] + ([s["tensor_norms"]] if s["tensor_norms"] is not None else [])


def _own_clip(s):
    from distributed_sgd_gradient_ef_amd import psgd

    psgd.psgd_grad_clip(s["plan"], s["grads"], s["out"], s["kind"], s["case"]["max_norm"], s["norms"], s["coefs"],
                        s["workspace"])
    return [s["out"], s["norms"], s["coefs"]]


def _own_adamw(s):
    from distributed_sgd_gradient_ef_amd import psgd

    clipped = s["case"]["max_norm"] > 0
    psgd.psgd_adamw_apply(s["plan"], s["config"], s["grads"], s["params"], s["m"], s["v"], s["copy"], s["step"],
                          s["norms"] if clipped else None, s["workspace"])
    return [s[k] for k in ("params", "m", "v", "step")] + ([s["norms"]] if clipped else []) + \
        ([s["copy"]] if s["copy"] is not None else [])


# ------------------------------------------------------------------ plain forms
def _norms(x, kind):
    """Norm of each row of x (padding is zero, so it adds nothing)."""
    if kind == "max":
        return x.abs().amax(1)
    return (x * x).sum(1, dtype=torch.float64).sqrt().float()


def _plain_norm(s):
    x, kind = s["grads"].float(), s["case"]["kind"]
    if s["tensor_norms"] is None:
        return [_norms(x, kind)]
    parts = torch.stack([_norms(p, kind) for p in x.split(s["parts"], 1)[::2]], 1)
    return [_norms(parts, kind), parts]


def _coefs(norms, max_norm):
    return torch.where(norms <= max_norm, torch.ones_like(norms), max_norm / norms)


def _plain_clip(s):
    x = s["grads"].float()
    norms = _norms(x, s["case"]["kind"])
    coefs = _coefs(norms, s["case"]["max_norm"])
    return [(x * coefs[:, None]).to(s["grads"].dtype), norms, coefs]


def _plain_adamw(s):
    g, case = s["grads"].float(), s["case"]
    norms = []
    if case["max_norm"] > 0:
        norms = [_norms(g, case["kind"])]
        g = g * _coefs(norms[0], case["max_norm"])
    g = g[0]
    x, m, v = s["params"], s["m"], s["v"]
    t = s["step"].add_(1).double()
    m.mul_(BETA1).add_(g, alpha=1 - BETA1)
    v.mul_(BETA2).addcmul_(g, g, value=1 - BETA2)
    rate = (LR / (1 - BETA1 ** t)).float()
    denom = (v * (1 / (1 - BETA2 ** t)).float()).sqrt_().add_(EPS)
    x.sub_(x * s["decay"] * (LR * DECAY)).sub_(m / denom * rate)
    outs = [x, m, v, s["step"]] + norms
    if s["copy"] is not None:
        outs.append(s["copy"].copy_(x))
    return outs


# ------------------------------------------------------------------ bytes, operations, 64-bit results
def work(case):
    slices, tensors = case["slices"], len(_shapes(case))
    n = sum(_parts(case)[::2])
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": slices * (n * e + 4) + (slices * tensors * 4 if case["tensors"] else 0), "flops": 2 * slices * n}
    if case["op"] == "clip":
        return {"bytes": slices * (2 * n * e + 8), "flops": 3 * slices * n}
    return {"bytes": n * (e + 24 + (2 if case["copy"] else 0)) + 16, "flops": 17 * n}


def exact(case, seed):
    s = prepare(case, seed)
    g = s["grads"].double()
    order = math.inf if case["kind"] == "max" else 2
    norms = torch.linalg.vector_norm(g, order, dim=1)
    if case["op"] == "norm":
        if not case["tensors"]:
            return [norms]
        ends = torch.tensor(s["parts"]).cumsum(0).tolist()
        spans = [(end - n, end) for n, end in zip(s["parts"][::2], ends[::2])]
        return [norms, torch.stack([torch.linalg.vector_norm(g[:, a:b], order, dim=1) for a, b in spans], 1)]
    if case["max_norm"] > 0:
        coefs = (case["max_norm"] / norms).clamp(max=1.0)
        g *= coefs[:, None]
    if case["op"] == "clip":
        return [g, norms, coefs]
    g = g[0]
    t = case["step"] + 1
    m = BETA1 * s["m"].double() + (1 - BETA1) * g
    v = BETA2 * s["v"].double() + (1 - BETA2) * g * g
    x = s["params"].double() * (1 - LR * DECAY * s["decay"].double())
    x -= LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    outs = [x, m, v, None] + ([norms] if case["max_norm"] > 0 else [])
    return outs + ([x] if case["copy"] else [])

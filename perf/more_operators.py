"""The losses of a large output layer and the experts' layers, as measured cases.

Kinds of case:

- "entropy": softmax cross entropy of an output layer, logits = x w^T over a vocabulary, from x and w: each row's
  loss, and with "grads" the gradients of x and w, without a matrix of logits;
- "distill": the same for a teacher's top logits: T^2 times the divergence of softmax(x w^T / T) from the softmax of the
  logits / T that the teacher kept;
- "experts_forward" / "experts_backward": linear layers of several experts over rows sorted by expert, ragged:
  y = act(x w_e^T + b_e), and the gradients of x, w and b.

`own` selects how run() computes a case: False, elementary torch operations in 32 bits, rounded once at the end; True,
the calls of ring_all_reduce_ddp_amd.
"""

import math
import random

import torch

own = False

_TORCH = {"fp32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"fp32": 4, "bf16": 2}


def listed():
    return [
        # a step of a small fp32 model's head: latency
        {"name": "entropy_small", "kind": "entropy", "rows": 64, "vocab": 1009, "ins": 96, "dtype": "fp32", "grads": "fp32",
         "accumulate": False, "ignored": 0.1, "pad": 0},
        # the loss of held-out text, without gradients
        {"name": "entropy_eval", "kind": "entropy", "rows": 4096, "vocab": 32000, "ins": 2048, "dtype": "bf16", "grads": "none",
         "accumulate": False, "ignored": 0.0, "pad": 0},
        # odd sizes everywhere, rows that are not 16-byte aligned, half of the tokens a prompt that is not learnt;
        # gradients of the weights' type
        {"name": "entropy_ragged", "kind": "entropy", "rows": 1037, "vocab": 32003, "ins": 1001, "dtype": "bf16", "grads": "bf16",
         "accumulate": False, "ignored": 0.5, "pad": 3},
        # a training micro-batch of 8192 tokens over a large vocabulary, its weight gradient added to the step's fp32 one
        {"name": "entropy_8k_tokens", "kind": "entropy", "rows": 8192, "vocab": 128000, "ins": 4096, "dtype": "bf16", "grads": "fp32",
         "accumulate": True, "ignored": 0.02, "pad": 0},
        # a small student that learns from 8 logits a token
        {"name": "distill_small", "kind": "distill", "rows": 33, "vocab": 1009, "ins": 96, "top": 8, "temperature": 1.0, "dtype": "fp32",
         "grads": "fp32", "accumulate": False, "ignored": 0.1, "pad": 0},
        # a micro-batch of 4096 tokens with the teacher's 64 largest logits each, softened
        {"name": "distill_4k_tokens", "kind": "distill", "rows": 4096, "vocab": 64000, "ins": 2048, "top": 64, "temperature": 2.0,
         "dtype": "bf16", "grads": "bf16", "accumulate": False, "ignored": 0.02, "pad": 0},
        # odd sizes, fp32 gradients, logits cut where the teacher's probability fell below a bound
        {"name": "distill_ragged", "kind": "distill", "rows": 777, "vocab": 32003, "ins": 1000, "top": 101, "temperature": 1.5,
         "dtype": "bf16", "grads": "fp32", "accumulate": True, "ignored": 0.2, "pad": 0},
        # eight tokens of an answer, two experts each: latency and the experts' weights
        {"name": "experts_8_tokens", "kind": "experts_forward", "rows": 16, "behind": 0, "experts": 32, "outs": 4096, "ins": 2048,
         "dtype": "bf16", "act": "silu", "bias": False, "keep": False, "skew": 1.0},
        # 8192 tokens, two experts each, through the experts' first layer; z is kept for the backward pass
        {"name": "experts_forward_8k", "kind": "experts_forward", "rows": 16384, "behind": 0, "experts": 64, "outs": 4096, "ins": 2048,
         "dtype": "bf16", "act": "silu", "bias": False, "keep": True, "skew": 1.0},
        # the second layer's backward pass over those tokens, its input gradient through the activation
        {"name": "experts_backward_8k", "kind": "experts_backward", "rows": 16384, "behind": 0, "experts": 64, "outs": 2048, "ins": 4096,
         "dtype": "bf16", "grads": "fp32", "act": "silu", "bias": True, "skew": 1.0},
        # a small fp32 layer of odd sizes, some experts without a row, a buffer longer than its rows
        {"name": "experts_ragged_fp32", "kind": "experts_forward", "rows": 1501, "behind": 99, "experts": 11, "outs": 517, "ins": 259,
         "dtype": "fp32", "act": "gelu", "bias": True, "keep": True, "skew": 3.0},
        # its gradients in bf16: few rows an expert
        {"name": "experts_backward_ragged", "kind": "experts_backward", "rows": 2203, "behind": 45, "experts": 24, "outs": 520, "ins": 264,
         "dtype": "bf16", "grads": "bf16", "act": "gelu_tanh", "bias": True, "skew": 2.0},
    ]


def _log_size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if rng.random() < 0.5 else n


def draw(rng):
    kind = rng.choice(["entropy", "entropy", "distill", "experts_forward", "experts_backward"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("entropy", "distill"):
        c = {"kind": kind, "rows": _log_size(rng, 1, 8000), "vocab": _log_size(rng, 500, 100_000), "ins": _log_size(rng, 32, 2048),
             "dtype": dtype, "grads": rng.choice([dtype, "fp32"]), "accumulate": rng.random() < 0.5,
             "ignored": rng.choice([0.0, 0.02, 0.5]), "pad": rng.choice([0, 0, 8, 3])}
        if kind == "distill":
            c["top"] = _log_size(rng, 1, 128)
            c["temperature"] = rng.choice([1.0, 2.0, 4.0])
        elif rng.random() < 0.3:
            c["grads"] = "none"
        if c["grads"] != dtype:   # a step's fp32 gradients are sums over its micro-batches
            c["accumulate"] = c["grads"] == "fp32"
        return c
    rows = _log_size(rng, 1, 16000)
    c = {"kind": kind, "rows": rows, "behind": rng.choice([0, 0, rows // 8 + 1]), "experts": _log_size(rng, 1, 96),
         "outs": _log_size(rng, 64, 4096), "ins": _log_size(rng, 64, 2048), "dtype": dtype,
         "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "bias": rng.random() < 0.5, "skew": rng.choice([0.0, 1.0, 3.0])}
    if kind == "experts_forward":
        c["keep"] = rng.random() < 0.5
    else:
        c["grads"] = rng.choice([dtype, "fp32"])
    return c


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device="cuda") * std


def _rows(values, dtype, pad):
    """The values as a matrix whose rows are `pad` elements longer than used."""
    full = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=_TORCH[dtype], device="cuda")
    full[:, :values.shape[1]].copy_(values)
    return full[:, :values.shape[1]]


def _counts(case):
    """Rows of each expert: a router's choices, the k-th most wanted expert's in proportion to k^-skew or so."""
    r = random.Random(1009 * case["rows"] + case["experts"])
    weights = [math.exp(0.3 * r.gauss(0.0, 1.0)) * (1.0 + k * 8.0 / case["experts"]) ** -case["skew"] for k in range(case["experts"])]
    r.shuffle(weights)
    got = [0] * case["experts"]
    for e in r.choices(range(case["experts"]), weights, k=case["rows"]):
        got[e] += 1
    return got


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    if case["kind"].startswith("experts"):
        e, n, k, dt = case["experts"], case["outs"], case["ins"], _TORCH[case["dtype"]]
        total = case["rows"] + case["behind"]
        counts = _counts(case)
        s["offsets"] = torch.tensor([0] + counts).cumsum(0).cuda()
        s["most"] = max(counts)   # an expert's rows at most: what the plain form pads to
        s["x"] = _normal(g, (total, k), 1.0).to(dt)
        s["w"] = _normal(g, (e, n, k), 1.0 / math.sqrt(k)).to(dt)
        if case["kind"] == "experts_forward":
            s["bias"] = _normal(g, (e, n), 0.1).to(dt) if case["bias"] else None
            s["y"] = torch.zeros(total, n, dtype=dt, device="cuda")
            s["z"] = torch.zeros(total, n, dtype=dt, device="cuda") if case["keep"] else None
        else:
            s["dz"] = _normal(g, (total, n), 1e-3).to(dt)
            s["z"] = _normal(g, (total, k), 1.0).to(dt) if case["act"] != "none" else None
            s["dx"] = torch.zeros(total, k, dtype=dt, device="cuda")
            s["dw"] = _normal(g, (e, n, k), 1e-2).to(_TORCH[case["grads"]])
            s["db"] = _normal(g, (e, n), 1e-2).to(_TORCH[case["grads"]]) if case["bias"] else None
        return s
    m, v, k = case["rows"], case["vocab"], case["ins"]
    # logits of deviation 2; where a token is known by now, its own logit stands out
    w = _normal(g, (v, k), 2.0 / math.sqrt(k))
    right = torch.randint(0, v, (m,), generator=g, device="cuda")
    known = torch.rand(m, generator=g, device="cuda") * 10.0 - 4.0
    x = _normal(g, (m, k), 1.0) + w[right] * (known.clamp(min=0) / 2.0)[:, None]
    s["x"], s["w"] = _rows(x, case["dtype"], case["pad"]), _rows(w, case["dtype"], case["pad"])
    ignored = torch.rand(m, generator=g, device="cuda") < case["ignored"]
    if case["kind"] == "entropy":
        s["targets"] = torch.where(ignored, -100, right)
    else:
        c = case["top"]
        # the right token first, the others spread over the vocabulary; logits that fall off as a sorted sample's do
        step = 1 + 2 * (v // (2 * c) // 2)
        ids = (right[:, None] + torch.arange(c, device="cuda")[None, :] * step) % v
        fall = torch.rand(m, c, generator=g, device="cuda").cumsum(1) * (12.0 / c)
        logits = 14.0 + _normal(g, (m, 1), 1.0) - fall
        kept = 1 + (torch.rand(m, generator=g, device="cuda") * c * 1.5).long().clamp(max=c - 1)
        cut = (torch.arange(c, device="cuda")[None, :] >= kept[:, None]) | ignored[:, None]
        s["ids"] = torch.where(cut, -1, ids)
        s["teacher"] = torch.where(cut, -math.inf, logits)
    s["dloss"] = (~ignored).float() / max(1, int((~ignored).sum()))   # of the mean over the rows that count
    if case["grads"] != "none":
        s["dw"] = _normal(g, (v, k), 1.0 / math.sqrt(m * k)).to(_TORCH[case["grads"]])
    return s


# ---------------------------------------------------------------- the plain forms

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros((), device=z.device))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _teacher(s):
    """(ids that may be indexed with, the teacher's probabilities of them): zeros where an entry is cut."""
    ids, t = s["ids"], s["teacher"].float() / s["case"]["temperature"]
    here = (ids >= 0) & (t > -math.inf)
    top = torch.where(here, t, -math.inf).amax(1, keepdim=True).clamp(min=-3e38)
    q = torch.where(here, torch.exp(t - top), 0.0)
    return torch.where(here, ids, 0), q / q.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_loss(s):
    case = s["case"]
    distill = case["kind"] == "distill"
    temperature = case["temperature"] if distill else 1.0
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.t()
    if distill:
        z /= temperature
        ids, q = _teacher(s)
        counted = q.sum(1) > 0
        own_terms = torch.where(q > 0, q * torch.log(q.clamp(min=1e-38)), 0.0)
    else:
        counted = s["targets"] >= 0
        ids = s["targets"].clamp(min=0)[:, None]
        q = counted.float()[:, None]
        own_terms = torch.zeros_like(q)
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    loss = (own_terms - q * (z.gather(1, ids) - lse[:, None])).sum(1) * temperature ** 2
    out = {"loss": torch.where(counted, loss, 0.0), "lse": torch.where(counted, lse, 0.0)}
    if case["grads"] == "none":
        return out
    dz = z.sub_(lse[:, None]).exp_()
    dz.scatter_add_(1, ids, -q)
    dz.mul_(torch.where(counted, s["dloss"] * temperature, 0.0)[:, None])
    out["dx"] = (dz @ w).to(_TORCH[case["dtype"]])
    dw = dz.t() @ x
    s["dw"].copy_(s["dw"].float() + dw if case["accumulate"] else dw)
    out["dw"] = s["dw"]
    return out


def _places(s):
    """For rows in [0, offsets[-1]): their expert and place in it; and for (expert, place): the row and whether there is one."""
    off, total = s["offsets"], s["x"].shape[0]
    row = torch.arange(total, device="cuda")
    expert = (row[:, None] >= off[None, 1:]).sum(1).clamp(max=len(off) - 2)
    place = torch.arange(s["most"], device="cuda")
    at = off[:-1, None] + place[None, :]
    here = at < off[1:, None]
    return expert, row - off[expert], at.clamp(max=total - 1), here, row < off[-1]


def _plain_experts(s):
    case = s["case"]
    dt = _TORCH[case["dtype"]]
    expert, place, at, here, inside = _places(s)
    place = place.clamp(max=s["most"] - 1)
    x = s["x"].float()[at] * here[:, :, None]
    w = s["w"].float()
    if case["kind"] == "experts_forward":
        z = torch.bmm(x, w.transpose(1, 2).contiguous())
        if s["bias"] is not None:
            z += s["bias"].float()[:, None, :]
        z = z[expert, place]
        s["y"].copy_(torch.where(inside[:, None], _act(z, case["act"]).to(dt), s["y"]))
        out = {"y": s["y"]}
        if s["z"] is not None:
            s["z"].copy_(torch.where(inside[:, None], z.to(dt), s["z"]))
            out["z"] = s["z"]
        return out
    dz = s["dz"].float()[at] * here[:, :, None]
    dx = torch.bmm(dz, w)[expert, place]
    if s["z"] is not None:
        dx = dx * _act_slope(s["z"].float(), case["act"])
    s["dx"].copy_(torch.where(inside[:, None], dx.to(dt), s["dx"]))
    s["dw"].copy_(s["dw"].float() + torch.bmm(dz.transpose(1, 2).contiguous(), x))
    out = {"dx": s["dx"], "dw": s["dw"]}
    if s["db"] is not None:
        s["db"].copy_(s["db"].float() + dz.sum(1))
        out["db"] = s["db"]
    return out


# ---------------------------------------------------------------- the framework's calls

def _framework(s):
    import ring_all_reduce_ddp_amd as rar
    case = s["case"]
    kind = case["kind"]
    if kind == "experts_forward":
        rar.experts_forward(s["x"], s["w"], s["offsets"], bias=s["bias"], act=case["act"], out=s["y"], z=s["z"])
        return {"y": s["y"], "z": s["z"]} if case["keep"] else {"y": s["y"]}
    if kind == "experts_backward":
        rar.experts_backward_input(s["dz"], s["w"], s["offsets"], act=case["act"], z=s["z"], out=s["dx"])
        rar.experts_backward_weight(s["dz"], s["x"], s["offsets"], s["dw"], s["db"], accumulate=True)
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]} if case["bias"] else {"dx": s["dx"], "dw": s["dw"]}
    if kind == "entropy":
        loss, lse = rar.cross_entropy_forward(s["x"], s["w"], s["targets"])
        if case["grads"] == "none":
            return {"loss": loss, "lse": lse}
        dx = rar.cross_entropy_backward(s["x"], s["w"], s["targets"], lse, s["dloss"], dw=s["dw"], accumulate=case["accumulate"])
    else:
        loss, lse = rar.distill_forward(s["x"], s["w"], s["ids"], s["teacher"], temperature=case["temperature"])
        dx = rar.distill_backward(s["x"], s["w"], s["ids"], s["teacher"], lse, s["dloss"], temperature=case["temperature"],
                                  dw=s["dw"], accumulate=case["accumulate"])
    return {"loss": loss, "lse": lse, "dx": dx, "dw": s["dw"]}


def run(state):
    if own:
        return _framework(state)
    return _plain_experts(state) if state["case"]["kind"].startswith("experts") else _plain_loss(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    k, e = case["ins"], _BYTES[case["dtype"]]
    if case["kind"].startswith("experts"):
        m, n = case["rows"], case["outs"]
        busy = sum(c > 0 for c in _counts(case))   # experts whose weights are needed
        if case["kind"] == "experts_forward":
            io = m * k + busy * n * (k + case["bias"]) + m * n * (1 + case["keep"])
            return {"bytes": io * e, "flops": 2 * m * n * k}
        io = m * n + busy * n * k + m * k * (2 + (case["act"] != "none"))
        grads = 2 * busy * n * (k + case["bias"]) * _BYTES[case["grads"]]
        return {"bytes": io * e + grads, "flops": 4 * m * n * k}
    # ignored rows take no part; the logits are not kept, so the gradients' pass makes them again
    m, v = max(1, round(case["rows"] * (1 - case["ignored"]))), case["vocab"]
    entries = m * (case["top"] * 12 if case["kind"] == "distill" else 8)
    if case["grads"] == "none":
        return {"bytes": (m * k + v * k) * e + entries + 8 * m, "flops": 2 * m * v * k}
    io = 3 * m * k + 2 * v * k
    grads = v * k * (1 + case["accumulate"]) * _BYTES[case["grads"]]
    return {"bytes": io * e + grads + 2 * entries + 16 * m, "flops": 8 * m * v * k}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_experts(s):
    case = s["case"]
    bounds = s["offsets"].tolist()
    if case["kind"] == "experts_forward":
        y, z = s["y"].double(), torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            t = torch.mm(s["x"][lo:hi].double(), s["w"][e].double().t())
            z[lo:hi] = t if s["bias"] is None else t + s["bias"][e].double()
            y[lo:hi] = _exact_act(z[lo:hi], case["act"])
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    dx, dw = s["dx"].double(), s["dw"].double()
    db = None if s["db"] is None else s["db"].double()
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        dz = s["dz"][lo:hi].double()
        dx[lo:hi] = torch.mm(dz, s["w"][e].double())
        dw[e] += torch.mm(dz.t().contiguous(), s["x"][lo:hi].double())
        if db is not None:
            db[e] += dz.sum(0)
    if s["z"] is not None:
        z = s["z"].double().requires_grad_(True)
        with torch.enable_grad():
            (slope,) = torch.autograd.grad(_exact_act(z, case["act"]).sum(), z)
        dx *= slope
    return {"dx": dx, "dw": dw} if db is None else {"dx": dx, "dw": dw, "db": db}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"].startswith("experts"):
        return _exact_experts(s)
    x, w = s["x"].double(), s["w"].double()
    temperature = case.get("temperature", 1.0)
    z = torch.mm(x, w.t()).div_(temperature)
    lse = torch.logsumexp(z, 1)
    if case["kind"] == "distill":
        log_q = torch.log_softmax(s["teacher"].double() / temperature, 1)   # rows without an entry: NaN
        counted = (s["ids"] >= 0).any(1)
        here = (s["ids"] >= 0) & counted[:, None]
        log_q = torch.where(here, log_q, 0.0)
        q = torch.where(here, log_q.exp(), 0.0)
        ids = torch.where(here, s["ids"], 0)
    else:
        counted = s["targets"] != -100
        ids = torch.where(counted, s["targets"], 0)[:, None]
        log_q, q = torch.zeros_like(ids, dtype=torch.float64), counted.double()[:, None]
    log_p = torch.gather(z, 1, ids) - lse[:, None]
    out = {"loss": temperature ** 2 * (q * (log_q - log_p)).sum(1), "lse": lse * counted}
    if case["grads"] == "none":
        return out
    # the rows' gradients with respect to x w^T
    dz = torch.softmax(z, 1)
    del z
    dz *= counted[:, None]
    dz = torch.scatter_add(dz, 1, ids, -q)
    dz *= (s["dloss"].double() * temperature)[:, None]
    out["dx"] = torch.mm(dz, w)
    dw = torch.mm(dz.t(), x)
    out["dw"] = s["dw"].double() + dw if case["accumulate"] else dw
    return out

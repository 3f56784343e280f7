"""The training-step operators around the gradient sync, as measured cases.

Four kinds of case:

- "norm": the global norm of a model's gradients (many tensors);
- "clip": that norm, and the gradients scaled by min(1, max_norm / (norm + 1e-6)) into the optimizer's gradient buffer;
- "adamw": an AdamW step on fp32 master weights, with the clipping factor taken from the norm on the device;
- "forward" / "backward": a linear layer, y = act(x w^T + b) + r, and its gradients, the weight's and the bias's added
  to the layer's main gradients.

`own` selects how run() computes a case: False, elementary torch operations in 32 bits, rounded once at the end; True,
the calls of ring_all_reduce_ddp_amd.
"""

import math
import random

import torch

own = False

_EPS_CLIP = 1e-6
_TORCH = {"fp32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"fp32": 4, "bf16": 2}
_OPT = {"lr": 1e-3, "b1": 0.9, "b2": 0.95, "eps": 1e-8, "wd": 0.1}


def listed():
    return [
        # a logging or skip decision on a small adapter's gradients: what counts is latency
        {"name": "norm_33_small", "kind": "norm", "tensors": 33, "elements": 20_011, "grads": "fp32", "aligned": False},
        # the norm alone of 1 GiB of gradients, for logging and for the fused step below
        {"name": "norm_1gib", "kind": "norm", "tensors": 290, "elements": 268_435_456, "grads": "fp32", "aligned": True},
        # as many gradients as ResNet-50 has, synced in fp32 and clipped for the optimizer
        {"name": "clip_resnet50", "kind": "clip", "tensors": 161, "elements": 25_557_032, "grads": "fp32", "into": "fp32",
         "aligned": True, "max_norm": 1.0},
        # 300M gradients that came out of a bf16 sync, clipped into the fp32 optimizer's buffer
        {"name": "clip_300m_bf16", "kind": "clip", "tensors": 411, "elements": 300_000_000, "grads": "bf16", "into": "fp32",
         "aligned": True, "max_norm": 1.0},
        # a small adapter's step, packed parameters with odd starts: latency
        {"name": "adamw_33_small", "kind": "adamw", "tensors": 33, "elements": 20_011, "grads": "fp32", "copy": False,
         "aligned": False, "max_norm": 1.0},
        # the fp32 step of a network of ResNet-50's size
        {"name": "adamw_resnet50", "kind": "adamw", "tensors": 161, "elements": 25_557_032, "grads": "fp32", "copy": False,
         "aligned": True, "max_norm": 1.0},
        # a 300M-parameter language model's step: bf16 gradients, fp32 master weights, bf16 weights for the next forward
        {"name": "adamw_300m_bf16", "kind": "adamw", "tensors": 411, "elements": 300_000_000, "grads": "bf16", "copy": True,
         "aligned": True, "max_norm": 1.0},
        # one token through an MLP's first layer while the model answers
        {"name": "forward_1_token", "kind": "forward", "rows": 1, "outs": 8192, "ins": 2048, "dtype": "bf16", "act": "gelu_tanh",
         "bias": True, "residual": False, "keep": False, "pad": 0},
        # a ragged fp32 layer: odd sizes everywhere, rows that are not 16-byte aligned
        {"name": "forward_ragged_fp32", "kind": "forward", "rows": 1037, "outs": 1023, "ins": 2049, "dtype": "fp32", "act": "silu",
         "bias": True, "residual": True, "keep": True, "pad": 0},
        # the first layer of an MLP over a training micro-batch of 8192 tokens; z is kept for the backward pass
        {"name": "forward_8k_tokens", "kind": "forward", "rows": 8192, "outs": 8192, "ins": 2048, "dtype": "bf16", "act": "gelu_tanh",
         "bias": True, "residual": False, "keep": True, "pad": 0},
        # the second layer's backward pass over those tokens: its input gradient passes the activation
        {"name": "backward_8k_tokens", "kind": "backward", "rows": 8192, "outs": 2048, "ins": 8192, "dtype": "bf16", "grads": "fp32",
         "act": "gelu_tanh", "residual": False, "pad": 0},
        # a small layer over a long ragged micro-batch: few output tiles, a long sum
        {"name": "backward_ragged", "kind": "backward", "rows": 5001, "outs": 257, "ins": 640, "dtype": "bf16", "grads": "fp32",
         "act": "none", "residual": True, "pad": 8},
    ]


def _log_size(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if rng.random() < 0.5 else n


def draw(rng):
    kind = rng.choice(["norm", "clip", "adamw", "forward", "forward", "backward", "backward"])
    if kind in ("norm", "clip", "adamw"):
        tensors = _log_size(rng, 1, 500)
        c = {"kind": kind, "tensors": tensors, "elements": max(tensors, _log_size(rng, 1000, 200_000_000)),
             "grads": rng.choice(["fp32", "bf16"]), "aligned": rng.random() < 0.7}
        if kind != "norm":
            c["max_norm"] = rng.choice([1.0, 1.0, 1e5])
        if kind == "clip":
            c["into"] = rng.choice([c["grads"], "fp32"])
        if kind == "adamw":
            c["copy"] = rng.random() < 0.5
        return c
    c = {"kind": kind, "rows": _log_size(rng, 1, 8000), "outs": _log_size(rng, 64, 4096), "ins": _log_size(rng, 64, 4096),
         "dtype": rng.choice(["bf16", "bf16", "fp32"]), "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
         "residual": rng.random() < 0.5, "pad": rng.choice([0, 0, 8, 3])}
    if kind == "forward":
        c["bias"] = rng.random() < 0.7
        c["keep"] = rng.random() < 0.5
    else:
        c["grads"] = rng.choice(["fp32", c["dtype"]])
    return c


# ---------------------------------------------------------------- inputs

def _numels(case):
    """Element counts of the case's tensors: log-uniform weights, as mixed as a network's biases and matrices."""
    n, total = case["tensors"], case["elements"]
    r = random.Random(1009 * total + n)
    w = [math.exp(r.uniform(0.0, 9.0)) for _ in range(n)]
    s = sum(w)
    sizes = [max(1, int(total * x / s)) for x in w]
    sizes[sizes.index(max(sizes))] += total - sum(sizes)
    return sizes


def _offsets(case):
    """Starts of the tensors in one arena, and its length: 16-byte aligned as the planner lays them out, or packed."""
    v = 16 // _BYTES[case["grads"]] if case["aligned"] else 1
    offs, at = [], 0
    for m in _numels(case):
        offs.append(at)
        at += -(-m // v) * v
    return offs, at


def _views(arena, case):
    offs, _ = _offsets(case)
    return [arena[o:o + m] for o, m in zip(offs, _numels(case))]


def _members(case, device):
    """1 for an arena element that belongs to a tensor, 0 for the alignment padding."""
    offs, length = _offsets(case)
    edge = torch.zeros(length + 1, dtype=torch.int32)
    starts = torch.tensor(offs)
    edge.index_add_(0, starts, torch.ones(len(offs), dtype=torch.int32))
    edge.index_add_(0, starts + torch.tensor(_numels(case)), -torch.ones(len(offs), dtype=torch.int32))
    return edge.to(device).cumsum(0)[:length].to(torch.float32)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device="cuda") * std


def _grad_arena(case, g):
    """Gradients N(0, 1e-3) with a heavy tail: 1 % of them a thousand times larger."""
    _, length = _offsets(case)
    x = _normal(g, (length,), 1e-3)
    x.mul_((torch.rand(length, generator=g, device="cuda") < 0.01).to(torch.float32).mul_(999.0).add_(1.0))
    return x.mul_(_members(case, "cuda")).to(_TORCH[case["grads"]])


def _rows(g, rows, cols, std, case):
    """A matrix of the case's type whose rows may be `pad` elements longer than used."""
    full = _normal(g, (rows, cols + case["pad"]), std).to(_TORCH[case["dtype"]])
    return full[:, :cols]


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": dict(case)}
    kind = case["kind"]
    if kind in ("norm", "clip", "adamw"):
        s["grads"] = _grad_arena(case, g)
        s["norm"] = torch.zeros((), device="cuda")
        if kind == "clip":
            s["into"] = torch.zeros(s["grads"].numel(), dtype=_TORCH[case["into"]], device="cuda")
        if kind == "adamw":
            member = _members(case, "cuda")
            length = s["grads"].numel()
            s["params"] = _normal(g, (length,), 0.02) * member
            s["exp_avg"] = _normal(g, (length,), 1e-4) * member
            s["exp_avg_sq"] = _normal(g, (length,), 1e-4).square_() * member
            s["steps"] = torch.full((), 1000 + int(seed) % 1000, dtype=torch.int64, device="cuda")
            s["copy"] = s["params"].to(torch.bfloat16) if case["copy"] else None
            # matrices decay, vectors do not: here the tensors of more than 4096 elements
            s["decays"] = [m > 4096 for m in _numels(case)]
            s["decay"] = torch.repeat_interleave(
                torch.tensor(s["decays"]).to("cuda"), _spans(case)).to(torch.bool)
        if own:
            import ring_all_reduce_ddp_amd as rar
            s["set"] = rar.GradSet(_views(s["grads"], case))
            if kind == "clip":
                s["into_set"] = rar.GradSet(_views(s["into"], case))
            if kind == "adamw":
                s["adamw"] = rar.AdamW(s["set"], _views(s["params"], case), _views(s["exp_avg"], case),
                                       _views(s["exp_avg_sq"], case), s["steps"], decay=s["decays"],
                                       params_bf16=None if s["copy"] is None else _views(s["copy"], case))
        return s
    m, n, k = case["rows"], case["outs"], case["ins"]
    s["x"] = _rows(g, m, k, 1.0, case)
    s["w"] = _rows(g, n, k, 1.0 / math.sqrt(k), case)
    if kind == "forward":
        s["bias"] = _normal(g, (n,), 0.1).to(_TORCH[case["dtype"]]) if case["bias"] else None
        s["residual"] = _rows(g, m, n, 1.0, case) if case["residual"] else None
    else:
        s["dz"] = _rows(g, m, n, 1e-3, case)
        s["z"] = _rows(g, m, k, 1.0, case) if case["act"] != "none" else None
        s["add"] = _rows(g, m, k, 1e-3, case) if case["residual"] else None
        s["dw"] = _normal(g, (n, k), 1e-2).to(_TORCH[case["grads"]])
        s["db"] = _normal(g, (n,), 1e-2).to(_TORCH[case["grads"]])
    return s


def _spans(case):
    """Arena elements from each tensor's start to the next one's."""
    offs, length = _offsets(case)
    return torch.tensor([b - a for a, b in zip(offs, offs[1:] + [length])], device="cuda")


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


def _plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind in ("norm", "clip", "adamw"):
        g = s["grads"].float()
        norm = torch.sqrt((g * g).sum())
        if kind == "norm":
            return {"norm": norm}
        factor = torch.clamp(case["max_norm"] / (norm + _EPS_CLIP), max=1.0)
        if kind == "clip":
            return {"norm": norm, "clipped": (g * factor).to(_TORCH[case["into"]])}
        g = g * factor
        p, m, v, t = s["params"], s["exp_avg"], s["exp_avg_sq"], s["steps"]
        t.add_(1)
        m.mul_(_OPT["b1"]).add_(g, alpha=1.0 - _OPT["b1"])
        v.mul_(_OPT["b2"]).add_(g * g, alpha=1.0 - _OPT["b2"])
        tf = t.float()
        step_size = _OPT["lr"] / (1.0 - _OPT["b1"] ** tf)
        denom = torch.sqrt(v / (1.0 - _OPT["b2"] ** tf)) + _OPT["eps"]
        p.mul_(torch.where(s["decay"], 1.0 - _OPT["lr"] * _OPT["wd"], 1.0))
        p.sub_(step_size * m / denom)
        out = {"norm": norm, "params": p, "exp_avg": m, "exp_avg_sq": v, "steps": t}
        if s["copy"] is not None:
            out["copy"] = p.to(torch.bfloat16)
        return out
    dt = _TORCH[case["dtype"]]
    x, w = s["x"].float(), s["w"].float()
    if kind == "forward":
        z = x @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(dt)}
        if case["keep"]:
            out["z"] = z.to(dt)
        return out
    dz = s["dz"].float()
    dx = dz @ w
    if s["z"] is not None:
        dx = dx * _act_slope(s["z"].float(), case["act"])
    if s["add"] is not None:
        dx = dx + s["add"].float()
    s["dw"].copy_(s["dw"].float() + dz.t() @ x)
    s["db"].copy_(s["db"].float() + dz.sum(0))
    return {"dx": dx.to(dt), "dw": s["dw"], "db": s["db"]}


# ---------------------------------------------------------------- the framework's calls

def _framework(s):
    import ring_all_reduce_ddp_amd as rar
    case = s["case"]
    kind = case["kind"]
    if kind == "norm":
        return {"norm": s["set"].norm(out=s["norm"])}
    if kind == "clip":
        s["set"].norm(out=s["norm"])
        s["set"].clip(case["max_norm"], s["norm"], into=s["into_set"])
        return {"norm": s["norm"], "clipped": s["into"]}
    if kind == "adamw":
        s["set"].norm(out=s["norm"])
        s["adamw"].step(_OPT["lr"], betas=(_OPT["b1"], _OPT["b2"]), eps=_OPT["eps"], weight_decay=_OPT["wd"],
                        max_norm=case["max_norm"], norm=s["norm"])
        out = {"norm": s["norm"], "params": s["params"], "exp_avg": s["exp_avg"], "exp_avg_sq": s["exp_avg_sq"],
               "steps": s["steps"]}
        if s["copy"] is not None:
            out["copy"] = s["copy"]
        return out
    if kind == "forward":
        got = rar.linear_forward(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=case["act"], keep=case["keep"])
        return {"y": got[0], "z": got[1]} if case["keep"] else {"y": got}
    dx = rar.linear_backward_input(s["dz"], s["w"], act=case["act"], z=s["z"], add=s["add"])
    rar.linear_backward_weight(s["dz"], s["x"], s["dw"], s["db"], accumulate=True)
    return {"dx": dx, "dw": s["dw"], "db": s["db"]}


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    kind = case["kind"]
    if kind in ("norm", "clip", "adamw"):
        n, e = case["elements"], _BYTES[case["grads"]]
        if kind == "norm":
            return {"bytes": n * e + 4, "flops": 2 * n}
        if kind == "clip":
            return {"bytes": n * (e + _BYTES[case["into"]]) + 4, "flops": 3 * n}
        return {"bytes": n * (e + 24 + (2 if case["copy"] else 0)) + 20, "flops": 16 * n}
    m, n, k = case["rows"], case["outs"], case["ins"]
    e = _BYTES[case["dtype"]]
    if kind == "forward":
        io = m * k + n * k + m * n * (1 + case["residual"] + case["keep"]) + n * case["bias"]
        return {"bytes": io * e, "flops": 2 * m * n * k}
    io = m * n + n * k + m * k * (2 + case["residual"] + (case["act"] != "none"))
    return {"bytes": io * e + 2 * (n * k + n) * _BYTES[case["grads"]], "flops": 4 * m * n * k + m * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        u = math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3)
        return z * torch.sigmoid(u)
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _exact_product(a, b):
    """a b in 64 bits."""
    return torch.mm(a.double().contiguous(), b.double().contiguous())


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("norm", "clip", "adamw"):
        g = s["grads"].double()
        norm = torch.linalg.vector_norm(g)
        if kind == "norm":
            return {"norm": norm}
        factor = min(1.0, case["max_norm"] / (float(norm) + _EPS_CLIP))
        if kind == "clip":
            return {"norm": norm, "clipped": g * factor}
        t = int(s["steps"]) + 1
        g = g * factor
        m = torch.lerp(g, s["exp_avg"].double(), _OPT["b1"])
        v = torch.lerp(g ** 2, s["exp_avg_sq"].double(), _OPT["b2"])
        p = s["params"].double()
        update = (m / (1 - _OPT["b1"] ** t)) / ((v / (1 - _OPT["b2"] ** t)) ** 0.5 + _OPT["eps"])
        p = p - _OPT["lr"] * (update + _OPT["wd"] * s["decay"] * p)
        out = {"norm": norm, "params": p, "exp_avg": m, "exp_avg_sq": v, "steps": None}
        if s["copy"] is not None:
            out["copy"] = p
        return out
    if kind == "forward":
        z = _exact_product(s["x"], s["w"].t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    dx = _exact_product(s["dz"], s["w"])
    if s["z"] is not None:
        z = s["z"].double().requires_grad_(True)
        with torch.enable_grad():
            (slope,) = torch.autograd.grad(_exact_act(z, case["act"]).sum(), z)
        dx *= slope
    if s["add"] is not None:
        dx += s["add"].double()
    return {"dx": dx, "dw": s["dw"].double() + _exact_product(s["dz"].t(), s["x"]),
            "db": s["db"].double() + s["dz"].double().sum(0)}

"""Cases for the dense operators around the quantized looped linear: a matrix
product with bias, activation and residual in its epilogue, the gated
projection pair of a feed-forward block, each with its backward pass, and the
distillation loss over a teacher's top logits with its gradient.

``own`` selects what ``run`` calls: the plain forms below (elementary torch
operations in float32) or the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")

# the widths of the looped block's linears (2048 -> 5632 -> 2048) and of its
# smallest test problem (256); 49152 and the odd sizes are generic vocabularies


def listed():
    return [
        # one token through a modulation projection of a decode step: bias and
        # activation, latency of one small launch
        {"name": "dense_token", "op": "dense", "M": 1, "N": 2048, "K": 2048, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": False, "save": False},
        # the down projection of a block on a calibration batch, added to the
        # residual stream
        {"name": "dense_down_residual", "op": "dense", "M": 2048, "N": 2048, "K": 5632,
         "dtype": "bf16", "act": "none", "bias": False, "residual": True, "save": False},
        # an output head over an odd vocabulary on a ragged batch
        {"name": "dense_head_odd", "op": "dense", "M": 1003, "N": 49155, "K": 2048,
         "dtype": "f16", "act": "none", "bias": True, "residual": False, "save": False},
        # training step of a projection with an activation: all its gradients
        {"name": "dense_backward", "op": "dense_bwd", "M": 8192, "N": 2048, "K": 2048,
         "dtype": "bf16", "act": "gelu", "bias": True},
        # four tokens of a decode step through gate and up
        {"name": "gated_tokens", "op": "gated", "M": 4, "N": 5632, "K": 2048, "dtype": "bf16",
         "act": "silu", "bias": False, "save": False},
        # a ragged prompt through gate and up
        {"name": "gated_prompt", "op": "gated", "M": 777, "N": 5632, "K": 2048, "dtype": "f16",
         "act": "gelu_tanh", "bias": True, "save": False},
        # a training batch (4 loops x 4096 tokens) through gate and up, with
        # what the backward pass needs kept
        {"name": "gated_train", "op": "gated", "M": 16384, "N": 5632, "K": 2048,
         "dtype": "bf16", "act": "silu", "bias": False, "save": True},
        # all gradients of gate and up on a training batch
        {"name": "gated_backward", "op": "gated_bwd", "M": 8192, "N": 5632, "K": 2048,
         "dtype": "bf16", "act": "silu", "bias": False},
        # the loss alone of a handful of tokens (evaluation of one short sequence)
        {"name": "distill_few", "op": "distill", "M": 4, "V": 49152, "k": 64, "dtype": "f32",
         "tail": False, "grad": False, "temp": 1.0},
        # loss and gradient on one calibration sample of 256 tokens less one,
        # odd vocabulary, the teacher's remaining mass as one class
        {"name": "distill_sample_tail", "op": "distill", "M": 255, "V": 100003, "k": 1000,
         "dtype": "f32", "tail": True, "grad": True, "temp": 2.0},
        # loss and gradient on a calibration batch, teacher's top 1000
        {"name": "distill_batch", "op": "distill", "M": 8192, "V": 49152, "k": 1000,
         "dtype": "bf16", "tail": False, "grad": True, "temp": 1.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("dense", "dense", "dense_bwd", "gated", "gated_bwd", "distill", "distill"))
    if op == "distill":
        V = _log_int(rng, 500, 131072)
        return {"op": op, "M": _log_int(rng, 1, min(8192, 400_000_000 // V)), "V": V,
                "k": _log_int(rng, 1, min(1024, V // 4)),
                "dtype": rng.choice(("bf16", "f16", "f32")), "tail": rng.random() < 0.4,
                "grad": rng.random() < 0.75, "temp": rng.choice((1.0, 1.0, 2.0, 0.5))}
    dtype = rng.choice(("bf16", "bf16", "f16"))
    K = 8 * _log_int(rng, 32, 704)
    N = _log_int(rng, 256, 5632)
    N = N if rng.random() < 0.3 else max(256, N // 64 * 64)
    M = _log_int(rng, 1, 8192)
    if op == "dense" and rng.random() < 0.25:  # an output head
        N, M = _log_int(rng, 8000, 50000), min(M, 512)
    case = {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "bias": rng.random() < 0.5}
    if op in ("gated", "gated_bwd"):
        case["act"] = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu"))
    else:
        case["act"] = rng.choice(ACTS)
    if op in ("dense", "gated"):
        case["save"] = rng.random() < 0.3
    if op == "dense":
        case["residual"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale

    dt = DTYPES[case["dtype"]]
    s = dict(case)
    M = case["M"]
    if case["op"] == "distill":
        V, k = case["V"], case["k"]
        teacher = normal(M, V, scale=3.0)
        s["logits"] = (teacher + normal(M, V, scale=0.7)).to(dt)
        top = torch.topk(teacher, k, dim=1)
        s["t_values"], s["t_index"] = top.values.contiguous(), top.indices.contiguous()
        s["t_lse"] = torch.logsumexp(teacher / case["temp"], 1) if case["tail"] else None
        # rows are averaged; about one in ten is padding and counts nothing
        keep = (torch.rand(M, generator=gen, device="cuda") > 0.1).float()
        keep[0] = 1.0
        s["weight"] = keep / M
        return s
    N, K = case["N"], case["K"]
    x = normal(M, K)
    # a few channels are large, as in a transformer's hidden state
    x[:, torch.randperm(K, generator=gen, device="cuda")[:max(1, K // 50)]] *= 8.0
    s["x"] = x.to(dt)
    scale = 1.0 / math.sqrt(K)
    if case["op"] in ("dense", "dense_bwd"):
        s["w"] = normal(N, K, scale=scale).to(dt)
        s["b"] = normal(N, scale=0.1).to(dt) if case["bias"] else None
        if case["op"] == "dense":
            s["r"] = normal(M, N).to(dt) if case["residual"] else None
        else:
            s["z"] = (s["x"] @ s["w"].T) if case["act"] != "none" else None
            s["dy"] = normal(M, N).to(dt)
    else:
        s["wg"], s["wu"] = normal(N, K, scale=scale).to(dt), normal(N, K, scale=scale).to(dt)
        s["bg"] = normal(N, scale=0.1).to(dt) if case["bias"] else None
        s["bu"] = normal(N, scale=0.1).to(dt) if case["bias"] else None
        if case["op"] == "gated_bwd":
            s["g"], s["u"] = s["x"] @ s["wg"].T, s["x"] @ s["wu"].T
            s["dh"] = normal(M, N).to(dt)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _act(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return sg * (1 + z * (1 - sg))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _project(x, w, b):
    z = x.float() @ w.float().T
    return z if b is None else z + b.float()


def _plain_dense(s):
    z = _project(s["x"], s["w"], s["b"])
    y = _act(s["act"], z)
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(s["x"].dtype)}
    if s["save"]:
        out["z"] = z.to(s["x"].dtype)
    return out


def _plain_dense_bwd(s):
    dt = s["x"].dtype
    dz = s["dy"].float()
    if s["act"] != "none":
        dz = dz * _act_slope(s["act"], s["z"].float())
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.T @ s["x"].float()).to(dt)}
    if s["bias"]:
        out["db"] = dz.sum(0).to(dt)
    return out


def _plain_gated(s):
    dt = s["x"].dtype
    g, u = _project(s["x"], s["wg"], s["bg"]), _project(s["x"], s["wu"], s["bu"])
    out = {"h": (_act(s["act"], g) * u).to(dt)}
    if s["save"]:
        out["g"], out["u"] = g.to(dt), u.to(dt)
    return out


def _plain_gated_bwd(s):
    dt = s["x"].dtype
    g, u, dh, x = s["g"].float(), s["u"].float(), s["dh"].float(), s["x"].float()
    dg = dh * u * _act_slope(s["act"], g)
    du = dh * _act(s["act"], g)
    out = {"dx": (dg @ s["wg"].float() + du @ s["wu"].float()).to(dt),
           "dwg": (dg.T @ x).to(dt), "dwu": (du.T @ x).to(dt)}
    if s["bias"]:
        out["dbg"], out["dbu"] = dg.sum(0).to(dt), du.sum(0).to(dt)
    return out


def _plain_distill(s):
    z = s["logits"].float() / s["temp"]
    # what remains per row and listed entry in float64: the remaining mass
    # 1 - sum(p) and the divergence are small next to the logarithms
    t = s["t_values"].double() / s["temp"]
    idx, w = s["t_index"], s["weight"].unsqueeze(1)
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True).double()
    if s["t_lse"] is None:
        tm = t.amax(1, keepdim=True)
        log_p = t - tm - torch.log(torch.exp(t - tm).sum(1, keepdim=True))
    else:
        log_p = t - s["t_lse"].unsqueeze(1)
    p = torch.exp(log_p)
    log_q = z.gather(1, idx).double() - m - torch.log(total)
    loss = (p * (log_p - log_q)).sum(1, keepdim=True)
    mass = p.sum(1, keepdim=True)
    coef = both = mass
    if s["t_lse"] is not None:
        rest = e.scatter(1, idx, 0.0).sum(1, keepdim=True).double()
        r = torch.clamp(1 - mass, min=0)
        loss = loss + torch.where(r > 0, r * (torch.log(r) - torch.log(rest / total)), 0 * r)
        both = mass + r
        coef = both - r * total / rest
    loss = (loss.float() * w).squeeze(1)
    if not s["grad"]:
        return {"loss": loss}
    q = e / total.float()
    grad = coef.float() * q
    grad = grad.scatter(1, idx, (both * q.gather(1, idx) - p).float())
    return {"loss": loss, "grad": (grad * (w / s["temp"])).to(s["logits"].dtype)}


PLAIN = {"dense": _plain_dense, "dense_bwd": _plain_dense_bwd, "gated": _plain_gated,
         "gated_bwd": _plain_gated_bwd, "distill": _plain_distill}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own(s):
    from bit_ptq_looped_b200 import lq

    op = s["op"]
    if op == "distill":
        got = lq.lq_distill_loss(s["logits"], s["t_values"], s["t_index"], t_lse=s["t_lse"],
                                 weight=s["weight"], temp=s["temp"], want_grad=s["grad"])
        return {"loss": got[0], "grad": got[1]} if s["grad"] else {"loss": got[0]}
    act = lq.LQ_ACTS[s["act"]]
    if op == "dense":
        y, z = lq.lq_dense_linear(s["x"], s["w"], s["b"], act=act, residual=s["r"],
                                  want_z=s["save"])
        return {"y": y, "z": z} if s["save"] else {"y": y}
    if op == "dense_bwd":
        dx, dw, db = lq.lq_dense_linear_bwd(s["dy"], s["x"], s["w"], s["z"], act=act,
                                            want_db=s["bias"])
        return {"dx": dx, "dw": dw, "db": db} if s["bias"] else {"dx": dx, "dw": dw}
    if op == "gated":
        h, g, u = lq.lq_gated_linear(s["x"], s["wg"], s["wu"], s["bg"], s["bu"], act=act,
                                     want_gu=s["save"])
        return {"h": h, "g": g, "u": u} if s["save"] else {"h": h}
    dx, dwg, dwu, dbg, dbu = lq.lq_gated_linear_bwd(s["dh"], s["g"], s["u"], s["x"], s["wg"],
                                                    s["wu"], act=act, want_db=s["bias"])
    out = {"dx": dx, "dwg": dwg, "dwu": dwu}
    return dict(out, dbg=dbg, dbu=dbu) if s["bias"] else out


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    M = case["M"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "distill":
        V, k = case["V"], case["k"]
        rows = M * V * e * (2 if case["grad"] else 1)
        return {"bytes": rows + M * (12 * k + 8 + (4 if case["tail"] else 0)),
                "flops": 4 * M * V}
    N, K, b = case["N"], case["K"], 1 if case["bias"] else 0
    mnk = 2 * M * N * K
    saved = case["act"] != "none"
    if case["op"] == "dense":
        n = M * K + N * K + b * N + M * N * (1 + case["residual"] + case["save"])
        return {"bytes": n * e, "flops": mnk}
    if case["op"] == "dense_bwd":
        return {"bytes": (M * N * (1 + saved) + 2 * M * K + 2 * N * K + b * N) * e,
                "flops": 2 * mnk}
    if case["op"] == "gated":
        return {"bytes": (M * K + 2 * N * K + 2 * b * N + M * N * (1 + 2 * case["save"])) * e,
                "flops": 2 * mnk}
    return {"bytes": (3 * M * N + 2 * M * K + 4 * N * K + 2 * b * N) * e, "flops": 4 * mnk}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _act64(name, z):
    F = torch.nn.functional
    if name == "none":
        return z * 1
    if name == "relu":
        return F.relu(z)
    if name == "silu":
        return F.silu(z)
    return F.gelu(z, approximate="tanh" if name == "gelu_tanh" else "none")


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    F = torch.nn.functional
    op = case["op"]
    if op == "dense":
        z = F.linear(d["x"], d["w"], d.get("b"))
        y = _act64(case["act"], z)
        y = y + d["r"] if case["residual"] else y
        return {"y": y, "z": z} if case["save"] else {"y": y}
    if op == "gated":
        g, u = F.linear(d["x"], d["wg"], d.get("bg")), F.linear(d["x"], d["wu"], d.get("bu"))
        h = _act64(case["act"], g) * u
        return {"h": h, "g": g, "u": u} if case["save"] else {"h": h}
    if op == "dense_bwd":
        dz = d["dy"]
        if case["act"] != "none":
            z = d["z"].requires_grad_()
            dz, = torch.autograd.grad(_act64(case["act"], z), z, d["dy"])
        out = {"dx": F.linear(dz, d["w"].T), "dw": F.linear(dz.T, d["x"].T)}
        return dict(out, db=dz.sum(0)) if case["bias"] else out
    if op == "gated_bwd":
        g, u = d["g"].requires_grad_(), d["u"].requires_grad_()
        dg, du = torch.autograd.grad(_act64(case["act"], g) * u, (g, u), d["dh"])
        out = {"dx": F.linear(dg, d["wg"].T) + F.linear(du, d["wu"].T),
               "dwg": F.linear(dg.T, d["x"].T), "dwu": F.linear(du.T, d["x"].T)}
        return dict(out, dbg=dg.sum(0), dbu=du.sum(0)) if case["bias"] else out
    # distillation: the divergence of two distributions over the listed
    # entries and, with the teacher's log-partition, one class for all others
    z = d["logits"].requires_grad_(case["grad"])
    idx = s["t_index"]
    log_q = F.log_softmax(z / case["temp"], 1)
    top = log_q.gather(1, idx)
    t = d["t_values"] / case["temp"]
    if case["tail"]:
        log_p = t - d["t_lse"].unsqueeze(1)
        r = (1 - log_p.exp().sum(1)).clamp(min=0)
        hidden = torch.zeros_like(log_q, dtype=torch.bool).scatter_(1, idx, True)
        log_rest = torch.logsumexp(log_q.masked_fill(hidden, -math.inf), 1)
        tail = torch.special.xlogy(r, r) - r * log_rest
    else:
        log_p, tail = F.log_softmax(t, 1), 0
    loss = ((log_p.exp() * (log_p - top)).sum(1) + tail) * d["weight"]
    if not case["grad"]:
        return {"loss": loss}
    grad, = torch.autograd.grad(loss.sum(), z)
    return {"loss": loss.detach(), "grad": grad}

"""The operators of a calibration pass through a feed-forward block, as they
are measured: dense sublayer products with their epilogue (linear), the gated
pair of projections (gated), and the distillation loss over a teacher's top
logits (distill), each with its backward pass.

With ``own`` false, ``run`` computes the plain form: elementary torch
operations in 32 bits, rounded once at the end. With ``own`` true it makes the
library calls a user makes. Layouts are the library's: row-major, bf16
matrices whose row strides are multiples of 8 elements (odd widths are views
of wider rows), fp32 biases, losses and weights, int32 indices.
"""
from __future__ import annotations

import math

import torch

own = False

# Shapes: 4096 -> 11008 -> 4096 is the 7B feed-forward block that this
# repository quantizes, 32000 and 128256 are vocabularies of that size of
# model; the ragged cases leave every tile of every kernel partly empty.
LARGEST_FLOPS = 8 * 4096 * 4096 * 11008     # ffn_train's
LARGEST_LOGITS = 4096 * 32000               # distill_step's (elements)


def listed():
    return [
        # one token through a square sublayer (output projection + residual
        # while generating): the smallest call, bound by reading W
        dict(name="linear_token", op="linear", n=1, d_in=4096, d_out=4096, bias=False,
             act="none", residual=True, keep=False),
        # a batch of sequences generating together: down projection + residual
        dict(name="linear_batch", op="linear", n=48, d_in=11008, d_out=4096, bias=False,
             act="none", residual=True, keep=False),
        # a short prompt through a sublayer with bias and activation, sizes
        # off every tile; the pre-activations are kept for a backward pass
        dict(name="linear_ragged", op="linear", n=1021, d_in=1351, d_out=2003, bias=True,
             act="gelu_tanh", residual=False, keep=True),
        # down projection + residual over calibration tokens
        dict(name="linear_prompt", op="linear", n=8192, d_in=11008, d_out=4096, bias=False,
             act="none", residual=True, keep=False),
        # backward pass of a square sublayer with bias and activation: G of
        # the sublayer, bias, input and weight gradients
        dict(name="linear_train", op="linear_bwd", n=4096, d_in=4096, d_out=4096, bias=True,
             act="gelu", residual=False, weights=True),
        # one token through gate and up
        dict(name="ffn_token", op="gated", n=1, d=4096, f=11008, act="silu", keep=False),
        # calibration forward through gate and up, pre-activations kept
        dict(name="ffn_prompt", op="gated", n=4096, d=4096, f=11008, act="silu", keep=True),
        # a ragged prompt through a narrow gated block
        dict(name="ffn_ragged", op="gated", n=333, d=1001, f=2739, act="gelu_tanh", keep=False),
        # calibration backward: G of gate and up, input and weight gradients
        dict(name="ffn_train", op="gated_bwd", n=4096, d=4096, f=11008, act="silu",
             weights=True),
        # loss and gradient of a training step's logits in one call
        dict(name="distill_step", op="distill_step", n=4096, vocab=32000, k=64, dtype="bf16",
             tau=2.0),
        # the same on few rows of fp32 logits of an odd width (no row but the
        # first starts on a 16-byte boundary)
        dict(name="distill_odd", op="distill_step", n=257, vocab=50257, k=17, dtype="f32",
             tau=1.0),
        # evaluation: the loss alone over a wide vocabulary
        dict(name="distill_eval", op="distill_fwd", n=768, vocab=128256, k=100, dtype="bf16",
             tau=1.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd",
                     "distill_step", "distill_fwd", "distill_bwd"])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    if op.startswith("distill"):
        vocab = _log_int(rng, 1000, 128256)
        n = _log_int(rng, 1, min(8192, LARGEST_LOGITS // vocab))
        return dict(op=op, n=n, vocab=vocab, k=_log_int(rng, 1, 128),
                    dtype=rng.choice(["bf16", "f32"]), tau=round(rng.uniform(0.5, 4.0), 3))
    if op.startswith("linear"):
        d_in, d_out = _log_int(rng, 100, 11008), _log_int(rng, 100, 11008)
        flops_row = (4 if op == "linear_bwd" else 2) * d_in * d_out
        n = _log_int(rng, 1, min(16384, LARGEST_FLOPS // flops_row))
        case = dict(op=op, n=n, d_in=d_in, d_out=d_out, bias=rng.random() < 0.5, act=act,
                    residual=rng.random() < 0.5)
        case["weights" if op == "linear_bwd" else "keep"] = rng.random() < 0.5
        return case
    d, f = _log_int(rng, 100, 8192), _log_int(rng, 100, 11008)
    flops_row = (8 if op == "gated_bwd" else 4) * d * f
    n = _log_int(rng, 1, min(16384, LARGEST_FLOPS // flops_row))
    case = dict(op=op, n=n, d=d, f=f, act=act)
    case["weights" if op == "gated_bwd" else "keep"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------- inputs
def _matrix(rows, cols, gen, scale=1.0, per_column=False):
    """rows x cols bf16 values, rows padded to a multiple of 8 elements."""
    ld = (cols + 7) // 8 * 8
    x = torch.randn(rows, ld, generator=gen, device="cuda") * scale
    if per_column:  # channels of activations differ in size
        x = x * torch.exp(torch.rand(ld, generator=gen, device="cuda") * 2 - 1)
    return x.to(torch.bfloat16)[:, :cols]


def _buffer(rows, cols):
    ld = (cols + 7) // 8 * 8
    return torch.zeros(rows, ld, dtype=torch.bfloat16, device="cuda")[:, :cols]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, n = case["op"], case["n"]
    s = {}
    if op.startswith("linear"):
        d_in, d_out = case["d_in"], case["d_out"]
        s["X"] = _matrix(n, d_in, gen, per_column=True)
        s["W"] = _matrix(d_out, d_in, gen, 1.3 / math.sqrt(d_in))
        s["bias"] = (torch.randn(d_out, generator=gen, device="cuda") * 0.3
                     if case["bias"] else None)
        if case["residual"]:  # the residual stream forward, its gradient backward
            s["R"] = _matrix(n, d_in if op == "linear_bwd" else d_out, gen, 2.0)
        if op == "linear_bwd":
            s["dY"] = _matrix(n, d_out, gen, 1e-3, per_column=True)
            s["Z"] = _matrix(n, d_out, gen, 1.3)
    elif op.startswith("gated"):
        d, f = case["d"], case["f"]
        s["X"] = _matrix(n, d, gen, per_column=True)
        s["Wg"] = _matrix(f, d, gen, 1.3 / math.sqrt(d))
        s["Wu"] = _matrix(f, d, gen, 1.3 / math.sqrt(d))
        if op == "gated_bwd":
            s["dH"] = _matrix(n, f, gen, 1e-3, per_column=True)
            s["A"], s["U"] = _matrix(n, f, gen, 1.3), _matrix(n, f, gen, 1.3)
    else:
        vocab, k = case["vocab"], case["k"]
        z = torch.randn(n, vocab, generator=gen, device="cuda") * 2.5
        t = z * 0.9 + torch.randn(n, vocab, generator=gen, device="cuda")
        top = t.topk(k, dim=1)
        s["Z"] = z.to(torch.bfloat16) if case["dtype"] == "bf16" else z
        s["T"] = top.values.contiguous()
        idx = top.indices.to(torch.int32)
        # some rows keep fewer logits than others, some positions do not count
        kept = torch.rand(n, 1, generator=gen, device="cuda") * 1.5 * k + 1
        s["idx"] = torch.where(torch.arange(k, device="cuda") < kept, idx, -1).contiguous()
        counts = (torch.rand(n, generator=gen, device="cuda") < 0.9).float()
        s["weight"] = counts / max(1, n)
        if op == "distill_bwd":
            s["lse"] = torch.logsumexp(s["Z"].double() / case["tau"], 1).float()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, n = case["op"], case["n"]
    if op == "linear":
        s["Y"] = _buffer(n, case["d_out"])
        s["Zout"] = _buffer(n, case["d_out"]) if case["keep"] else None
    elif op == "linear_bwd":
        s["dZ"], s["dX"] = _buffer(n, case["d_out"]), _buffer(n, case["d_in"])
        s["dW"] = _buffer(case["d_out"], case["d_in"]) if case["weights"] else None
        s["db"] = torch.zeros(case["d_out"], device="cuda") if case["bias"] else None
    elif op == "gated":
        s["H"] = _buffer(n, case["f"])
        s["Aout"] = _buffer(n, case["f"]) if case["keep"] else None
        s["Uout"] = _buffer(n, case["f"]) if case["keep"] else None
    elif op == "gated_bwd":
        s["Gg"], s["Gu"] = _buffer(n, case["f"]), _buffer(n, case["f"])
        s["dX"] = _buffer(n, case["d"])
        s["dWg"] = _buffer(case["f"], case["d"]) if case["weights"] else None
        s["dWu"] = _buffer(case["f"], case["d"]) if case["weights"] else None
    else:
        if op != "distill_fwd":
            s["dZ"] = torch.zeros_like(s["Z"])
        if op != "distill_bwd":
            s["loss"] = torch.zeros(n, device="cuda")
            s["lse"] = torch.zeros(n, device="cuda")
    s["info"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["case"] = case
    return s


# ---------------------------------------------------------------- plain form
_SQRT_2_PI = math.sqrt(2 / math.pi)


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(_SQRT_2_PI * (z + 0.044715 * z * z * z)))
    return z


def _dact(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        g = torch.sigmoid(z)
        return g * (1 + z * (1 - g))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z / math.sqrt(2)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(_SQRT_2_PI * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _SQRT_2_PI * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _bf(x):
    return None if x is None else x.to(torch.bfloat16)


def _plain_linear(s, case):
    z = s["X"].float() @ s["W"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(z, case["act"])
    if case["residual"]:
        y = y + s["R"].float()
    return {"Y": _bf(y), "Z": _bf(z) if case["keep"] else None}


def _plain_linear_bwd(s, case):
    dz = s["dY"].float() * _dact(s["Z"].float(), case["act"])
    dx = dz @ s["W"].float()
    if case["residual"]:
        dx = dx + s["R"].float()
    return {"dZ": _bf(dz), "dX": _bf(dx),
            "db": dz.sum(0, dtype=torch.float64).float() if case["bias"] else None,
            "dW": _bf(dz.T @ s["X"].float()) if case["weights"] else None}


def _plain_gated(s, case):
    x = s["X"].float()
    a, u = x @ s["Wg"].float().T, x @ s["Wu"].float().T
    return {"H": _bf(_act(a, case["act"]) * u),
            "A": _bf(a) if case["keep"] else None, "U": _bf(u) if case["keep"] else None}


def _plain_gated_bwd(s, case):
    dh, a, u, x = s["dH"].float(), s["A"].float(), s["U"].float(), s["X"].float()
    gg, gu = dh * u * _dact(a, case["act"]), dh * _act(a, case["act"])
    dx = gg @ s["Wg"].float() + gu @ s["Wu"].float()
    return {"Gg": _bf(gg), "Gu": _bf(gu), "dX": _bf(dx),
            "dWg": _bf(gg.T @ x) if case["weights"] else None,
            "dWu": _bf(gu.T @ x) if case["weights"] else None}


def _plain_distill(s, case):
    tau, op = case["tau"], case["op"]
    kept = s["idx"] >= 0
    idx = torch.where(kept, s["idx"], 0).long()
    t = torch.where(kept, s["T"] / tau, -math.inf)
    lp = t - torch.logsumexp(t.double(), 1, keepdim=True)   # log p, -inf where not kept
    p = torch.where(kept, lp.exp(), 0)
    z = s["Z"].float()
    counts = s["weight"] != 0
    if op == "distill_bwd":
        lse = s["lse"].double()
    else:
        m = z.amax(1, keepdim=True)
        lse = (m[:, 0].double() / tau
               + torch.exp((z - m) / tau).sum(1, dtype=torch.float64).log())
    out = {}
    if op != "distill_bwd":
        lq = z.gather(1, idx).double() / tau - lse[:, None]
        loss = tau * tau * (p * torch.where(kept, lp - lq, 0)).sum(1)
        out["loss"] = torch.where(counts, loss, 0).float()
        out["lse"] = torch.where(counts, lse, 0).float()
    if op != "distill_fwd":
        q = torch.exp((z / tau - lse[:, None].float()))
        q = q.scatter_add_(1, idx, -p.float())
        out["dZ"] = (s["weight"][:, None] * tau * q).to(s["Z"].dtype)
    return out


_PLAIN = {"linear": _plain_linear, "linear_bwd": _plain_linear_bwd, "gated": _plain_gated,
          "gated_bwd": _plain_gated_bwd, "distill_step": _plain_distill,
          "distill_fwd": _plain_distill, "distill_bwd": _plain_distill}


# ---------------------------------------------------------------- the library
def _own_run(s, case):
    from second_order_post_b200 import kronq as K
    op = case["op"]
    if op == "linear":
        K.kronq_linear(s["X"], s["W"], s["Y"], s["info"], bias=s["bias"],
                       act=K.KRONQ_ACTS[case["act"]], Z=s["Zout"], R=s.get("R"))
        return {"Y": s["Y"], "Z": s["Zout"]}
    if op == "linear_bwd":
        K.kronq_linear_bwd(s["dY"], s["X"], s["W"], s["info"], act=K.KRONQ_ACTS[case["act"]],
                           Z=s["Z"], dZ=s["dZ"], db=s["db"], dX=s["dX"], dXr=s.get("R"),
                           dW=s["dW"])
        return {"dZ": s["dZ"], "dX": s["dX"], "db": s["db"], "dW": s["dW"]}
    if op == "gated":
        K.kronq_gated(s["X"], s["Wg"], s["Wu"], s["H"], s["info"],
                      act=K.KRONQ_ACTS[case["act"]], A=s["Aout"], U=s["Uout"])
        return {"H": s["H"], "A": s["Aout"], "U": s["Uout"]}
    if op == "gated_bwd":
        K.kronq_gated_bwd(s["dH"], s["A"], s["U"], s["X"], s["Wg"], s["Wu"], s["Gg"], s["Gu"],
                          s["info"], act=K.KRONQ_ACTS[case["act"]], dX=s["dX"], dWg=s["dWg"],
                          dWu=s["dWu"])
        return {"Gg": s["Gg"], "Gu": s["Gu"], "dX": s["dX"], "dWg": s["dWg"], "dWu": s["dWu"]}
    if op == "distill_step":
        K.kronq_distill_step(s["Z"], s["T"], s["idx"], s["loss"], s["lse"], s["dZ"], s["info"],
                             tau=case["tau"], weight=s["weight"])
        return {"loss": s["loss"], "lse": s["lse"], "dZ": s["dZ"]}
    if op == "distill_fwd":
        K.kronq_distill_fwd(s["Z"], s["T"], s["idx"], s["loss"], s["lse"], s["info"],
                            tau=case["tau"], weight=s["weight"])
        return {"loss": s["loss"], "lse": s["lse"]}
    K.kronq_distill_bwd(s["Z"], s["T"], s["idx"], s["lse"], s["dZ"], s["info"],
                        tau=case["tau"], weight=s["weight"])
    return {"dZ": s["dZ"]}


def run(state):
    case = state["case"]
    if own:
        return _own_run(state, case)
    return _PLAIN[case["op"]](state, case)


# ---------------------------------------------------------------- work, exact
def work(case):
    op, n = case["op"], case["n"]
    if op == "linear":
        i, o = case["d_in"], case["d_out"]
        outs = 1 + case["residual"] + case["keep"]
        return {"bytes": 2 * (n * i + i * o + outs * n * o) + 4 * o * case["bias"],
                "flops": 2 * n * i * o}
    if op == "linear_bwd":
        i, o = case["d_in"], case["d_out"]
        w = case["weights"]
        return {"bytes": 2 * (3 * n * o + n * i * (1 + w + case["residual"]) + i * o * (1 + w))
                + 4 * o * case["bias"],
                "flops": 2 * n * i * o * (1 + w)}
    if op == "gated":
        d, f = case["d"], case["f"]
        return {"bytes": 2 * (n * d + 2 * d * f + n * f * (1 + 2 * case["keep"])),
                "flops": 4 * n * d * f}
    if op == "gated_bwd":
        d, f = case["d"], case["f"]
        w = case["weights"]
        return {"bytes": 2 * (5 * n * f + n * d * (1 + w) + 2 * d * f * (1 + w)),
                "flops": 4 * n * d * f * (1 + w)}
    es = 2 if case["dtype"] == "bf16" else 4
    elems, passes = n * case["vocab"], 1 if op == "distill_fwd" else 2
    # a maximum, an exponential and a sum per logit; the gradient's product
    return {"bytes": passes * es * elems + n * (8 * case["k"] + 12), "flops": 6 * elems}


def _e_act(z, act):
    """(act, its derivative) in 64 bits, from the functions' definitions."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return z * e, e + z * e * (1 - e)
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # 0.5 (1 + tanh(v)) = 1 / (1 + exp(-2 v))
    v = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    e = 1 / (1 + torch.exp(-v))
    dv = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)
    return z * e, e + z * e * (1 - e) * dv


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    d = {k: (v.double() if torch.is_tensor(v) and v.is_floating_point() else v)
         for k, v in s.items()}
    if op == "linear":
        z = d["X"].matmul(d["W"].T)
        z = z if d["bias"] is None else z + d["bias"][None, :]
        y = _e_act(z, case["act"])[0]
        y = y + d["R"] if case["residual"] else y
        return {"Y": y, "Z": z if case["keep"] else None}
    if op == "linear_bwd":
        dz = d["dY"] * _e_act(d["Z"], case["act"])[1]
        dx = dz.matmul(d["W"])
        return {"dZ": dz, "dX": dx + d["R"] if case["residual"] else dx,
                "db": dz.sum(0) if case["bias"] else None,
                "dW": dz.T.matmul(d["X"]) if case["weights"] else None}
    if op == "gated":
        a, u = d["X"].matmul(d["Wg"].T), d["X"].matmul(d["Wu"].T)
        h = _e_act(a, case["act"])[0] * u
        return {"H": h, "A": a if case["keep"] else None, "U": u if case["keep"] else None}
    if op == "gated_bwd":
        h, dh = _e_act(d["A"], case["act"])
        gg, gu = d["dH"] * d["U"] * dh, d["dH"] * h
        w = case["weights"]
        return {"Gg": gg, "Gu": gu, "dX": gg.matmul(d["Wg"]) + gu.matmul(d["Wu"]),
                "dWg": gg.T.matmul(d["X"]) if w else None,
                "dWu": gu.T.matmul(d["X"]) if w else None}
    tau, rows = case["tau"], d["weight"] > 0
    keep = s["idx"] >= 0
    at = s["idx"].clamp_min(0).long()
    e = torch.exp((d["T"] - d["T"].amax(1, keepdim=True)) / tau) * keep
    p = e / e.sum(1, keepdim=True)
    if op == "distill_bwd":
        logq = d["Z"] / tau - d["lse"][:, None]
    else:
        logq = torch.log_softmax(d["Z"] / tau, dim=1)
    out = {}
    if op != "distill_bwd":
        terms = torch.xlogy(p, p) - p * logq.gather(1, at)
        out["loss"] = torch.where(rows, tau ** 2 * terms.sum(1), 0.0)
        out["lse"] = torch.where(rows, d["Z"][:, 0] / tau - logq[:, 0], 0.0)
    if op != "distill_fwd":
        g = torch.exp(logq)
        g.scatter_add_(1, at, -p)
        out["dZ"] = d["weight"][:, None] * tau * g
    return out

"""Measured cases of the state-space-block operators.

The operators are the ones a selective state-space block strings together
around its recurrence: ``linear`` (a matrix product with bias, activation and
residual), ``causal_conv`` / ``causal_conv_step`` (the short depthwise causal
convolution over a prompt and for one token) and ``selective_scan`` /
``selective_step`` (the recurrence over a prompt and for one token).

``listed()`` gives the cases, ``draw()`` more of the same ranges, ``prepare()``
the inputs a program holds before the call, ``run()`` one pass (the plain torch
form in 32 bits, or the library's kernels when ``own`` is set), ``work()`` the
bytes and operations a pass cannot do without, and ``exact()`` the same outputs
from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # input projection of a block over a long packed prompt: width 2048 -> value and gate of 4096
        {"name": "linear_prompt", "op": "linear", "dtype": "bf16", "m": 16384, "k": 2048, "n": 8192,
         "act": "none", "bias": False, "residual": False},
        # output projection with the residual stream added, a ragged number of tokens
        {"name": "linear_ragged", "op": "linear", "dtype": "bf16", "m": 1777, "k": 4096, "n": 2048,
         "act": "none", "bias": True, "residual": True},
        # one decoding step of sixteen sequences through an input projection
        {"name": "linear_tokens", "op": "linear", "dtype": "bf16", "m": 16, "k": 2048, "n": 8192,
         "act": "silu", "bias": True, "residual": False},
        # the step-size projection of a block kept in fp32, an odd number of tokens
        {"name": "linear_f32", "op": "linear", "dtype": "f32", "m": 777, "k": 128, "n": 4096,
         "act": "softplus", "bias": True, "residual": False},
        # the block's convolution over a batch of prompts, reading the value half of the projection
        {"name": "conv_prompt", "op": "conv", "dtype": "bf16", "batch": 4, "n": 8192, "d": 4096, "w": 4,
         "act": "silu", "state": False, "ragged": False},
        # prompts of different lengths continued from an earlier part, fp32, a width off the powers of two
        {"name": "conv_ragged", "op": "conv", "dtype": "f32", "batch": 3, "n": 1501, "d": 1000, "w": 3,
         "act": "silu", "state": True, "ragged": True},
        # one decoding step of the convolution for a full batch
        {"name": "conv_step", "op": "conv_step", "dtype": "bf16", "batch": 256, "d": 4096, "w": 4,
         "act": "silu"},
        # the scan over a batch of prompts with the gate
        {"name": "scan_prompt", "op": "scan", "dtype": "bf16", "batch": 4, "n": 2048, "d": 4096, "s": 16,
         "gate": True, "state": False, "ragged": False},
        # one very long sequence
        {"name": "scan_long", "op": "scan", "dtype": "bf16", "batch": 1, "n": 65536, "d": 2048, "s": 16,
         "gate": True, "state": False, "ragged": False},
        # short fp32 prompts of different lengths continued from a state, wider state, no gate
        {"name": "scan_ragged", "op": "scan", "dtype": "f32", "batch": 7, "n": 333, "d": 520, "s": 32,
         "gate": False, "state": True, "ragged": True},
        # a single sequence's next token: latency
        {"name": "step_single", "op": "step", "dtype": "bf16", "batch": 1, "d": 4096, "s": 16, "gate": True},
        # a full batch's next token: the bandwidth of the state
        {"name": "step_batch", "op": "step", "dtype": "bf16", "batch": 256, "d": 4096, "s": 16, "gate": True},
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / multiple)) * multiple
    v = max(multiple, v)
    return v + multiple if v == 3072 else v


def draw(rng):
    op = rng.choice(["linear", "linear", "conv", "conv_step", "scan", "scan", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear":
        m = _log_int(rng, 1, 16384)
        k = _log_int(rng, 64, 4096, 8)
        n = _log_int(rng, 64, 8192, 8)
        if dtype == "f32":   # 32-bit products stay at the sizes of the small projections
            m, k, n = min(m, 4096), min(k, 2048), min(n, 4096)
        return {"op": op, "dtype": dtype, "m": m, "k": k, "n": n,
                "act": rng.choice(["none", "relu", "silu", "gelu", "softplus"]),
                "bias": rng.random() < 0.6, "residual": rng.random() < 0.5}
    if op == "conv":
        d = _log_int(rng, 64, 4096, 8)
        batch = _log_int(rng, 1, 16)
        n = _log_int(rng, 1, max(2, min(32768, (1 << 27) // (batch * d))))
        return {"op": op, "dtype": dtype, "batch": batch, "n": n, "d": d, "w": rng.choice([2, 3, 4]),
                "act": rng.choice(["silu", "none"]), "state": rng.random() < 0.5,
                "ragged": rng.random() < 0.5}
    if op == "conv_step":
        return {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 256), "d": _log_int(rng, 64, 4096, 8),
                "w": rng.choice([2, 3, 4]), "act": rng.choice(["silu", "none"])}
    s = rng.choice([8, 16, 16, 32, 64])
    d = _log_int(rng, 64, 4096, 8)
    if op == "step":
        return {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 256), "d": d, "s": min(s, 32),
                "gate": rng.random() < 0.7}
    batch = _log_int(rng, 1, 16)
    n = _log_int(rng, 1, max(2, min(65536, (1 << 30) // (batch * d * s))))
    return {"op": op, "dtype": dtype, "batch": batch, "n": n, "d": d, "s": s, "gate": rng.random() < 0.7,
            "state": rng.random() < 0.5, "ragged": rng.random() < 0.5}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        x = torch.empty(*shape, device=dev, dtype=dtype)
        x.normal_(0.0, scale, generator=g)
        return x

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=g)

    st = dict(case)
    op = case["op"]
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        st["x"] = normal(m, k)
        st["weight"] = normal(n, k, scale=k ** -0.5)
        st["bias"] = normal(n, scale=0.5) if case["bias"] else None
        st["residual"] = normal(m, n) if case["residual"] else None
        return st
    B, d = case["batch"], case["d"]
    if op in ("conv", "conv_step"):
        w = case["w"]
        st["weight"] = normal(d, w, scale=w ** -0.5)
        st["bias"] = normal(d, scale=0.2)
        if op == "conv_step":
            st["x"] = normal(B, d)
            st["state"] = normal(B, w - 1, d)
            return st
        # the value half of a projection's output: rows 2·d apart
        st["x"] = normal(B, case["n"], 2 * d)[..., :d]
        st["state"] = normal(B, w - 1, d) if case["state"] else None
        st["lengths"] = _lengths(case, uniform)
        return st
    s = case["s"]
    lead = (B,) if op == "step" else (B, case["n"])
    # value and gate halves of one projection; b and c columns of another, after eight others
    xz = normal(*lead, 2 * d)
    bc = normal(*lead, 8 + 2 * s)
    st["x"], st["gate"] = xz[..., :d], (xz[..., d:] if case["gate"] else None)
    st["b"], st["c"] = bc[..., 8:8 + s], bc[..., 8 + s:]
    st["dt"] = normal(*lead, d, scale=0.5)
    # rates near −1 … −s and initial steps log-uniform in [0.001, 0.1], the usual start of training
    rate = torch.arange(1, s + 1, device=dev, dtype=torch.float32)
    st["a"] = -(rate * torch.exp(0.1 * normal(d, s, dtype=torch.float32))).contiguous()
    step0 = torch.exp(uniform(d) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = (step0 + torch.log(-torch.expm1(-step0))).contiguous()
    st["skip"] = normal(d, dtype=torch.float32)
    if op == "step":
        st["state"] = normal(B, d, s, dtype=torch.float32)
        return st
    st["state"] = normal(B, d, s, dtype=torch.float32) if case["state"] else None
    st["lengths"] = _lengths(case, uniform)
    return st


def _lengths(case, uniform):
    if not case["ragged"]:
        return None
    n = case["n"]
    lens = (uniform(case["batch"]) * (n + 1)).floor().clamp(0, n).to(torch.int32)
    lens[0] = n
    return lens


def run(state):
    op = state["op"]
    if own:
        return _run_own(op, state)
    return {"linear": _plain_linear, "conv": _plain_conv, "conv_step": _plain_conv_step,
            "scan": _plain_scan, "step": _plain_step}[op](state)


def _run_own(op, s):
    import causal_kernelized_linear_gb300 as la
    if op == "linear":
        return la.linear(s["x"], s["weight"], bias=s["bias"], activation=s["act"],
                         residual=s["residual"])
    if op == "conv":
        return la.causal_conv(s["x"], s["weight"], bias=s["bias"], activation=s["act"],
                              state=s["state"], lengths=s["lengths"], return_state=True)
    if op == "conv_step":
        return la.causal_conv_step(s["state"], s["x"], s["weight"], bias=s["bias"],
                                   activation=s["act"]), s["state"]
    if op == "scan":
        return la.selective_scan(s["x"], s["dt"], s["a"], s["b"], s["c"], skip=s["skip"],
                                 gate=s["gate"], dt_bias=s["dt_bias"], softplus=True,
                                 state=s["state"], lengths=s["lengths"], return_state=True)
    return la.selective_step(s["state"], s["x"], s["dt"], s["a"], s["b"], s["c"], skip=s["skip"],
                             gate=s["gate"], dt_bias=s["dt_bias"], softplus=True), s["state"]


# ------------------------------------------------------------------ plain forms, 32 bits

def _activate(x, act):
    if act == "relu":
        return torch.clamp(x, min=0.0)
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "softplus":
        return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))
    return x


def _plain_linear(s):
    y = s["x"].float() @ s["weight"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _activate(y, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _plain_conv(s):
    x, weight = s["x"], s["weight"].float()
    B, n, d = x.shape
    w = weight.shape[1]
    past = s["state"] if s["state"] is not None else x.new_zeros(B, w - 1, d)
    full = torch.cat([past, x], 1)                                     # [B, w - 1 + n, d]
    y = (full.float().unfold(1, w, 1) * weight).sum(-1) + s["bias"].float()
    y = _activate(y, s["act"]).to(x.dtype)
    lens = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), n, device=x.device)
    y = torch.where(torch.arange(n, device=x.device)[None, :, None] < lens[:, None, None], y, 0.0)
    last = lens[:, None] + torch.arange(w - 1, device=x.device)        # the last w − 1 inputs
    return y.to(x.dtype), torch.gather(full, 1, last[..., None].expand(B, w - 1, d))


def _plain_conv_step(s):
    full = torch.cat([s["state"], s["x"][:, None]], 1)                 # [B, w, d]
    y = (full.float() * s["weight"].float().t()).sum(1) + s["bias"].float()
    s["state"].copy_(full[:, 1:])
    return _activate(y, s["act"]).to(s["x"].dtype), s["state"]


def _plain_scan(s):
    x = s["x"].float()
    B, n, d = x.shape
    dt = _activate(s["dt"].float() + s["dt_bias"], "softplus")
    decay = torch.exp(dt[..., None] * s["a"])                          # [B, n, d, s]
    h = (dt * x)[..., None] * s["b"].float()[:, :, None]
    if s["lengths"] is not None:                                       # later tokens leave the state alone
        live = torch.arange(n, device=x.device) < s["lengths"].long()[:, None]
        decay = torch.where(live[..., None, None], decay, 1.0)
        h = torch.where(live[..., None, None], h, 0.0)
    if s["state"] is not None:
        h[:, 0] += decay[:, 0] * s["state"]
    # prefixes by doubling: after the step of width k every token covers 2k tokens
    k = 1
    while k < n:
        h[:, k:] += decay[:, k:] * h[:, :-k].clone()
        decay[:, k:] *= decay[:, :-k].clone()
        k *= 2
    y = (h * s["c"].float()[:, :, None]).sum(-1) + s["skip"] * x
    if s["gate"] is not None:
        y = y * _activate(s["gate"].float(), "silu")
    if s["lengths"] is not None:
        y = torch.where(live[..., None], y, 0.0)
    return y.to(s["x"].dtype), h[:, -1].clone()


def _plain_step(s):
    x = s["x"].float()
    dt = _activate(s["dt"].float() + s["dt_bias"], "softplus")
    h = torch.exp(dt[..., None] * s["a"]) * s["state"] + (dt * x)[..., None] * s["b"].float()[:, None]
    s["state"].copy_(h)
    y = (h * s["c"].float()[:, None]).sum(-1) + s["skip"] * x
    if s["gate"] is not None:
        y = y * _activate(s["gate"].float(), "silu")
    return y.to(s["x"].dtype), s["state"]


# ------------------------------------------------------------------ work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": e * (m * k + n * k + m * n * (2 if case["residual"] else 1)
                              + (n if case["bias"] else 0)),
                "flops": 2.0 * m * n * k}
    B, d = case["batch"], case["d"]
    if op == "conv_step":
        w = case["w"]
        return {"bytes": e * (B * d * (2 + 2 * (w - 1)) + d * (w + 1)), "flops": 2.0 * B * d * w}
    if op == "conv":
        n, w = case["n"], case["w"]
        states = (2 if case["state"] else 1) * B * (w - 1) * d
        return {"bytes": e * (2 * B * n * d + states + d * (w + 1)), "flops": 2.0 * B * n * d * w}
    s = case["s"]
    # per state element: the decay's product and exponential, two for the update, one for the readout
    if op == "step":
        return {"bytes": e * B * (d * (4 if case["gate"] else 3) + 2 * s) + 8 * B * d * s + 4 * d * (s + 2),
                "flops": 7.0 * B * d * s}
    n = case["n"]
    return {"bytes": e * B * n * (d * (4 if case["gate"] else 3) + 2 * s)
            + 4 * B * d * s * (2 if case["state"] else 1) + 4 * d * (s + 2),
            "flops": 7.0 * B * n * d * s}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in st.items()}
    sigmoid = torch.sigmoid
    if op == "linear":
        y = torch.einsum("mk,nk->mn", f["x"], f["weight"])
        if f["bias"] is not None:
            y += f["bias"]
        y = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * sigmoid(v),
             "gelu": lambda v: v * torch.special.ndtr(v),
             "softplus": lambda v: torch.logaddexp(v, torch.zeros_like(v))}[case["act"]](y)
        return y + f["residual"] if f["residual"] is not None else y
    if op == "conv_step":
        y = (f["state"] * f["weight"].t()[None, :-1]).sum(1) + f["x"] * f["weight"][:, -1] + f["bias"]
        y = y * sigmoid(y) if case["act"] == "silu" else y
        return y, torch.cat([f["state"], f["x"][:, None]], 1)[:, 1:]
    if op == "conv":
        B, n, d, w = case["batch"], case["n"], case["d"], case["w"]
        lens = st["lengths"].tolist() if st["lengths"] is not None else [n] * B
        y, last = torch.zeros_like(f["x"]), []
        for i in range(B):
            row = f["x"][i, :lens[i]]
            past = f["state"][i] if f["state"] is not None else row.new_zeros(w - 1, d)
            row = torch.cat([past, row])
            o = f["bias"].expand(lens[i], d).clone()
            for j in range(w):
                o += row[j:j + lens[i]] * f["weight"][:, j]
            y[i, :lens[i]] = o * sigmoid(o) if case["act"] == "silu" else o
            last.append(row[lens[i]:])
        return y, torch.stack(last)
    softplus = torch.logaddexp
    if op == "step":
        x, dt = f["x"], f["dt"] + f["dt_bias"]
        dt = softplus(dt, torch.zeros_like(dt))
        h = f["state"] * torch.exp(dt.unsqueeze(-1) * f["a"])
        h += torch.einsum("bd,bs->bds", dt * x, f["b"])
        y = torch.einsum("bds,bs->bd", h, f["c"]) + f["skip"] * x
        return (y * f["gate"] * sigmoid(f["gate"]) if f["gate"] is not None else y), h
    B, n, d, s = case["batch"], case["n"], case["d"], case["s"]
    h = f["state"].clone() if f["state"] is not None else torch.zeros(B, d, s, device="cuda", dtype=torch.float64)
    dt = f["dt"] + f["dt_bias"]
    dt = softplus(dt, torch.zeros_like(dt))
    if st["lengths"] is not None:   # a step of size zero leaves the state as it is
        dead = torch.arange(n, device="cuda")[None] >= st["lengths"][:, None]
        dt[dead] = 0.0
    u, y = dt * f["x"], torch.empty_like(dt)
    for t in range(n):
        h.mul_(torch.exp(dt[:, t].unsqueeze(-1) * f["a"])).add_(u[:, t].unsqueeze(-1) * f["b"][:, t].unsqueeze(1))
        y[:, t] = torch.matmul(h, f["c"][:, t].unsqueeze(-1)).squeeze(-1)
    y += f["skip"] * f["x"]
    if f["gate"] is not None:
        y *= f["gate"] * sigmoid(f["gate"])
    if st["lengths"] is not None:
        y[dead] = 0.0
    return y, h

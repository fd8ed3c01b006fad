"""Measured cases of the gated-delta block's operators.

The operators are the ones a gated delta-rule block needs beside those of
``perf/operators.py``: ``gated_delta`` / ``gated_delta_step`` (the gated delta
rule over a prompt and for one token), ``rms_norm`` (the norm between blocks,
with the residual's addition, and the gated norm of each head behind the rule,
in 16 bits or in 8 with a scale per token) and ``linear_e4m3`` (the projections
that read those 8 bits).

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
        # a batch of prompts through a block of 32 value heads, two to a query and key head
        {"name": "delta_prompt", "op": "delta", "dtype": "bf16", "batch": 4, "n": 4096, "hk": 16, "hv": 32,
         "dk": 128, "dv": 128, "state": False, "ragged": False},
        # one very long sequence, few heads
        {"name": "delta_long", "op": "delta", "dtype": "bf16", "batch": 1, "n": 65536, "hk": 16, "hv": 16,
         "dk": 128, "dv": 128, "state": False, "ragged": False},
        # short fp32 prompts of different lengths continued from a state, narrower keys
        {"name": "delta_ragged", "op": "delta", "dtype": "f32", "batch": 7, "n": 333, "hk": 4, "hv": 8,
         "dk": 64, "dv": 128, "state": True, "ragged": True},
        # one short prompt, or the part of a conversation that is new: latency
        {"name": "delta_short", "op": "delta", "dtype": "bf16", "batch": 1, "n": 37, "hk": 16, "hv": 32,
         "dk": 128, "dv": 128, "state": True, "ragged": False},
        # a single sequence's next token: latency
        {"name": "delta_step_single", "op": "delta_step", "dtype": "bf16", "batch": 1, "hk": 16, "hv": 32,
         "dk": 128, "dv": 128},
        # a full batch's next token: the bandwidth of the state
        {"name": "delta_step_batch", "op": "delta_step", "dtype": "bf16", "batch": 256, "hk": 16, "hv": 32,
         "dk": 128, "dv": 128},
        # between two blocks: the residual stream added, the norm, and 8 bits for the projection that follows
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "m": 16384, "d": 2048, "group": 2048,
         "gate": False, "residual": True, "quantize": True},
        # behind the rule: the norm of each head of 128, gated by the other half of a projection
        {"name": "norm_heads", "op": "norm", "dtype": "bf16", "m": 8192, "d": 4096, "group": 128,
         "gate": True, "residual": False, "quantize": False},
        # one decoding step of sixteen sequences in fp32, a width off the powers of two
        {"name": "norm_tokens", "op": "norm", "dtype": "f32", "m": 16, "d": 1000, "group": 1000,
         "gate": False, "residual": True, "quantize": False},
        # input projection of a block over a long packed prompt: width 2048 -> value and gate of 4096
        {"name": "linear8_prompt", "op": "linear8", "m": 16384, "k": 2048, "n": 8192, "act": "none",
         "bias": False, "residual": False},
        # output projection with the residual stream added, a ragged number of tokens
        {"name": "linear8_ragged", "op": "linear8", "m": 1777, "k": 4096, "n": 2048, "act": "none",
         "bias": True, "residual": True},
        # one decoding step of sixteen sequences through an input projection
        {"name": "linear8_tokens", "op": "linear8", "m": 16, "k": 2048, "n": 8192, "act": "silu",
         "bias": True, "residual": False},
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / multiple)) * multiple
    return max(multiple, v)


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "delta_step", "norm", "norm", "linear8", "linear8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "linear8":
        return {"op": op, "m": _log_int(rng, 1, 16384), "k": _log_int(rng, 64, 4096, 16),
                "n": _log_int(rng, 64, 8192, 8), "act": rng.choice(["none", "relu", "silu", "gelu", "softplus"]),
                "bias": rng.random() < 0.6, "residual": rng.random() < 0.5}
    if op == "norm":
        group = rng.choice([64, 128, 256, 0, 0, 0])
        heads = _log_int(rng, 1, 32) if group else 1
        group = group or _log_int(rng, 64, 8192, 8)
        d = heads * group
        return {"op": op, "dtype": dtype, "m": _log_int(rng, 1, min(16384, (1 << 26) // d)), "d": d,
                "group": group, "gate": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "quantize": rng.random() < 0.5}
    hk = _log_int(rng, 1, 16)
    case = {"op": op, "dtype": dtype, "batch": 1, "hk": hk, "hv": hk * rng.choice([1, 1, 2, 4]),
            "dk": rng.choice([64, 96, 128, 128]), "dv": rng.choice([64, 128, 128, 192])}
    if op == "delta_step":
        case["batch"] = _log_int(rng, 1, 8192 // case["hv"])
        return case
    case["batch"] = _log_int(rng, 1, 16)
    heads = case["batch"] * case["hv"]
    # in all at most half the head-tokens of the longest listed case, fp32 at most an eighth of those
    case["n"] = _log_int(rng, 1, max(2, min(65536, (1 << (19 if dtype == "bf16" else 16)) // heads)))
    return {**case, "state": rng.random() < 0.5, "ragged": rng.random() < 0.5}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[case.get("dtype", "bf16")]

    def normal(*shape, scale=1.0, dtype=dt):
        x = torch.empty(*shape, device=dev, dtype=dtype)
        x.normal_(0.0, scale, generator=g)
        return x

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=g)

    st = dict(case)
    op = case["op"]
    if op == "linear8":
        m, k, n = case["m"], case["k"], case["n"]
        st["x"], st["x_scale"] = _to_e4m3(normal(m, k, dtype=torch.float32))
        st["weight"], st["weight_scale"] = _to_e4m3(normal(n, k, scale=k ** -0.5, dtype=torch.float32))
        st["bias"] = normal(n, scale=0.5) if case["bias"] else None
        st["residual"] = normal(m, n) if case["residual"] else None
        return st
    if op == "norm":
        m, d = case["m"], case["d"]
        # a few features far larger than the others, as residual streams have them
        st["x"] = normal(m, d) * (1.0 + 8.0 * (uniform(d) < 0.01)).to(dt)
        st["weight"] = (1.0 + normal(case["group"], scale=0.2, dtype=torch.float32)).to(dt)
        st["gate"] = normal(m, 2 * d)[:, d:] if case["gate"] else None   # half of a projection
        st["residual"] = normal(m, d, scale=2.0) if case["residual"] else None
        return st
    B, hk, hv, dk, dv = (case[i] for i in ("batch", "hk", "hv", "dk", "dv"))
    lead = (B,) if op == "delta_step" else (B, case["n"])
    # queries, keys and values side by side as the convolution with silu leaves them
    qkv = normal(*lead, 2 * hk * dk + hv * dv)
    qkv.mul_(torch.sigmoid(qkv))
    q, k, v = qkv.split([hk * dk, hk * dk, hv * dv], -1)
    st["q"], st["k"] = q.unflatten(-1, (hk, dk)), k.unflatten(-1, (hk, dk))
    st["v"] = v.unflatten(-1, (hv, dv))
    # step sizes and writing strengths: two parts of a projection
    db = normal(*lead, 2 * hv)
    st["dt"], st["beta"] = db[..., :hv], db[..., hv:]
    # rates in [-16, -1] and initial steps log-uniform in [0.001, 0.1], the usual start of training
    st["a"] = -(1.0 + 15.0 * uniform(hv))
    step0 = torch.exp(uniform(hv) * math.log(100.0) + math.log(1e-3))
    st["dt_bias"] = step0 + torch.log(-torch.expm1(-step0))
    if op == "delta_step":
        st["state"] = normal(B, hv, dk, dv, scale=0.3, dtype=torch.float32)
        return st
    st["state"] = normal(B, hv, dk, dv, scale=0.3, dtype=torch.float32) if case["state"] else None
    st["lengths"] = None
    if case["ragged"]:
        n = case["n"]
        st["lengths"] = (uniform(B) * (n + 1)).floor().clamp(0, n).to(torch.int32)
        st["lengths"][0] = n
    return st


def run(state):
    op = state["op"]
    if own:
        return _run_own(op, state)
    return {"delta": _plain_delta, "delta_step": _plain_delta_step, "norm": _plain_norm,
            "linear8": _plain_linear8}[op](state)


def _run_own(op, s):
    import causal_kernelized_linear_gb300 as la
    if op == "delta":
        return la.gated_delta(s["q"], s["k"], s["v"], s["dt"], s["a"], s["beta"], dt_bias=s["dt_bias"],
                              state=s["state"], lengths=s["lengths"], return_state=True)
    if op == "delta_step":
        return la.gated_delta_step(s["state"], s["q"], s["k"], s["v"], s["dt"], s["a"], s["beta"],
                                   dt_bias=s["dt_bias"]), s["state"]
    if op == "norm":
        return la.rms_norm(s["x"], s["weight"], gate=s["gate"], residual=s["residual"],
                           quantize=s["quantize"])
    return la.linear_e4m3(s["x"], s["x_scale"], s["weight"], s["weight_scale"], bias=s["bias"],
                          activation=s["act"], residual=s["residual"])


# ------------------------------------------------------------------ plain forms, 32 bits

def _activate(x, act):
    if act == "relu":
        return torch.clamp(x, min=0.0)
    if act == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "softplus":
        return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))
    return x


def _to_e4m3(y):
    """Rows in 8 bits, each with the scale that takes its largest value to 448."""
    scale = y.abs().amax(-1) / 448.0
    scale = torch.where(scale > 0, scale, 1.0)
    return (y / scale[..., None]).to(torch.float8_e4m3fn), scale


def _gates(s):
    """What the rule goes by: unit queries and keys (the query scaled), log decays and writing strengths."""
    q, k = s["q"].float(), s["k"].float()
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + 1e-6) * s["dk"] ** -0.5
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + 1e-6)
    log_decay = s["a"] * _activate(s["dt"].float() + s["dt_bias"], "softplus")
    return q, k, s["v"].float(), log_decay, _activate(s["beta"].float(), "sigmoid")


def _plain_delta(s):
    C = 64
    q, k, v, log_decay, beta = _gates(s)
    B, n, hv = log_decay.shape
    dk, dv = s["dk"], s["dv"]
    live = None
    if s["lengths"] is not None:   # later tokens leave the state alone
        live = torch.arange(n, device=q.device) < s["lengths"].long()[:, None]
        log_decay, beta = log_decay * live[..., None], beta * live[..., None]
    pad = -n % C

    def chunks(x):   # [B, n, h, d] -> [B, hv, chunks, C, d]
        x = x.repeat_interleave(hv // x.shape[2], 2)
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1)
        return x.unflatten(1, (-1, C)).permute(0, 3, 1, 2, 4)

    q, k, v = chunks(q), chunks(k), chunks(v)
    log_decay, beta = chunks(log_decay[..., None])[..., 0], chunks(beta[..., None])
    b = torch.cumsum(log_decay.double(), -1)                           # [B, hv, chunks, C]
    upto = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    pair = torch.exp(torch.where(upto, b[..., :, None] - b[..., None, :], -math.inf).float())
    # T = (1 + A)^-1 of the strictly lower A, by blocks of 1, 2, 4 ...: T21 = -T22 A21 T11
    A = (beta * (k @ k.mT) * pair).tril(-1)
    T = torch.eye(C, device=q.device).expand_as(A).clone()
    w = 1
    while w < C:
        lower = A.unflatten(-1, (-1, 2, w)).unflatten(-4, (-1, 2, w))  # [.., r, 2, w, c, 2, w]
        blocks = T.unflatten(-1, (-1, 2, w)).unflatten(-4, (-1, 2, w))
        i = torch.arange(C // (2 * w), device=q.device)
        at = lambda x, r, c: x[..., i, r, :, i, c, :]                  # noqa: E731  [pairs, .., w, w]
        blocks[..., i, 1, :, i, 0, :] = -(at(blocks, 1, 1) @ at(lower, 1, 0) @ at(blocks, 0, 0))
        T = blocks.flatten(-3).flatten(-4, -2)
        w *= 2
    eb = torch.exp(b.float())[..., None]
    U, W = T @ (beta * v), T @ (beta * eb * k)
    left = torch.exp((b[..., -1:] - b).float())[..., None]             # decay from a token to the chunk's end
    P, qe, kl = (q @ k.mT) * pair, q * eb, k * left
    S = s["state"].clone() if s["state"] is not None else q.new_zeros(B, hv, dk, dv)
    out = torch.empty_like(v)
    for c in range(q.shape[2]):
        new = U[:, :, c] - W[:, :, c] @ S
        out[:, :, c] = qe[:, :, c] @ S + P[:, :, c] @ new
        S = eb[:, :, c, -1:] * S + kl[:, :, c].mT @ new
    out = out.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :n]
    if live is not None:
        out = torch.where(live[..., None, None], out, 0.0)
    return out.to(s["v"].dtype).contiguous(), S


def _plain_delta_step(s):
    q, k, v, log_decay, beta = _gates(s)
    q, k = (x.repeat_interleave(s["hv"] // s["hk"], 1)[:, :, None] for x in (q, k))
    S = torch.exp(log_decay)[..., None, None] * s["state"]
    new = beta[..., None, None] * (v[:, :, None] - k @ S)              # [B, hv, 1, dv]
    S = S + k.mT * new
    s["state"].copy_(S)
    return (q @ S)[:, :, 0].to(s["v"].dtype), s["state"]


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    g = h.unflatten(-1, (-1, s["group"]))
    y = (g * torch.rsqrt((g * g).mean(-1, keepdim=True) + 1e-6) * s["weight"].float()).flatten(-2)
    if s["gate"] is not None:
        y = y * _activate(s["gate"].float(), "silu")
    out = _to_e4m3(y) if s["quantize"] else (y.to(s["x"].dtype),)
    if s["residual"] is not None:
        out += (h.to(s["x"].dtype),)
    return out if len(out) > 1 else out[0]


def _plain_linear8(s):
    y = s["x"].float() @ s["weight"].float().t()
    y = y * s["x_scale"][:, None] * s["weight_scale"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _activate(y, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ work

def work(case):
    e = 2 if case.get("dtype", "bf16") == "bf16" else 4
    op = case["op"]
    if op == "linear8":
        m, k, n = case["m"], case["k"], case["n"]
        return {"bytes": m * k + n * k + 4 * (m + n) + 2 * m * n * (2 if case["residual"] else 1)
                + (2 * n if case["bias"] else 0), "flops": 2.0 * m * n * k}
    if op == "norm":
        m, d = case["m"], case["d"]
        rows = 1 + (1 if case["gate"] else 0) + (2 if case["residual"] else 0)
        out = m * d + 4 * m if case["quantize"] else e * m * d
        return {"bytes": e * m * d * rows + out + e * case["group"], "flops": 4.0 * m * d}
    B, hk, hv, dk, dv = (case[i] for i in ("batch", "hk", "hv", "dk", "dv"))
    n = case.get("n", 1)
    states = 2 if op == "delta_step" or case["state"] else 1
    # per token and head: k·S, the outer product added, q·S, each with a multiply and an add
    return {"bytes": e * B * n * (2 * hk * dk + 2 * hv * dv + 2 * hv) + 4 * states * B * hv * dk * dv + 8 * hv,
            "flops": 6.0 * B * n * hv * dk * dv}


# ------------------------------------------------------------------ 64 bits, from the definitions

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f = {k: (v.double() if isinstance(v, torch.Tensor) else v) for k, v in st.items()}
    if op == "linear8":
        y = torch.einsum("mk,nk->mn", f["x"] * f["x_scale"][:, None], f["weight"] * f["weight_scale"][:, None])
        if f["bias"] is not None:
            y += f["bias"]
        y = {"none": lambda v: v, "relu": torch.relu, "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * torch.special.ndtr(v),
             "softplus": lambda v: torch.logaddexp(v, torch.zeros_like(v))}[case["act"]](y)
        return y + f["residual"] if f["residual"] is not None else y
    if op == "norm":
        h = f["x"] if f["residual"] is None else f["x"] + f["residual"]
        y = torch.empty_like(h)
        for i in range(0, case["d"], case["group"]):
            part = h[:, i:i + case["group"]]
            length = torch.linalg.vector_norm(part, dim=1, keepdim=True)
            y[:, i:i + case["group"]] = part * f["weight"] / torch.sqrt(length ** 2 / case["group"] + 1e-6)
        if f["gate"] is not None:
            y *= f["gate"] * torch.sigmoid(f["gate"])
        out = (y,)
        if case["quantize"]:
            scale = y.abs().max(1).values / 448
            scale[scale == 0] = 1
            out = (y / scale[:, None], scale)
        if f["residual"] is not None:
            out += (h,)
        return out if len(out) > 1 else out[0]
    B, hv, dk, dv = case["batch"], case["hv"], case["dk"], case["dv"]
    step = op == "delta_step"
    if step:
        for name in ("q", "k", "v", "dt", "beta"):
            f[name] = f[name][:, None]
    n = f["v"].shape[1]
    group = torch.arange(hv, device="cuda") // (hv // case["hk"])     # the query and key head of a value head
    unit = lambda x: x / torch.sqrt(torch.einsum("...i,...i->...", x, x) + 1e-6)[..., None]  # noqa: E731
    q, k = unit(f["q"]) / math.sqrt(dk), unit(f["k"])
    decay = torch.exp(f["a"] * torch.logaddexp(f["dt"] + f["dt_bias"], torch.zeros((), device="cuda", dtype=torch.float64)))
    beta = torch.sigmoid(f["beta"])
    S = f["state"].clone() if f["state"] is not None else torch.zeros(B, hv, dk, dv, device="cuda", dtype=torch.float64)
    if not step and st["lengths"] is not None:
        dead = torch.arange(n, device="cuda")[None] >= st["lengths"][:, None]
        decay[dead], beta[dead] = 1.0, 0.0
    S = S.view(B * hv, dk, dv)
    out = torch.empty(n, B * hv, 1, dv, device="cuda", dtype=torch.float64)
    for i0 in range(0, n, 4096):   # heads side by side, for a part of the tokens
        part = slice(i0, min(n, i0 + 4096))
        qt, kt = (x[:, part][:, :, group].transpose(0, 1).reshape(-1, B * hv, 1, dk) for x in (q, k))
        vt = f["v"][:, part].transpose(0, 1).reshape(-1, B * hv, 1, dv)
        at, bt = (x[:, part].transpose(0, 1).reshape(-1, B * hv, 1, 1) for x in (decay, beta))
        for t in range(qt.shape[0]):
            S *= at[t]
            write = torch.baddbmm(vt[t], kt[t], S, alpha=-1.0).mul_(bt[t])
            S.baddbmm_(kt[t].transpose(1, 2), write)
            torch.bmm(qt[t], S, out=out[i0 + t])
    out = out.view(n, B, hv, dv).transpose(0, 1)
    if not step and st["lengths"] is not None:
        out[dead] = 0.0
    return (out[:, 0] if step else out).contiguous(), S.view(B, hv, dk, dv)

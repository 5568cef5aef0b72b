"""What is measured of the dense operators beside the packed experts: the projection with bias, activation and residual
in its epilogue, the norms of queries and keys with their position rotation, and the distillation of a teacher's top
logits, each with its gradients.

Each case is a dict of plain values:
  op "linear"  moe_linear (way "fwd"), moe_linear_grad (way "bwd")
  op "heads"   moe_head_norm (way "fwd"), moe_head_norm_grad (way "bwd")
  op "distill" moe_distill_loss alone (way "fwd"), with the gradient in the same pass (way "step"), or followed by
               moe_distill_loss_grad as a separate backward pass (way "two")
`own` chooses between the plain torch form and the calls of mixed_precision_bit_amd.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token of a served batch of one, through a square projection
        {"name": "linear-one-token", "op": "linear", "way": "fwd", "T": 1, "Kd": 4096, "N": 4096, "dtype": "f16", "y": "f16", "act": "none", "bias": False, "res": False},
        # a decode batch through a shared projection whose fp32 output the requests' adapters are added to
        {"name": "linear-decode", "op": "linear", "way": "fwd", "T": 72, "Kd": 4096, "N": 5120, "dtype": "bf16", "y": "f32", "act": "none", "bias": True, "res": False},
        # a prefill batch through a dense layer's first product, ragged number of tokens
        {"name": "linear-prefill", "op": "linear", "way": "fwd", "T": 4093, "Kd": 2816, "N": 5632, "dtype": "bf16", "y": "bf16", "act": "gelu_tanh", "bias": True, "res": True},
        # a tuning step of a few short sequences
        {"name": "linear-grad-short", "op": "linear", "way": "bwd", "T": 200, "Kd": 2048, "N": 2048, "dtype": "f16", "dy": "f16", "act": "none", "bias": True},
        # the dense layer's backward pass, through its activation
        {"name": "linear-grad-act", "op": "linear", "way": "bwd", "T": 4093, "Kd": 2816, "N": 4096, "dtype": "bf16", "dy": "bf16", "act": "gelu_tanh", "bias": True},
        # a long batch's backward pass of a square projection
        {"name": "linear-grad-long", "op": "linear", "way": "bwd", "T": 8192, "Kd": 4096, "N": 4096, "dtype": "bf16", "dy": "bf16", "act": "none", "bias": True},
        # a decode batch: one far position for each request
        {"name": "heads-decode", "op": "heads", "way": "fwd", "T": 64, "Hq": 16, "Hk": 16, "D": 128, "Dr": 128, "A": 1, "pairs": "halves", "norm": True, "dtype": "f16"},
        # a prefill batch of text and images: positions in time, height and width
        {"name": "heads-prefill", "op": "heads", "way": "fwd", "T": 4093, "Hq": 32, "Hk": 8, "D": 128, "Dr": 128, "A": 3, "pairs": "halves", "norm": True, "dtype": "bf16"},
        # a tuning step's backward pass with wide heads, half of each rotated
        {"name": "heads-grad", "op": "heads", "way": "bwd", "T": 8192, "Hq": 16, "Hk": 8, "D": 256, "Dr": 128, "A": 1, "pairs": "neighbours", "norm": True, "dtype": "bf16"},
        # the loss of a few tokens (a monitor of what lower bitwidths cost), fp32 logits
        {"name": "distill-loss-small", "op": "distill", "way": "fwd", "T": 9, "V": 32003, "k": 20, "rest": False, "dtype": "f32", "masked": False, "tau": 1.0},
        # a tuning step against the stored top logits of the teacher, odd vocabulary
        {"name": "distill-step", "op": "distill", "way": "step", "T": 2048, "V": 151677, "k": 64, "rest": True, "dtype": "bf16", "masked": True, "tau": 2.0},
        # loss and gradient as two passes, the teacher renormalised over its top logits
        {"name": "distill-two", "op": "distill", "way": "two", "T": 1021, "V": 65536, "k": 32, "rest": False, "dtype": "f16", "masked": True, "tau": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "heads", "distill"])
    way = rng.choice(["fwd", "bwd"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "linear":
        c = {"op": op, "way": way, "T": _log(rng, 1, 8000), "Kd": 64 * _log(rng, 1, 64), "N": 8 * _log(rng, 4, 500), "dtype": dtype,
             "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.5}
        more = {"y": rng.choice([dtype, "f32"]), "res": rng.random() < 0.5} if way == "fwd" else {"dy": rng.choice([dtype, "f32"])}
        return c | more
    if op == "heads":
        D = 16 * rng.randint(2, 16)
        return {"op": op, "way": way, "T": _log(rng, 1, 8000), "Hq": rng.randint(1, 32), "Hk": rng.randint(1, 8), "D": D,
                "Dr": 16 * rng.randint(0, D // 16), "A": rng.randint(1, 3), "pairs": rng.choice(["halves", "neighbours"]),
                "norm": rng.random() < 0.8, "dtype": dtype}
    V = _log(rng, 1000, 150000)
    return {"op": op, "way": rng.choice(["fwd", "step", "two"]), "T": _log(rng, 1, min(4000, 200000000 // V)), "V": V,
            "k": _log(rng, 1, 128), "rest": rng.random() < 0.5, "dtype": rng.choice(["f16", "bf16", "f32"]),
            "masked": rng.random() < 0.5, "tau": rng.choice([1.0, 2.0, 4.0])}


# ---------------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def randint(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    dt, T = DT[case["dtype"]], case["T"]
    s = {"case": dict(case)}
    if case["op"] == "linear":
        Kd, N = case["Kd"], case["N"]
        s["X"], s["W"] = randn(T, Kd, dtype=dt), randn(N, Kd, std=Kd ** -0.5, dtype=dt)
        s["bias"] = randn(N, std=0.5) if case["bias"] else None
        if case["way"] == "fwd":
            y = DT[case["y"]]
            s["res"] = randn(T, N, dtype=y) if case["res"] else None
            s |= {"y": empty(T, N, dtype=y), "z": None if case["act"] == "none" else empty(T, N, dtype=dt)}
        else:
            s["z"] = None if case["act"] == "none" else randn(T, N, dtype=dt)     # as the forward pass kept it
            s["dy"] = randn(T, N, std=0.1, dtype=DT[case["dy"]])
            s |= {"dX": empty(T, Kd, dtype=dt), "dW": empty(N, Kd), "dbias": empty(N) if case["bias"] else None}
    elif case["op"] == "heads":
        Hq, Hk, D, Dr, A = case["Hq"], case["Hk"], case["D"], case["Dr"], case["A"]
        qkv = randn(T, Hq + 2 * Hk, D, std=1.5, dtype=dt)     # what the projection of a token's query, key and value heads gave
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        s["g_q"] = 1 + randn(D, std=0.1) if case["norm"] else None
        s["g_k"] = 1 + randn(D, std=0.1) if case["norm"] else None
        # positions up to a long context's, one row an axis
        s["pos"] = randint(0, 1 << 20, A, T) if Dr else None
        s["axis"] = (torch.arange(Dr // 2, device="cuda", dtype=torch.int32) * A // max(1, Dr // 2)).to(torch.int32) if Dr and A > 1 else None
        s["freq"] = (1e6 ** (-torch.arange(Dr // 2, device="cuda", dtype=torch.float64) * 2 / max(1, Dr))).float() if Dr else None
        s |= {"q_out": empty(T, Hq, D, dtype=dt), "k_out": empty(T, Hk, D, dtype=dt)}
        if case["way"] == "bwd":
            s |= {"dq_out": randn(T, Hq, D, dtype=dt), "dk_out": randn(T, Hk, D, dtype=dt)}
            s |= {"dg_q": empty(D) if case["norm"] else None, "dg_k": empty(D) if case["norm"] else None}
    else:
        V, k = case["V"], case["k"]
        S = randn(T, V, std=2.0)
        k = min(k, V)
        step = V // k
        ids = (randint(0, V, T, 1) + torch.arange(k, device="cuda", dtype=torch.int32) * step + randint(0, step, T, k)) % V
        s["ids"] = ids.to(torch.int32).contiguous()           # distinct
        s["teacher"] = (12 - 1.5 * torch.log1p(torch.arange(k, device="cuda").float()) + 0.5 * randn(T, k)).contiguous()
        S.scatter_(1, s["ids"].long(), s["teacher"] + 0.7 * randn(T, k))
        s["S"] = S.to(dt)
        tau = case["tau"]
        # over the teacher's whole vocabulary at this temperature: its top logits hold 0.5 to 0.98 of the probability
        s["t_lse"] = torch.logsumexp(s["teacher"] / tau, 1) - torch.log(0.5 + 0.48 * rand(T)) if case["rest"] else None
        w = torch.ones(T, device="cuda") if not case["masked"] else (rand(T) < 0.9).float()
        s["w"] = w / w.sum().clamp(min=1)                     # 0: padding
        s |= {"stats": empty(T, 4), "kl": empty(T), "loss": empty(1)}
        s["dS"] = None if case["way"] == "fwd" else torch.empty_like(s["S"])
        # fp16 gradients come with a loss scale, as always: those of a mean over a batch are below its range
        s["gloss"] = torch.full((1,), 32768.0, device="cuda") if case["dtype"] == "f16" and case["way"] != "fwd" else None
    return s


# ---------------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    return {"linear": _linear_own if own else _linear, "heads": _heads_own if own else _heads,
            "distill": _distill_own if own else _distill}[c["op"]](s, c)


def _ws(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def _linear_own(s, c):
    import mixed_precision_bit_amd as M
    xd = M.MPB_BF16 if c["dtype"] == "bf16" else M.MPB_F16
    act = {"none": M.MPB_ACT_NONE, "relu": M.MPB_ACT_RELU, "silu": M.MPB_ACT_SILU, "gelu": M.MPB_ACT_GELU,
           "gelu_tanh": M.MPB_ACT_GELU_TANH}[c["act"]]
    T, Kd, N = c["T"], c["Kd"], c["N"]
    if c["way"] == "fwd":
        M.moe_linear(s["X"], xd, s["W"], s["bias"], act, s["res"], s["z"], s["y"], _ws(M.moe_linear_workspace_bytes(T, Kd, N)))
        return {"y": s["y"], "z": s["z"]}
    M.moe_linear_grad(s["X"], xd, s["W"], act, s["z"], s["dy"], s["dX"], s["dW"], s["dbias"],
                      _ws(M.moe_linear_grad_workspace_bytes(T, Kd, N, act, M.MPB_F32 if c["dy"] == "f32" else xd)))
    return {"dX": s["dX"], "dW": s["dW"], "dbias": s["dbias"]}


def _act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = (z > 0).to(z.dtype)
        return z * on, on
    if act == "silu":
        g = torch.sigmoid(z)
        return z * g, g * (1 + z * (1 - g))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a, b = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)


def _linear(s, c):
    dt = DT[c["dtype"]]
    X, W = s["X"].float(), s["W"].float()
    if c["way"] == "fwd":
        z = X @ W.t()
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"])[0]
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(DT[c["y"]]), "z": None if s["z"] is None else z.to(dt)}
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act(s["z"].float(), c["act"])[1]
    return {"dX": (dz @ W).to(dt), "dW": dz.t() @ X, "dbias": dz.sum(0) if c["bias"] else None}


def _heads_own(s, c):
    import mixed_precision_bit_amd as M
    xd = M.MPB_BF16 if c["dtype"] == "bf16" else M.MPB_F16
    pairs = M.MPB_PAIRS_HALVES if c["pairs"] == "halves" else M.MPB_PAIRS_NEIGHBOURS
    rot = (s["pos"], s["axis"], s["freq"], pairs)
    if c["way"] == "fwd":
        M.moe_head_norm(s["q"], s["k"], xd, s["g_q"], s["g_k"], EPS, *rot, s["q_out"], s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    M.moe_head_norm_grad(s["q"], s["k"], xd, s["g_q"], s["g_k"], EPS, *rot, s["dq_out"], s["dk_out"], s["q_out"], s["k_out"],
                         s["dg_q"], s["dg_k"], _ws(M.moe_head_norm_grad_workspace_bytes(c["T"], c["Hq"], c["Hk"], c["D"])))
    return {"dq": s["q_out"], "dk": s["k_out"], "dg_q": s["dg_q"], "dg_k": s["dg_k"]}


def _angles(s, c):
    """cos and sin [T][1][Dr / 2], from 64-bit angles."""
    which = s["axis"].long() if s["axis"] is not None else torch.zeros(c["Dr"] // 2, device="cuda", dtype=torch.long)
    a = s["pos"].double()[which].t() * s["freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _split(v, c):
    Dr = c["Dr"]
    if c["pairs"] == "halves":
        return v[..., :Dr // 2], v[..., Dr // 2:Dr], v[..., Dr:]
    return v[..., 0:Dr:2], v[..., 1:Dr:2], v[..., Dr:]


def _join(a, b, rest, c):
    turned = torch.cat([a, b], -1) if c["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _turn(v, c, cos, sin):
    a, b, rest = _split(v, c)
    return _join(a * cos - b * sin, a * sin + b * cos, rest, c)


def _heads(s, c):
    dt, out = DT[c["dtype"]], {}
    cos, sin = _angles(s, c) if c["Dr"] else (None, None)
    for n in ("q", "k"):
        x, gamma = s[n].float(), s["g_" + n]
        r = torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) if c["norm"] else None
        if c["way"] == "fwd":
            v = x * r * gamma if c["norm"] else x
            out[n] = (_turn(v, c, cos, sin) if c["Dr"] else v).to(dt)
            continue
        d = s["d" + n + "_out"].float()
        d = _turn(d, c, cos, -sin) if c["Dr"] else d
        out["dg_" + n] = None
        if c["norm"]:
            xh = x * r
            out["dg_" + n] = (d * xh).sum((0, 1))
            d = d * gamma
            d = r * (d - xh * (d * xh).mean(2, keepdim=True))
        out["d" + n] = d.to(dt)
    return out if c["way"] == "fwd" else {n: out[n] for n in ("dq", "dk", "dg_q", "dg_k")}


def _distill_own(s, c):
    import mixed_precision_bit_amd as M
    sd = {"f16": M.MPB_F16, "bf16": M.MPB_BF16, "f32": M.MPB_F32}[c["dtype"]]
    dS = s["dS"] if c["way"] == "step" else None
    M.moe_distill_loss(s["S"], sd, s["ids"], s["teacher"], s["t_lse"], s["w"], c["tau"], s["stats"], s["kl"], s["loss"], dS,
                       s["gloss"])
    if c["way"] == "two":
        M.moe_distill_loss_grad(s["S"], sd, s["ids"], s["teacher"], s["t_lse"], s["w"], c["tau"], s["stats"], s["dS"],
                                s["gloss"])
    out = {"loss": s["loss"], "kl": s["kl"]}
    return out if s["dS"] is None else out | {"dS": s["dS"]}


def _distill(s, c):
    tau, ids, w = c["tau"], s["ids"].long(), s["w"][:, None]
    S = s["S"].float() / tau
    logp = S - torch.logsumexp(S, 1, keepdim=True)
    top = logp.gather(1, ids)
    if s["t_lse"] is None:
        logq = torch.log_softmax(s["teacher"] / tau, 1)
    else:
        logq = s["teacher"] / tau - s["t_lse"][:, None]
    q = torch.exp(logq)
    kl = (q * (logq - top)).sum(1)
    if s["t_lse"] is not None:
        q_rest = (1 - q.sum(1)).clamp(min=0)
        log_rest = torch.logsumexp(logp.scatter(1, ids, -math.inf), 1)
        kl = kl + q_rest * (torch.log(q_rest) - log_rest)
    kl = kl * (s["w"] != 0)
    out = {"loss": tau * tau * (s["w"] * kl).sum()[None], "kl": kl}
    if c["way"] != "fwd":
        p, total = torch.exp(logp), q.sum(1, keepdim=True)
        if s["t_lse"] is None:
            d = p * total
        else:
            total = total + q_rest[:, None]
            d = p * (total - (q_rest / torch.exp(log_rest))[:, None])
        d = d.scatter(1, ids, torch.exp(top) * total - q)
        d = tau * w * d
        out["dS"] = (d if s["gloss"] is None else d * s["gloss"]).to(DT[c["dtype"]])
    return out


# ---------------------------------------------------------------------------------------------------- the cost
def work(case):
    T = case["T"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if case["op"] == "linear":
        Kd, N, kept = case["Kd"], case["N"], 0 if case["act"] == "none" else 2 * T * case["N"]
        io = 2 * T * Kd + 2 * N * Kd + kept + (4 * N if case["bias"] else 0)
        if case["way"] == "fwd":
            return {"bytes": io + size[case["y"]] * T * N * (2 if case["res"] else 1), "flops": 2 * T * Kd * N}
        return {"bytes": io + size[case["dy"]] * T * N + 2 * T * Kd + 4 * N * Kd, "flops": 4 * T * Kd * N}
    if case["op"] == "heads":
        rows = 2 * T * (case["Hq"] + case["Hk"]) * case["D"]
        at = 4 * T * case["A"] if case["Dr"] else 0
        if case["way"] == "fwd":
            return {"bytes": 2 * rows + at, "flops": 5 * rows}
        return {"bytes": (3 if case["norm"] else 2) * rows + at, "flops": 8 * rows}
    V, k, b = case["V"], min(case["k"], case["V"]), size[case["dtype"]]
    few = T * (8 * k + 20)
    # the separate backward pass begins after the loss is known: the logits are read again
    passes = {"fwd": 1, "step": 2, "two": 3}[case["way"]]
    return {"bytes": passes * T * V * b + few, "flops": (4 if case["way"] == "fwd" else 8) * T * V}


# ---------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "distill":
        return _distill_exact(s, case)
    f8 = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return (_linear_exact if case["op"] == "linear" else _heads_exact)(f8, case)


def _smooth(z, act):
    """The activation from library functions, differentiable."""
    f = torch.nn.functional
    return {"none": lambda: z * 1, "relu": lambda: f.relu(z), "silu": lambda: f.silu(z), "gelu": lambda: f.gelu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[act]()


def _linear_exact(s, c):
    if c["way"] == "fwd":
        z = torch.nn.functional.linear(s["X"], s["W"], s["bias"])
        y = _smooth(z, c["act"])
        return {"y": y if s["res"] is None else y + s["res"], "z": None if s["z"] is None else z}
    dz = s["dy"]
    if s["z"] is not None:
        z = s["z"].requires_grad_()
        dz = torch.autograd.grad(_smooth(z, c["act"]), z, s["dy"])[0]
    return {"dX": torch.mm(dz, s["W"]), "dW": torch.mm(s["X"].t(), dz).t(), "dbias": dz.t().sum(1) if c["bias"] else None}


def _heads_exact(s, c):
    Dr, out = c["Dr"], {}

    def heads(x, gamma):
        if gamma is not None:
            x = x / (x.pow(2).sum(2, keepdim=True) / c["D"] + EPS).sqrt() * gamma
        if not Dr:
            return x
        axis = [0] * (Dr // 2) if s["axis"] is None else s["axis"].tolist()
        angle = torch.stack([s["pos"][a].double() * f for a, f in zip(axis, s["freq"].tolist())], 1)[:, None]
        unit = torch.polar(torch.ones_like(angle), angle)
        if c["pairs"] == "halves":
            v = torch.complex(x[..., :Dr // 2], x[..., Dr // 2:Dr]) * unit
            return torch.cat([v.real, v.imag, x[..., Dr:]], 2)
        v = torch.view_as_complex(x[..., :Dr].reshape(*x.shape[:2], Dr // 2, 2)) * unit
        return torch.cat([torch.view_as_real(v).flatten(2), x[..., Dr:]], 2)

    if c["way"] == "fwd":
        return {n: heads(s[n], s["g_" + n]) for n in ("q", "k")}
    for n in ("q", "k"):
        leaves = [s[n].clone().requires_grad_()] + ([s["g_" + n].requires_grad_()] if c["norm"] else [None])
        got = torch.autograd.grad(heads(*leaves), [v for v in leaves if v is not None], s["d" + n + "_out"])
        out["d" + n], out["dg_" + n] = got[0], got[1] if c["norm"] else None
    return {n: out[n] for n in ("dq", "dk", "dg_q", "dg_k")}


def _distill_exact(s, c):
    """A few rows at a time: 64-bit logits of the whole batch would not fit beside the rest."""
    T, V, tau = c["T"], c["V"], c["tau"]
    kls, grads, rows = [], [], max(1, (1 << 26) // V)
    for t in range(0, T, rows):
        x = s["S"][t:t + rows].double().requires_grad_()
        ids, y = s["ids"][t:t + rows].long(), s["teacher"][t:t + rows].double() / tau
        w = s["w"][t:t + rows].double()
        logp = torch.log_softmax(x / tau, 1)
        if s["t_lse"] is None:
            q = torch.softmax(y, 1)
            kl = (torch.xlogy(q, q) - q * logp.gather(1, ids)).sum(1)
        else:
            q = torch.exp(y - s["t_lse"][t:t + rows, None].double())
            left = (1 - q.sum(1)).clamp(min=0)
            listed_p = torch.zeros_like(logp, dtype=torch.bool).scatter_(1, ids, True)
            p_left = torch.exp(logp).masked_fill(listed_p, 0).sum(1)
            kl = (torch.xlogy(q, q) - q * logp.gather(1, ids)).sum(1) + torch.xlogy(left, left) - torch.xlogy(left, p_left)
        kl = torch.where(w != 0, kl, 0.0)
        if c["way"] != "fwd":
            up = torch.ones((), device="cuda", dtype=torch.float64) if s["gloss"] is None else s["gloss"].double()[0]
            grads.append(torch.autograd.grad((tau * tau * w * kl).sum(), x, up)[0].to(torch.float32 if T * V > (1 << 27) else torch.float64))
        kls.append(kl.detach())
    kl = torch.cat(kls)
    out = {"loss": tau * tau * (s["w"].double() * kl).sum()[None], "kl": kl}
    return out if c["way"] == "fwd" else out | {"dS": torch.cat(grads)}

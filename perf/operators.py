"""What is measured of the operators that stand around the packed experts of a MoE block: the norms before and
after the block with its gate and residual scale, the router's balance and z loss with its gradients, and the
low-rank adapters of many requests.

Each case is a dict of plain values:
  op "norm"     moe_block_norm (way "fwd"), moe_block_norm_grad (way "bwd")
  op "router"   moe_router_loss (way "fwd"), both that and moe_router_loss_grad (way "step")
  op "adapters" moe_adapters
`own` chooses between the plain torch form and the calls of mixed_precision_bit_amd.
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one token of a served batch of one: the gated block output joins the residual, and the next block's norm
        {"name": "norm-one-token", "op": "norm", "way": "fwd", "T": 1, "H": 2048, "dtype": "f16", "gate": "token", "post": True},
        # a decode batch between two blocks, without a post norm or gate
        {"name": "norm-decode", "op": "norm", "way": "fwd", "T": 128, "H": 4096, "dtype": "f16", "gate": "none", "post": False},
        # a prefill batch with the norm after the block, and an elementwise gate
        {"name": "norm-prefill", "op": "norm", "way": "fwd", "T": 4096, "H": 2816, "dtype": "bf16", "gate": "full", "post": True},
        # a tuning step's backward pass, ragged number of tokens
        {"name": "norm-grad", "op": "norm", "way": "bwd", "T": 4093, "H": 2816, "dtype": "bf16", "gate": "token", "post": True},
        {"name": "norm-grad-long", "op": "norm", "way": "bwd", "T": 8192, "H": 4096, "dtype": "bf16", "gate": "full", "post": True},
        # the smallest tuning step: a few tokens, a few of them padding
        {"name": "router-step-small", "op": "router", "way": "step", "T": 72, "H": 2048, "E": 60, "K": 4, "dtype": "f16", "masked": True, "gw": True},
        # the loss alone over a prefill-size batch (a monitor of the balance)
        {"name": "router-loss", "op": "router", "way": "fwd", "T": 4096, "H": 2816, "E": 128, "K": 8, "dtype": "bf16", "masked": False, "gw": False},
        # tuning steps over padded batches, with and without a gradient of the routing weights
        {"name": "router-step", "op": "router", "way": "step", "T": 4096, "H": 2816, "E": 128, "K": 8, "dtype": "bf16", "masked": True, "gw": False},
        {"name": "router-step-long", "op": "router", "way": "step", "T": 16381, "H": 4096, "E": 128, "K": 8, "dtype": "bf16", "masked": True, "gw": True},
        # one token of one request
        {"name": "adapters-one-token", "op": "adapters", "T": 1, "Kd": 2048, "N": 2048, "n": 4, "R": 16, "dtype": "f16", "mixed": False, "runs": False},
        # a decode batch in which nearly every token brings its own adapter
        {"name": "adapters-decode", "op": "adapters", "T": 128, "Kd": 4096, "N": 4096, "n": 64, "R": 32, "dtype": "bf16", "mixed": True, "runs": False},
        # a prefill batch: runs of tokens of one request each
        {"name": "adapters-prefill", "op": "adapters", "T": 4093, "Kd": 2816, "N": 2816, "n": 16, "R": 64, "dtype": "bf16", "mixed": True, "runs": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "router", "adapters"])
    dtype = rng.choice(["f16", "bf16"])
    H = 64 * _log(rng, 4, 64)
    if op == "norm":
        return {"op": op, "way": rng.choice(["fwd", "bwd"]), "T": _log(rng, 1, 8192), "H": H, "dtype": dtype,
                "gate": rng.choice(["none", "token", "full"]), "post": rng.random() < 0.7}
    if op == "router":
        E = _log(rng, 2, 128)
        return {"op": op, "way": rng.choice(["fwd", "step"]), "T": _log(rng, 1, 16000), "H": H, "E": E,
                "K": rng.randint(1, min(E, 8)), "dtype": dtype, "masked": rng.random() < 0.5, "gw": rng.random() < 0.5}
    return {"op": op, "T": _log(rng, 1, 4000), "Kd": H, "N": 64 * _log(rng, 4, 64), "n": _log(rng, 1, 32),
            "R": rng.choice([8, 16, 32, 64]), "dtype": dtype, "mixed": rng.random() < 0.5, "runs": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    dt, T = DT[case["dtype"]], case["T"]
    s = {"case": dict(case)}
    if case["op"] == "norm":
        H = case["H"]
        s["o"] = randn(T, H, std=0.3)                       # the block's output, fp32 as moe_ffn writes it
        s["r"] = randn(T, H, std=1.5, dtype=dt)             # the residual stream before (fwd) or after (bwd) the block
        s["gate"] = {"none": None, "token": randn(T), "full": randn(T, H, dtype=dt)}[case["gate"]]
        s["g_post"] = 1 + randn(H, std=0.1) if case["post"] else None
        s["g_next"] = 1 + randn(H, std=0.1)
        s["scale"] = 0.7
        if case["way"] == "fwd":
            s |= {"r_out": empty(T, H, dtype=dt), "x": empty(T, H, dtype=dt)}
        else:
            s |= {"dr_out": randn(T, H, dtype=dt), "dx": randn(T, H, dtype=dt)}
            s |= {"dr": empty(T, H, dtype=dt), "do": empty(T, H), "dg_next": empty(H)}
            s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
            s["dg_post"] = empty(H) if case["post"] else None
    elif case["op"] == "router":
        H, E, K = case["H"], case["E"], case["K"]
        s["X"] = randn(T, H, dtype=dt)
        s["W"] = randn(E, H, std=H ** -0.5)
        s["bias"] = -0.5 * torch.log1p(torch.randperm(E, generator=g, device="cuda").float())  # some experts run hot
        logits = s["X"].float() @ s["W"].t() + s["bias"]
        s["idx"] = torch.topk(logits, K, dim=1).indices.to(torch.int32).contiguous()   # as moe_route gives them
        s["mask"] = (rand(T) < 0.9).to(torch.uint8) if case["masked"] else None         # 0: padding
        s["alpha"], s["beta"] = 0.01, 0.001
        s["gw"] = randn(T, K, std=0.01 / T) if case["gw"] else None
        s |= {"logits": empty(T, E), "lse": empty(T), "counts": empty(E + 1, dtype=torch.int32), "prob": empty(E), "loss": empty(3)}
        if case["way"] == "step":
            s |= {"dX": empty(T, H), "dW": empty(E, H), "dbias": empty(E)}
    else:
        Kd, N, n, R = case["Kd"], case["N"], case["n"], case["R"]
        s["X"] = randn(T, Kd, dtype=dt)
        s["A"] = randn(n, R, Kd, std=Kd ** -0.5, dtype=dt)
        s["B"] = randn(n, N, R, std=R ** -0.5, dtype=dt)
        s["ranks"] = torch.randint(1, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if case["mixed"] \
            else torch.full((n,), R, device="cuda", dtype=torch.int32)
        s["scales"] = 0.5 + rand(n)
        adapter = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)  # -1: a request without one
        s["adapter"] = torch.sort(adapter).values.contiguous() if case["runs"] else adapter
        s["base"] = randn(T, N)                             # what the shared projection gave
        s["out"] = empty(T, N)
    return s


# ---------------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    return {"norm": _norm_own if own else _norm, "router": _router_own if own else _router,
            "adapters": _adapters_own if own else _adapters}[c["op"]](s, c)


def _norm_own(s, c):
    import mixed_precision_bit_amd as M
    xd = M.MPB_BF16 if c["dtype"] == "bf16" else M.MPB_F16
    if c["way"] == "fwd":
        M.moe_block_norm(s["o"], s["r"], xd, s["gate"], s["g_post"], s["g_next"], s["scale"], EPS, s["r_out"], s["x"])
        return {"r": s["r_out"], "x": s["x"]}
    ws = torch.empty(M.moe_block_norm_grad_workspace_bytes(c["T"], c["H"]), dtype=torch.uint8, device="cuda")
    M.moe_block_norm_grad(s["o"], s["r"], xd, s["gate"], s["g_post"], s["g_next"], s["scale"], EPS, s["dr_out"], s["dx"],
                          s["dr"], s["do"], s["dgate"], s["dg_post"], s["dg_next"], ws)
    return {"dr": s["dr"], "do": s["do"], "dgate": s["dgate"], "dg_post": s["dg_post"], "dg_next": s["dg_next"]}


def _rms(v):
    return torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)


def _norm(s, c):
    dt, k = DT[c["dtype"]], s["scale"]
    o, r = s["o"], s["r"].float()
    gate = None if s["gate"] is None else torch.sigmoid(s["gate"].float())
    if gate is not None and gate.dim() == 1:
        gate = gate[:, None]
    oh = o * _rms(o) if c["post"] else o
    u = oh * s["g_post"] if c["post"] else o
    if c["way"] == "fwd":
        y = r + k * (u if gate is None else gate * u)
        return {"r": y.to(dt), "x": (y * _rms(y) * s["g_next"]).to(dt)}
    # backward: r holds the stream after the block, y
    dx, ry = s["dx"].float(), _rms(r)
    yh, d = r * ry, dx * s["g_next"]
    dy = s["dr_out"].float() + ry * (d - yh * (d * yh).mean(1, keepdim=True))
    dv = k * dy
    dgate = None
    if gate is not None:
        dgate = dv * u * gate * (1 - gate)
        dgate = (dgate.sum(1) if s["gate"].dim() == 1 else dgate).to(s["gate"].dtype)
        dv = dv * gate
    dg_post = None
    if c["post"]:
        dg_post = (dv * oh).sum(0)
        d = dv * s["g_post"]
        dv = _rms(o) * (d - oh * (d * oh).mean(1, keepdim=True))
    return {"dr": dy.to(dt), "do": dv, "dgate": dgate, "dg_post": dg_post, "dg_next": (dx * yh).sum(0)}


def _router_own(s, c):
    import mixed_precision_bit_amd as M
    xd = M.MPB_BF16 if c["dtype"] == "bf16" else M.MPB_F16
    ws = torch.empty(M.moe_router_loss_workspace_bytes(c["T"], c["H"], c["E"]), dtype=torch.uint8, device="cuda")
    M.moe_router_loss(s["X"], xd, s["W"], s["bias"], s["idx"], s["mask"], s["alpha"], s["beta"], s["logits"], s["lse"],
                      s["counts"], s["prob"], s["loss"], ws)
    out = {"logits": s["logits"], "lse": s["lse"], "counts": s["counts"], "prob": s["prob"], "loss": s["loss"]}
    if c["way"] == "step":
        M.moe_router_loss_grad(s["X"], xd, s["W"], s["idx"], s["mask"], s["logits"], s["lse"], s["counts"], s["alpha"],
                               s["beta"], s["gw"], None, s["dX"], s["dW"], s["dbias"], ws)
        out |= {"dX": s["dX"], "dW": s["dW"], "dbias": s["dbias"]}
    return out


def _router(s, c):
    X, W, E, K = s["X"].float(), s["W"], c["E"], c["K"]
    T, idx = c["T"], s["idx"].long()
    live = torch.ones(T, 1, device="cuda") if s["mask"] is None else (s["mask"] != 0).float()[:, None]
    X = torch.where(live != 0, X, 0.0)
    logits = (X @ W.t() + s["bias"]) * live             # padding: zeros
    lse = torch.logsumexp(logits, 1, keepdim=True) * live
    p = torch.exp(logits - lse) * live
    counts = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
    counts.index_add_(0, idx.flatten(), live.to(torch.int32).expand(T, K).reshape(-1))
    n_int = live.to(torch.int32).sum()
    counts[E:] = n_int
    n = n_int.float().clamp(min=1)
    f, prob = counts[:E].float() / (K * n), p.sum(0)
    balance, z = E * (f * prob).sum() / n, (lse * lse).sum() / n
    out = {"logits": logits, "lse": lse[:, 0], "counts": counts, "prob": prob,
           "loss": torch.stack([s["alpha"] * balance + s["beta"] * z, balance, z])}
    if c["way"] == "step":
        a = s["alpha"] * E / n * (f - (p * f).sum(1, keepdim=True))
        dl = p * (a + 2 * s["beta"] / n * lse)
        if s["gw"] is not None:
            w = torch.softmax(logits.gather(1, idx), 1)
            gw = s["gw"]
            dl = dl.scatter_add(1, idx, live * w * (gw - (w * gw).sum(1, keepdim=True)))
        out |= {"dX": dl @ W, "dW": dl.t() @ X, "dbias": dl.sum(0)}
    return out


def _adapters_own(s, c):
    import mixed_precision_bit_amd as M
    xd = M.MPB_BF16 if c["dtype"] == "bf16" else M.MPB_F16
    ws = torch.empty(M.moe_adapters_workspace_bytes(c["T"], c["Kd"], c["n"], c["R"]), dtype=torch.uint8, device="cuda")
    M.moe_adapters(s["X"], xd, s["A"], s["B"], s["ranks"], s["scales"], s["adapter"], s["base"], s["out"], ws)
    return s["out"]


def _adapters(s, c):
    n, R, Kd, N = c["n"], c["R"], c["Kd"], c["N"]
    # every adapter's product for every token, the other adapters' and those past the rank masked
    z = (s["X"].float() @ s["A"].float().reshape(n * R, Kd).t()).reshape(-1, n, R)
    mine = s["adapter"][:, None] == torch.arange(n, device="cuda")
    low = torch.arange(R, device="cuda") < s["ranks"][:, None]
    z = torch.where(mine[:, :, None] & low, z * s["scales"][:, None], 0.0)
    return s["base"] + z.reshape(-1, n * R) @ s["B"].float().transpose(1, 2).reshape(n * R, N)


# ---------------------------------------------------------------------------------------------------- the cost
def work(case):
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        gate = {"none": 0, "token": 4 * T, "full": 2 * T * H}[case["gate"]]
        vec = 4 * H * (2 if case["post"] else 1)
        if case["way"] == "fwd":        # o, r, gate in; r, x out
            return {"bytes": T * H * (4 + 2 + 2 + 2) + gate + vec, "flops": 10 * T * H}
        o = 4 if case["gate"] != "none" or case["post"] else 0   # o is needed for the gate's and the norm's gradients
        return {"bytes": T * H * (o + 2 + 2 + 2 + 2 + 4) + 2 * gate + 2 * vec, "flops": 30 * T * H}
    if case["op"] == "router":
        H, E, K = case["H"], case["E"], case["K"]
        fwd = 2 * T * H + 4 * E * H + 4 * T * K + 4 * T * E + 4 * T
        flops = 2 * T * H * E
        if case["way"] == "fwd":
            return {"bytes": fwd, "flops": flops}
        return {"bytes": fwd + (4 * T * K if case["gw"] else 0) + 4 * T * H + 4 * E * H, "flops": 3 * flops}
    Kd, N, n, R = case["Kd"], case["N"], case["n"], case["R"]
    rank = (R + 1) / 2 if case["mixed"] else R
    used = n * (1 - (1 - 1 / (n + 1)) ** T)               # adapters that some token brings
    return {"bytes": 2 * T * Kd + 2 * used * rank * (Kd + N) + 8 * T * N,
            "flops": 2 * T * (n / (n + 1)) * rank * (Kd + N)}


# ---------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f8 = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return {"norm": _norm_exact, "router": _router_exact, "adapters": _adapters_exact}[case["op"]](f8, case)


def _unit_rows(v):
    return v / (v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt()


def _norm_exact(s, c):
    gate = s["gate"]

    def added(o, gate, g_post):
        v = _unit_rows(o) * g_post if c["post"] else o
        if gate is not None:
            v = v / (1 + torch.exp(-(gate.unsqueeze(1) if gate.dim() == 1 else gate)))
        return s["scale"] * v

    if c["way"] == "fwd":
        y = s["r"] + added(s["o"], gate, s["g_post"])
        return {"r": y, "x": _unit_rows(y) * s["g_next"]}
    leaf = {k: s[k].requires_grad_() for k in ("r", "o", "gate", "g_post", "g_next") if s[k] is not None}
    # the stream's gradient first (r is the stream after the block), then what the block adds receives it
    gr, gn = torch.autograd.grad((_unit_rows(leaf["r"]) * leaf["g_next"] * s["dx"]).sum(), [leaf["r"], leaf["g_next"]])
    dy = s["dr_out"] + gr
    names = [k for k in ("o", "gate", "g_post") if k in leaf]
    got = dict(zip(names, torch.autograd.grad((added(leaf["o"], leaf.get("gate"), leaf.get("g_post")) * dy).sum(),
                                              [leaf[k] for k in names])))
    return {"dr": dy, "do": got["o"], "dgate": got.get("gate"), "dg_post": got.get("g_post"), "dg_next": gn}


def _router_exact(s, c):
    E, K, T = c["E"], c["K"], c["T"]
    keep = torch.arange(T, device="cuda") if s["mask"] is None else s["mask"].nonzero()[:, 0]
    n = max(1, len(keep))
    X, W, b = s["X"][keep].requires_grad_(), s["W"].requires_grad_(), s["bias"].requires_grad_()
    idx = s["idx"].long()[keep]
    l = torch.addmm(b, X, W.t())
    m = l.detach().amax(1, keepdim=True) if len(keep) else 0.0
    ex = (l - m).exp()
    lse = (ex.sum(1).log() + m[:, 0]) if len(keep) else l.sum(1)
    p = ex / ex.sum(1, keepdim=True)
    hist = torch.bincount(idx.flatten(), minlength=E)[:E].double()
    prob = p.sum(0)
    balance = E * torch.dot(hist / (K * n), prob / n)
    z = lse.square().sum() / n
    total = s["alpha"] * balance + s["beta"] * z

    def whole(v, *shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda").index_copy(0, keep, v.detach())

    out = {"logits": whole(l, T, E), "lse": whole(lse, T), "counts": torch.cat([hist, torch.tensor([len(keep)], device="cuda")]).int(),
           "prob": prob.detach(), "loss": torch.stack([total, balance, z]).detach()}
    if c["way"] == "step":
        if s["gw"] is not None:
            w = p.gather(1, idx)
            total = total + (w / w.sum(1, keepdim=True) * s["gw"][keep]).sum()
        dX, dW, db = torch.autograd.grad(total, [X, W, b])
        out |= {"dX": whole(dX, T, c["H"]), "dW": dW, "dbias": db}
    return out


def _adapters_exact(s, c):
    out = s["base"].clone()
    for a, rank in enumerate(s["ranks"].tolist()):
        rows = (s["adapter"] == a).nonzero()[:, 0]
        low = s["A"][a, :rank] @ s["X"][rows].t()
        out[rows] += s["scales"][a] * (s["B"][a, :, :rank] @ low).t()
    return out

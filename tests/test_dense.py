"""The dense operators as they are used together: the projection of a block's normed stream to query, key and value
heads with its requests' adapters, the heads' norms and rotation; an output head, the distillation of its logits and
the backward pass to the stream. Each step is held to its formula in 64 bits on the step's own inputs, eager, on a
stream of its own and replayed from graphs; offsets past 32 bits."""
import pytest

import test_adapters as TA
import test_block_norm as TN
import test_distill as TD
import test_head_norm as TH
import test_linear as TL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def layer(layer_cache, cfg=0):
    from mixed_precision_bit_amd import _lib as M
    from mixed_precision_bit_amd.layer import DeviceLayer
    L = layer_cache(cfg)
    D = DeviceLayer.from_synth(L)
    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q)
    return L, D


def operands(H, T, xd, seed=0, V=1003, k=12):
    """A block's stream and norms, the projection to 4 + 2 + 2 heads of 64 with adapters, an output head of V ids."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t, N = TL.DT[xd], 8 * 64
    o = {"d": TN.inputs(T, H, xd, "token", True, True, seed=seed), "ad": TA.inputs(T, H, N, 3, 16, xd, seed=seed)}
    o["Wqkv"], o["bqkv"] = (rn(N, H) * H ** -0.5).to(t), rn(N)
    o["Wo"], o["Wh"] = (rn(H, 4 * 64) * 256 ** -0.5).to(t), (rn(-(-V // 8) * 8, H) * H ** -0.5).to(t)
    o["gq"], o["gk"] = 1 + 0.1 * rn(64), 1 + 0.1 * rn(64)
    o["pos"] = torch.randint(0, 5000, (3, T), generator=g, device="cuda", dtype=torch.int32)
    o["axis"] = torch.arange(32, device="cuda", dtype=torch.int32) % 3
    o["freq"] = 1e4 ** (-torch.arange(32, device="cuda") / 32.0)
    o["ids"] = torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(T)]).int()
    o["y"], o["w"] = 2 + rn(T, k), torch.rand(T, generator=g, device="cuda")
    o["lse"] = torch.logsumexp(o["y"], 1) + 0.3
    o["V"], o["xd"], o["dk0"] = V, xd, torch.zeros(T, 2, 64, device="cuda", dtype=t)
    return o


def run(D, o, stream=None):
    """Forward and backward; every result by name."""
    xd, d, T = o["xd"], o["d"], o["d"]["r"].shape[0]
    r = {"x": D.norm_in(d["r"], xd, d["gn"], stream=stream)}
    r["qkv32"] = D.project(r["x"], xd, o["Wqkv"], o["bqkv"], adapters=o["ad"], stream=stream)
    r["plain32"] = D.project(r["x"], xd, o["Wqkv"], o["bqkv"], f32=True, stream=stream)
    qkv = D.project(r["x"], xd, o["Wqkv"], o["bqkv"], stream=stream).view(T, 8, 64)
    rot = dict(pos=o["pos"], freq=o["freq"], axis=o["axis"], pairs="neighbours", stream=stream)
    r["qkv"] = qkv
    r["q"], r["k"] = D.heads(qkv[:, :4], qkv[:, 4:6], xd, o["gq"], o["gk"], **rot)
    # the heads back onto the stream through a projection with residual, then the output head and its loss
    r["y"], r["z"] = D.project(r["q"].view(T, 256), xd, o["Wo"], act="silu", res=d["r"], keep=True, stream=stream)
    r["xh"] = D.norm_in(r["y"], xd, d["gn"], stream=stream)
    r["logits"] = D.project(r["xh"], xd, o["Wh"], f32=True, stream=stream)
    S = r["logits"][:, :o["V"]]
    s = D.distill(S, o["ids"], o["y"], o["lse"], o["w"], 2.0, stream=stream)
    r["kl"], r["loss"], r["dS"] = s["kl"], s["loss"], D.distill_grad(s, stream=stream)
    # the gradient of the logits' whole width: zeros in the columns that pad the vocabulary
    dy = torch.as_strided(r["dS"], r["logits"].shape, r["logits"].stride())
    r["dlogits"] = dy
    h = D.project_grad(r["xh"], xd, o["Wh"], dy, stream=stream)
    r["dxh"], r["dWh"] = h["X"], h["W"]
    n = D.block_norm_grad(None, r["y"], xd, None, h["X"], gamma_next=d["gn"], stream=stream)
    r["dy"] = n["r"]
    p = D.project_grad(r["q"].view(T, 256), xd, o["Wo"], n["r"], "silu", r["z"], stream=stream)
    r["dq_out"], r["dWo"], r["dbo"] = p["X"], p["W"], p["bias"]
    b = D.heads_grad(qkv[:, :4], qkv[:, 4:6], xd, p["X"].view(T, 4, 64), o["dk0"], o["gq"], o["gk"], **rot)
    r["dq"], r["dgq"], r["dk"], r["dgk"] = b["q"], b["gamma_q"], b["k"], b["gamma_k"]
    return r


def check(o, r):
    xd, d, T = o["xd"], o["d"], o["d"]["r"].shape[0]
    fwd = lambda X, W, b=None, res=None: {"X": X, "W": W, "b": b, "res": res}  # noqa: E731
    TN.check_fwd({**d, "gate": None, "gp": None}, xd, 1.0, None, r["x"], no_o=True)
    TL.check_fwd(fwd(r["x"], o["Wqkv"], o["bqkv"]), xd, "f32", "none", r["plain32"], None)
    TA.check({**o["ad"], "X": r["x"], "base": r["plain32"]}, r["qkv32"])
    TL.check_fwd(fwd(r["x"], o["Wqkv"], o["bqkv"]), xd, xd, "none", r["qkv"].reshape(T, -1), None)
    h = {"q": r["qkv"][:, :4], "k": r["qkv"][:, 4:6], "gq": o["gq"], "gk": o["gk"], "pos": o["pos"], "axis": o["axis"], "freq": o["freq"], "pairs": 1}
    TH.check_fwd(h, xd, r["q"], r["k"])
    TL.check_fwd(fwd(r["q"].view(T, 256), o["Wo"], None, d["r"]), xd, xd, "silu", r["y"], r["z"])
    TL.check_fwd(fwd(r["xh"], o["Wh"]), xd, "f32", "none", r["logits"], None)
    s = {"S": r["logits"][:, :o["V"]], "ids": o["ids"], "y": o["y"], "lse": o["lse"], "w": o["w"], "tau": 2.0}
    TD.check_loss(s, r["kl"], r["loss"])
    TD.check_grad(s, "f32", r["dS"])
    assert not r["dlogits"][:, o["V"]:].any()
    TL.check_grad({"X": r["xh"], "W": o["Wh"], "z": torch.zeros_like(r["dlogits"])}, xd, r["dlogits"], "none", {"dX": r["dxh"], "dW": r["dWh"], "db": None})
    TL.check_grad({"X": r["q"].view(T, 256), "W": o["Wo"], "z": r["z"]}, xd, r["dy"], "silu", {"dX": r["dq_out"], "dW": r["dWo"], "db": r["dbo"]})
    TH.check_grad({**h, "dq": r["dq_out"].view(T, 4, 64), "dk": torch.zeros_like(r["k"])}, xd, {"q": r["dq"], "k": r["dk"], "gq": r["dgq"], "gk": r["dgk"]})


@pytest.mark.parametrize("cfg,T", [(0, 1), (0, 16), (10, 200), (11, 700)])
def test_a_block_s_dense_side_and_its_gradients(layer_cache, cfg, T):
    L, D = layer(layer_cache, cfg)
    o = operands(D.H, T, L.cfg["xdtype"], seed=cfg)
    check(o, run(D, o))


def test_on_a_stream_of_its_own(layer_cache):
    L, D = layer(layer_cache)
    o = operands(D.H, 40, "f16")
    want = run(D, o)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [run(D, o, s) for s in (s1, s2, s1)]  # two at once
    torch.cuda.synchronize()
    for g in got:
        for k in want:
            assert torch.equal(g[k], want[k]), k


def test_graphs_replayed_between_eager_work(layer_cache):
    """Two captured graphs, replayed in turn on changing inputs, eager calls and synchronisations between."""
    L, D = layer(layer_cache)
    sets = [operands(D.H, T, "f16", seed=T) for T in (16, 130)]
    want = [{k: v.clone() for k, v in run(D, o).items()} for o in sets]
    graphs, outs = [], []
    for o in sets:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            outs.append(run(D, o))
        graphs.append(g)
    for rep in range(3):
        for i in (0, 1, 1, 0):
            for v in outs[i].values():
                v.fill_(float("nan")) if v.is_floating_point() else v.zero_()
            graphs[i].replay()
            run(D, sets[1 - i])
            torch.cuda.synchronize()
            for k in want[i]:
                assert torch.equal(outs[i][k], want[i][k]), (rep, i, k)
        changed = sets[0]["d"]["r"].clone()
        sets[0]["d"]["r"].copy_(torch.randn_like(changed))
        want[0] = {k: v.clone() for k, v in run(D, sets[0]).items()}


def test_adapters_need_a_projection_without_activation(layer_cache):
    from mixed_precision_bit_amd import MpbError
    L, D = layer(layer_cache)
    o = operands(D.H, 4, "f16")
    with pytest.raises(MpbError):
        D.project(D.norm_in(o["d"]["r"], "f16", o["d"]["gn"]), "f16", o["Wqkv"], act="silu", adapters=o["ad"])


# ------------------------------------------------------------------------------------------------ offsets past 32 bits
def test_projection_past_32_bits():
    T, N = 1 << 20, 4104  # 4.3e9 results, 8.6e9 bytes of them
    d = TL.inputs(T, 64, N, "bf16", seed=8, bias=True)
    y, _ = TL.run_fwd(d, "bf16", "bf16", keep=False)
    rows = torch.tensor([0, 1, 523263, 523264, T - 257, T - 1], device="cuda")
    TL.check_fwd({**d, "X": d["X"][rows]}, "bf16", "bf16", "none", y[rows], None)
    out = TL.run_grad(d, "bf16", y, "none", want=("dX", "dW"))
    TL.check_grad({**d, "X": d["X"][rows], "z": y[rows]}, "bf16", y[rows], "none", {"dX": out["dX"][rows], "dW": None, "db": None})
    cols = slice(N - 16, N)
    X, g = d["X"].double(), y[:, cols].double()
    TL.check(out["dW"][cols], g.t() @ X, TL.E(T) * (g.abs().t() @ X.abs()), "dW")


def test_heads_past_32_bits():
    T, Hq, Hk, Dh = 1 << 20, 30, 2, 128  # 4.3e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.empty(T, Hq + Hk, Dh, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    d = {"q": qkv[:, :Hq], "k": qkv[:, Hq:], "gq": torch.ones(Dh, device="cuda"), "gk": None, "axis": None, "pairs": 0,
         "pos": torch.arange(T, device="cuda", dtype=torch.int32)[None], "freq": 1e4 ** (-torch.arange(64, device="cuda") / 64.0)}
    q, k = TH.run_fwd(d, "bf16")
    rows = torch.tensor([0, 555555, T - 2, T - 1], device="cuda")
    at = {**d, "q": d["q"][rows], "k": d["k"][rows], "pos": d["pos"][:, rows]}
    TH.check_fwd(at, "bf16", q[rows], k[rows])
    d["dq"], d["dk"] = q, k
    out = TH.run_grad(d, "bf16")
    TH.check_grad({**at, "dq": q[rows], "dk": k[rows]}, "bf16", {"q": out["q"][rows], "k": out["k"][rows], "gq": None, "gk": None} | {"gq": _rows_gamma(at, q[rows])})


def _rows_gamma(at, dq):
    """The gamma gradient of a few rows alone (that of the whole batch is checked at smaller sizes)."""
    x = at["q"].double()
    n, _ = TH.turn(dq.double(), at, back=True)
    return (n * x / (x.square().mean(2, keepdim=True) + TH.EPS).sqrt()).sum((0, 1)).float()


def test_distillation_past_32_bits():
    T, V = 30001, 150001  # 4.5e9 logits, 9e9 bytes
    g = torch.Generator(device="cuda").manual_seed(2)
    S = torch.empty(T, V, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    ids = (torch.randint(0, V, (T, 1), generator=g, device="cuda") + torch.arange(8, device="cuda") * 17000).remainder(V).int()
    y = torch.randn(T, 8, generator=g, device="cuda")
    d = {"S": S, "ids": ids, "y": y, "lse": torch.logsumexp(y, 1) + 0.5, "w": None, "tau": 1.0}
    dS = torch.empty_like(S)
    _, kl, _ = TD.call(d, "bf16", dS, torch.full((1,), float(T), device="cuda"))
    rows = torch.tensor([0, 14316, 14317, 28633, T - 1], device="cuda")
    at = {**d, **{k: d[k][rows] for k in ("S", "ids", "y", "lse")}, "w": torch.ones(5, device="cuda")}
    TD.check_loss(at, kl[rows], kl[rows].double().sum()[None])
    TD.check_grad(at, "bf16", dS[rows])

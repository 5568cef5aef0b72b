"""The rest of the chain of test_dense: from the heads' gradients on to those of the query, key and value projection and
of the block's normed stream, and of the stream itself. moe_head_norm_grad writes the heads' gradients into views of one
packed tensor, next to the value heads', which the projection's gradients take as it is. The projections of a frozen
weight ask for dX alone. Each step is held to its formula in 64 bits on the step's own inputs."""
import pytest

import test_block_norm as TN
import test_dense as TDe
import test_head_norm as TH
import test_linear as TL

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def onward(D, o, r, stream=None):
    """From the results r of test_dense.run to the stream, without a copy of the heads' gradients."""
    M = TL.lib_m()
    xd, d, T = o["xd"], o["d"], o["d"]["r"].shape[0]
    xt = M.MPB_BF16 if xd == "bf16" else M.MPB_F16
    with D._on(stream):
        packed = torch.empty(T, 8, 64, device="cuda", dtype=TL.DT[xd])
        packed[:, 6:].copy_(o["dv"])
        dgq, dgk = torch.empty_like(o["gq"]), torch.empty_like(o["gk"])
        ws = torch.empty(M.moe_head_norm_grad_workspace_bytes(T, 4, 2, 64), dtype=torch.uint8, device="cuda")
        alone = torch.empty(T, D.H, device="cuda", dtype=TL.DT[xd])
        ws_x = torch.empty(M.moe_linear_grad_workspace_bytes(T, D.H, 512, M.MPB_ACT_NONE, xt), dtype=torch.uint8, device="cuda")
    qkv = r["qkv"]
    M.moe_head_norm_grad(qkv[:, :4], qkv[:, 4:6], xt, o["gq"], o["gk"], 1e-6, o["pos"], o["axis"], o["freq"], M.MPB_PAIRS_NEIGHBOURS,
                         r["dq_out"].view(T, 4, 64), o["dk0"], packed[:, :4], packed[:, 4:6], dgq, dgk, ws, stream)
    g = D.project_grad(r["x"], xd, o["Wqkv"], packed.view(T, 512), stream=stream)
    M.moe_linear_grad(r["x"], xt, o["Wqkv"], M.MPB_ACT_NONE, None, packed.view(T, 512), alone, None, None, ws_x, stream)
    n = D.block_norm_grad(None, d["r"], xd, r["dy"], g["X"], gamma_next=d["gn"], stream=stream)
    return {"packed": packed, "dgq": dgq, "dgk": dgk, "dx": g["X"], "dx_alone": alone, "dWqkv": g["W"], "dbqkv": g["bias"], "dr": n["r"],
            "dgn": n["gamma_next"]}


def operands(H, T, xd, seed):
    o = TDe.operands(H, T, xd, seed=seed)
    o["dv"] = (0.01 * torch.randn(T, 2, 64, device="cuda")).to(TL.DT[xd])
    return o


def check(o, r, s):
    xd, d, T = o["xd"], o["d"], o["d"]["r"].shape[0]
    p = s["packed"]
    assert torch.equal(p[:, :4], r["dq"]) and torch.equal(p[:, 4:6], r["dk"]) and torch.equal(p[:, 6:], o["dv"])
    assert torch.equal(s["dgq"], r["dgq"]) and torch.equal(s["dgk"], r["dgk"])
    TL.check_grad({"X": r["x"], "W": o["Wqkv"], "z": torch.zeros(T, 512, device="cuda")}, xd, p.view(T, 512), "none",
                  {"dX": s["dx"], "dW": s["dWqkv"], "db": s["dbqkv"]})
    assert torch.equal(s["dx_alone"], s["dx"])
    # the stream's: what came past the block, and through its norm
    leaf, gn = d["r"].double().requires_grad_(), d["gn"].double().requires_grad_()
    dx, dy = s["dx"].double(), r["dy"].double()
    a, b = torch.autograd.grad((leaf * TN.rms(leaf) * gn * dx).sum(), [leaf, gn])
    leaf = leaf.detach()
    ry = TN.rms(leaf)
    e, yh = (dx * d["gn"].double()).abs(), (leaf * ry).abs()
    size = dy.abs() + ry * (e + yh * (e * yh).mean(1, keepdim=True))
    TN.check(s["dr"], dy + a, TN.E1 * size + 1.01 * TN.half_step(TL.DT[xd], dy + a), "dr")
    TN.check(s["dgn"], b, (TN.E1 + TN.U * (T / 512 + 48)) * (dx.abs() * yh).sum(0) + 1e-30, "dgn")


@pytest.mark.parametrize("cfg,T", [(0, 1), (0, 16), (10, 200), (11, 700)])
def test_to_the_stream_s_gradient(layer_cache, cfg, T):
    L, D = TDe.layer(layer_cache, cfg)
    o = operands(D.H, T, L.cfg["xdtype"], cfg)
    r = TDe.run(D, o)
    check(o, r, onward(D, o, r))


def test_on_streams_and_from_replayed_graphs(layer_cache):
    L, D = TDe.layer(layer_cache)
    o = operands(D.H, 130, "f16", 1)
    r = TDe.run(D, o)
    want = {k: v.clone() for k, v in onward(D, o, r).items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [onward(D, o, r, s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(g[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = onward(D, o, r)
    for rep in range(3):
        for v in out.values():
            v.fill_(float("nan"))
        graph.replay()
        onward(D, o, r)  # eager work between
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want), rep
        r["dq_out"].neg_()
        want = {k: v.clone() for k, v in onward(D, o, r).items()}
        torch.cuda.synchronize()

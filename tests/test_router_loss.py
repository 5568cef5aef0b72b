"""moe_router_loss and moe_router_loss_grad against the formulas in 64 bits.

Tolerances. u = 2^-24. A logit is a sum of H products of parts, at most five
matrix instructions for 32 of them, each instruction's result rounded to fp32
after up to 32 additions of its own, over ranges that are added once more: within
n(H) u of the sum of the products' absolute values, n(L) = 6 L / 32 + 96; what the
cut parts leave out is below 4 u of it. The gradients' products have the same form
with L = E rounded up to 64 or the number of tokens; dX takes three instructions
instead of up to six and its halves leave out 12 u: 3 L / 32 + 96 + 12 is below
n(L) + 8 from L = 64. Sums of p over tokens pass at
most T / 2048 + 32 additions, exponentials and logarithms are within 4 u of their
value and carry their argument's error."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def n_of(length):
    return 6 * length / 32 + 100


def formula(X, W, b, idx, mask, alpha, beta, gw=None, counts=None):
    """Everything by the definition; differentiable in X, W and b."""
    T, E, K = X.shape[0], W.shape[0], idx.shape[1]
    live = torch.ones(T, dtype=torch.bool, device=X.device) if mask is None else mask.bool()
    l = torch.where(live[:, None], X, torch.zeros_like(X)) @ W.t()
    if b is not None:
        l = l + b
    dead = (l == -float("inf")).all(1)
    live = live & ~dead
    ls = torch.where(live[:, None], l, torch.zeros_like(l))  # keeps nan out of the others' gradients
    lse = torch.logsumexp(ls, 1)
    p = torch.softmax(ls, 1) * live[:, None]
    if counts is None:
        counts = torch.zeros(E + 1, dtype=torch.int64, device=X.device)
        ok = live[:, None] & (idx >= 0) & (idx < E)
        counts.index_add_(0, idx[ok].long(), torch.ones_like(idx[ok].long()))
        counts[E] = live.sum()
    N = max(1, int(counts[E]))
    prob = p.sum(0)
    bal = E / (K * N * N) * (counts[:E].double() * prob).sum()
    z = (lse * lse * live).sum() / N
    loss = alpha * bal + beta * z
    total = loss
    if gw is not None:
        ok = (idx >= 0) & (idx < E)
        lk = torch.where(ok, ls.gather(1, idx.clamp(0, E - 1).long()), torch.full_like(gw, -float("inf")))
        some = ok.any(1) & live
        w = torch.softmax(torch.where(some[:, None], lk, torch.zeros_like(lk)), 1)
        total = loss + (w * gw * ok * some[:, None]).sum()
    return {"l": l, "lse": lse, "p": p, "live": live, "dead": dead, "counts": counts, "prob": prob, "loss": loss, "bal": bal, "z": z, "total": total, "N": N}


def inputs(T, H, E, K, dt, masked, bias=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, H, generator=g, device="cuda").to(DT[dt])
    W = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    b = -0.5 * torch.log1p(torch.arange(E, device="cuda").float()) if bias else None
    l = X.float() @ W.t() + (b if bias else 0)
    idx = torch.topk(l, K, dim=1).indices.int().contiguous()
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if masked else None
    gw = torch.randn(T, K, generator=g, device="cuda") / T
    return {"X": X, "W": W, "b": b, "idx": idx, "mask": mask, "gw": gw}


def run_fwd(d, dt, alpha=0.01, beta=0.001, stream=None, ws=None):
    M = lib_m()
    (T, H), E = d["X"].shape, d["W"].shape[0]
    nan = float("nan")
    full = lambda *s: torch.full(s, nan, device="cuda")  # noqa: E731
    o = {"logits": full(T, E), "lse": full(T), "counts": torch.full((E + 1,), -7, dtype=torch.int32, device="cuda"),
         "prob": full(E), "loss": full(3)}
    if ws is None:
        ws = torch.empty(M.moe_router_loss_workspace_bytes(T, H, E), dtype=torch.uint8, device="cuda")
    M.moe_router_loss(d["X"], M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["W"], d["b"], d["idx"], d["mask"], alpha, beta,
                      o["logits"], o["lse"], o["counts"], o["prob"], o["loss"], ws, stream)
    return o


def run_grad(d, dt, o, alpha=0.01, beta=0.001, gw=True, gloss=None, counts=None, want=("dX", "dW", "db"), stream=None, ws=None):
    M = lib_m()
    (T, H), E = d["X"].shape, d["W"].shape[0]
    full = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    g = {"dX": full(T, H), "dW": full(E, H), "db": full(E)}
    if ws is None:
        ws = torch.empty(M.moe_router_loss_workspace_bytes(T, H, E), dtype=torch.uint8, device="cuda")
    M.moe_router_loss_grad(d["X"], M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["W"], d["idx"], d["mask"], o["logits"],
                           o["lse"], o["counts"] if counts is None else counts, alpha, beta, d["gw"] if gw else None,
                           gloss, *(g[k] if k in want else None for k in ("dX", "dW", "db")), ws, stream)
    return {k: g[k] for k in want}


def dbl(d):
    return {k: v.double() if v is not None and v.is_floating_point() else v for k, v in d.items()}


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


def clean(D):
    """Inputs with what masked rows hold replaced by zeros (their values are not used)."""
    if D["mask"] is None:
        return D
    return {**D, "X": torch.where(D["mask"].bool()[:, None], D["X"], torch.zeros_like(D["X"]))}


def logit_tol(D):
    b = 0 if D["b"] is None else torch.nan_to_num(D["b"], neginf=0.0).abs()
    return n_of(D["X"].shape[1]) * U * (D["X"].abs() @ D["W"].abs().t()) + 2 * U * b


def check_fwd(d, dt, o, alpha=0.01, beta=0.001):
    D = clean(dbl(d))
    f = formula(D["X"], D["W"], D["b"], D["idx"], D["mask"], alpha, beta)
    T, E, K = D["X"].shape[0], D["W"].shape[0], D["idx"].shape[1]
    assert torch.equal(o["counts"].long(), f["counts"])
    masked = torch.zeros(T, dtype=torch.bool, device="cuda") if D["mask"] is None else ~D["mask"].bool()
    tl = logit_tol(D)
    fin = torch.isfinite(f["l"]) & ~masked[:, None]
    assert not o["logits"][masked].any() and not o["lse"][masked].any()
    assert torch.equal(o["logits"][~fin & ~masked[:, None]].double(), f["l"][~fin & ~masked[:, None]])
    check(o["logits"][fin], f["l"][fin], tl[fin] + U * f["l"][fin].abs(), "logits")
    el = torch.where(fin, tl, torch.zeros_like(tl)).amax(1)
    lv = f["live"]
    assert (o["lse"][f["dead"] & ~masked] == -float("inf")).all()
    tlse = el + 16 * U * (1 + f["lse"].abs())
    check(o["lse"][lv], f["lse"][lv], tlse[lv], "lse")
    tp = (f["p"] * (2 * (el + tlse)[:, None] + 64 * U)).sum(0) + (T / 2048 + 64) * U * f["prob"] + 1e-37
    check(o["prob"], f["prob"], tp, "prob")
    tb = E / (K * f["N"] ** 2) * (f["counts"][:E].double() * tp).sum() + 4 * U * f["bal"]
    tz = (2 * f["lse"].abs() * tlse * lv).sum() / f["N"] + (T / 2048 + 64) * U * f["z"]
    check(o["loss"], torch.stack([f["loss"], f["bal"], f["z"]]), torch.stack([abs(alpha) * tb + abs(beta) * tz, tb, tz]) * 1.01 + 1e-37, "loss")
    return f


def check_grad(d, dt, g, alpha=0.01, beta=0.001, gw=True, gloss=1.0, counts=None):
    D = clean(dbl(d))
    T, H, E, K = *D["X"].shape, D["W"].shape[0], D["idx"].shape[1]
    X, W = D["X"].clone().requires_grad_(), D["W"].clone().requires_grad_()
    b = (torch.zeros(E, dtype=torch.float64, device="cuda") if D["b"] is None else D["b"].clone()).requires_grad_()
    f = formula(X, W, b, D["idx"], D["mask"], gloss * alpha, gloss * beta, D["gw"] if gw else None, counts)
    ref = dict(zip(("dX", "dW", "db"), torch.autograd.grad(f["total"], [X, W, b])))
    f = {k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in f.items()}
    # the tolerance of dl, element by element, and the absolute value it is made of
    el = torch.where(torch.isfinite(f["l"]), logit_tol(D), torch.zeros_like(f["l"])).amax(1, keepdim=True)
    N = f["N"]
    fr = f["counts"][:E].double() / (K * N)
    a, c = abs(gloss * alpha) * E / N, abs(gloss * beta) * 2 / N
    mag = f["p"] * (a * (fr + (f["p"] * fr).sum(1, keepdim=True)) + c * f["lse"].abs()[:, None])
    if gw:
        ok = (D["idx"] >= 0) & (D["idx"] < E) & f["live"][:, None]
        lk = torch.where(ok, f["l"].gather(1, D["idx"].clamp(0, E - 1).long()), torch.full_like(D["gw"], -1e30))
        w = torch.softmax(lk, 1) * ok
        m = w * (D["gw"].abs() + (w * D["gw"].abs()).sum(1, keepdim=True))
        mag = mag.scatter_add(1, D["idx"].clamp(0, E - 1).long(), m * ok)
    tol = mag * (6 * el + 160 * U) + f["p"] * c * (el + 16 * U * (1 + f["lse"].abs()[:, None]))
    if "dX" in g:
        check(g["dX"], ref["dX"], tol @ D["W"].abs() + (n_of(-(-E // 64) * 64) + 4) * U * (mag @ D["W"].abs()) + 1e-37, "dX")
    if "dW" in g:
        check(g["dW"], ref["dW"], tol.t() @ D["X"].abs() + (n_of(T) + 4) * U * (mag.t() @ D["X"].abs()) + 1e-37, "dW")
    if "db" in g:
        check(g["db"], ref["db"], tol.sum(0) + 64 * U * mag.sum(0) + 1e-37, "dbias")


SHAPES = [(1, 64, 1, 1), (1, 2048, 60, 4), (5, 64, 2, 2), (72, 2048, 60, 4), (130, 192, 8, 2), (33, 128, 512, 16),
          (700, 320, 129, 8), (4099, 256, 60, 4), (65, 65536, 4, 2), (1000, 2816, 128, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,H,E,K", SHAPES)
def test_loss_and_gradients(T, H, E, K, masked, dt):
    d = inputs(T, H, E, K, dt, masked)
    o = run_fwd(d, dt)
    check_fwd(d, dt, o)
    for gw in (True, False):
        check_grad(d, dt, run_grad(d, dt, o, gw=gw), gw=gw)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_masked_rows_may_hold_anything(dt):
    d = inputs(300, 128, 16, 2, dt, True, seed=1)
    dead = (d["mask"] == 0).nonzero()[:, 0]
    assert len(dead) > 20
    want = run_fwd(d, dt)
    wg = run_grad(d, dt, want)
    d["X"][dead] = float("nan")
    d["X"][dead[::2]] = float("inf")
    d["idx"][dead[0]] = 1 << 30
    o = run_fwd(d, dt)
    g = run_grad(d, dt, o)
    for a, b in ((o, want), (g, wg)):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    assert not g["dX"][dead].any()


@pytest.mark.gpu
def test_no_live_token():
    """Every token masked, and every logit -inf: losses and gradients are zeros."""
    d = inputs(70, 128, 8, 2, "bf16", True, seed=2)
    d["mask"].zero_()
    e = inputs(70, 128, 8, 2, "bf16", False, seed=2)
    e["b"] = torch.full((8,), -float("inf"), device="cuda")
    for v in (d, e):
        o = run_fwd(v, "bf16")
        assert not o["loss"].any() and not o["counts"].any() and not o["prob"].any()
        for k, x in run_grad(v, "bf16", o).items():
            assert not x.any(), k


@pytest.mark.gpu
def test_switched_off_experts_and_infinite_activations():
    """A bias of -inf takes an expert out; an infinite logit makes its own row's values nan and the sums over rows nan."""
    d = inputs(200, 128, 12, 3, "bf16", True, seed=3)
    d["b"][4] = d["b"][11] = -float("inf")
    l = d["X"].float() @ d["W"].t() + d["b"]
    d["idx"] = torch.topk(l, 3, dim=1).indices.int().contiguous()
    o = run_fwd(d, "bf16")
    check_fwd(d, "bf16", o)
    assert not o["prob"][4].any() and not o["prob"][11].any()
    check_grad(d, "bf16", run_grad(d, "bf16", o))
    row = int(d["mask"].nonzero()[0, 0])
    d["X"][row, 5] = float("inf")
    n = run_fwd(d, "bf16")
    assert torch.isnan(n["lse"][row]) and torch.isnan(n["loss"]).all()
    keep = torch.arange(200, device="cuda") != row
    assert torch.equal(n["logits"][keep], o["logits"][keep]) and torch.equal(n["lse"][keep], o["lse"][keep])


@pytest.mark.gpu
def test_ids_out_of_range_and_named_twice():
    d = inputs(150, 256, 20, 4, "f16", False, seed=4)
    d["idx"][3] = torch.tensor([5, 5, 5, 2])
    d["idx"][4] = torch.tensor([-1, 20, 1 << 30, -(1 << 31)])
    d["idx"][5] = torch.tensor([7, -1, 8, 20])
    o = run_fwd(d, "f16")
    check_fwd(d, "f16", o)
    check_grad(d, "f16", run_grad(d, "f16", o))


@pytest.mark.gpu
def test_single_gradients_scale_and_repeatability():
    """Each gradient alone is bit-equal to the same one of a full call; gloss scales the loss's part."""
    d = inputs(513, 448, 60, 4, "bf16", True, seed=5)
    o = run_fwd(d, "bf16")
    p = run_fwd(d, "bf16")
    for k in o:
        assert torch.equal(o[k], p[k]), k
    g = run_grad(d, "bf16", o)
    for k in g:
        assert torch.equal(run_grad(d, "bf16", o, want=(k,))[k], g[k]), k
    s = torch.tensor([128.0], device="cuda")
    check_grad(d, "bf16", run_grad(d, "bf16", o, gloss=s), gloss=128.0)
    check_grad(d, "bf16", run_grad(d, "bf16", o, alpha=0.0, beta=0.0), alpha=0.0, beta=0.0)


@pytest.mark.gpu
def test_counts_of_a_group_of_batches():
    """Two halves with their counts added give the gradients of the whole batch's loss."""
    d = inputs(256, 128, 16, 2, "bf16", True, seed=6)
    o = run_fwd(d, "bf16")
    half = [{k: v[s] if v is not None and k in ("X", "idx", "mask", "gw") else v for k, v in d.items()}
            for s in (slice(0, 100), slice(100, 256))]
    oh = [run_fwd(h, "bf16") for h in half]
    counts = oh[0]["counts"] + oh[1]["counts"]
    assert torch.equal(counts, o["counts"])
    for h, q in zip(half, oh):
        check_grad(h, "bf16", run_grad(h, "bf16", q, counts=counts), counts=counts.long())


@pytest.mark.gpu
def test_empty_batch():
    M = lib_m()
    X = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(8, 128, device="cuda")
    d = {"X": X, "W": W, "b": None, "idx": torch.empty(0, 2, dtype=torch.int32, device="cuda"), "mask": None,
         "gw": torch.empty(0, 2, device="cuda")}
    o = run_fwd(d, "bf16")
    assert not o["loss"].any() and not o["counts"].any() and not o["prob"].any()
    g = run_grad(d, "bf16", o)
    assert not g["dW"].any() and not g["db"].any()
    assert M.moe_router_loss_workspace_bytes(0, 128, 8) > 0


@pytest.mark.gpu
def test_stream_and_graph_replays():
    d, e = (inputs(200, 320, 24, 3, "f16", True, seed=s) for s in (7, 8))
    want = []
    for v in (d, e):
        o = run_fwd(v, "f16")
        want.append((o, run_grad(v, "f16", o)))
    st = {k: v.clone() for k, v in d.items()}
    M = lib_m()
    ws = torch.empty(M.moe_router_loss_workspace_bytes(200, 320, 24), dtype=torch.uint8, device="cuda")

    def both():
        o = run_fwd(st, "f16", ws=ws)
        return o, run_grad(st, "f16", o, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both()
    s.synchronize()
    for a, b in zip(got, want[0]):
        for k in a:
            assert torch.equal(a[k], b[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in (0, 1, 0, 1):
        for k, v in st.items():
            v.copy_((d, e)[i][k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want[i]):
            for k in a:
                assert torch.equal(a[k], b[k]), k
        run_fwd(e, "f16")


def test_formula_gradients_against_differences():
    """The 64-bit gradients that the kernels are held to, against central differences (CPU); the counts stay fixed."""
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, H, E, K = 6, 10, 5, 2
    v = {"X": rn(T, H), "W": rn(E, H), "b": rn(E)}
    mask = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.uint8)
    idx = torch.topk(v["X"] @ v["W"].t() + v["b"], K).indices.int()
    gw = rn(T, K)
    loss = lambda q: formula(q["X"], q["W"], q["b"], idx, mask, 0.3, 0.2, gw)["total"]  # noqa: E731
    leaf = {k: x.clone().requires_grad_() for k, x in v.items()}
    grads = dict(zip(leaf, torch.autograd.grad(loss(leaf), list(leaf.values()))))
    # and by hand, as the kernels form them
    f = formula(v["X"], v["W"], v["b"], idx, mask, 0.3, 0.2)
    fr = f["counts"][:E].double() / (K * f["N"])
    dl = f["p"] * (0.3 * E / f["N"] * (fr - (f["p"] * fr).sum(1, keepdim=True)) + 2 * 0.2 / f["N"] * f["lse"][:, None])
    w = torch.softmax(f["l"].gather(1, idx.long()), 1)
    dl = dl.scatter_add(1, idx.long(), mask[:, None] * w * (gw - (w * gw).sum(1, keepdim=True)))
    for k, x in {"X": dl @ v["W"], "W": dl.t() @ v["X"], "b": dl.sum(0)}.items():
        assert torch.allclose(grads[k], x, rtol=1e-12, atol=1e-14), k
        way, h = rn(*v[k].shape), 1e-6
        diff = float(loss({**v, k: v[k] + h * way}) - loss({**v, k: v[k] - h * way})) / (2 * h)
        want = float((x * way).sum())
        assert abs(diff - want) <= 1e-7 * (1 + abs(want)), k


def test_refusals():
    M = lib_m()
    from mixed_precision_bit_amd import _lib
    L = _lib.lib()
    p, odd, big = ctypes.c_void_p(16), ctypes.c_void_p(4), 1 << 34

    def fwd(X=p, xd=0, W=p, b=None, i=p, m=None, T=4, H=256, E=8, K=2, al=0.1, be=0.1, l=p, s=p, c=p, pr=p, lo=p, ws=p, n=big):
        return L.moe_router_loss(X, xd, W, b, i, m, T, H, E, K, al, be, l, s, c, pr, lo, ws, n, None)

    assert fwd(xd=2) == -1 and fwd(T=-1) == -1 and fwd(T=(1 << 20) + 1) == -2 and fwd(H=96) == -2 and fwd(H=65600) == -2
    assert fwd(E=0) == -2 and fwd(E=513) == -2 and fwd(K=0) == -2 and fwd(K=9) == -2 and fwd(E=64, K=17) == -2
    assert fwd(al=float("inf")) == -1 and fwd(be=float("nan")) == -1
    for k in ("X", "W", "i", "l", "s", "c", "pr", "lo", "ws"):
        assert fwd(**{k: None}) == -1, k
    assert fwd(X=odd) == -1 and fwd(W=odd) == -1 and fwd(ws=odd) == -1 and fwd(n=255) == -5

    def bwd(X=p, xd=1, W=p, i=p, m=None, l=p, s=p, c=p, T=4, H=256, E=8, K=2, al=0.1, be=0.1, gw=p, gl=None, dX=p, dW=p, db=p, ws=p, n=big):
        return L.moe_router_loss_grad(X, xd, W, i, m, l, s, c, T, H, E, K, al, be, gw, gl, dX, dW, db, ws, n, None)

    assert bwd(xd=3) == -1 and bwd(H=1) == -2 and bwd(E=600) == -2 and bwd(K=9) == -2
    for k in ("X", "W", "i", "l", "s", "c", "ws"):
        assert bwd(**{k: None}) == -1, k
    assert bwd(dX=None, dW=None, db=None) == -1 and bwd(dX=odd) == -1 and bwd(dW=odd) == -1 and bwd(n=100) == -5
    assert M.moe_router_loss_workspace_bytes(4, 100, 8) == 0 == M.moe_router_loss_workspace_bytes(4, 128, 513)


def test_tensor_refusals():
    M = lib_m()
    X, W = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, 128)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    o = [torch.zeros(4, 8), torch.zeros(4), torch.zeros(9, dtype=torch.int32), torch.zeros(8), torch.zeros(3)]
    ws = torch.zeros(1 << 20, dtype=torch.uint8)

    def code(X=X, W=W, idx=idx, mask=None, o=o):
        with pytest.raises(M.MpbError) as e:
            M.moe_router_loss(X, M.MPB_BF16, W, None, idx, mask, 0.1, 0.1, *o, ws)
        return e.value.code

    assert code() == -1                                    # on the CPU
    assert code(X=X.float()) == -1 and code(W=W.double()) == -1 and code(idx=idx.long()) == -1
    assert code(W=W[:, :64]) == -2 and code(idx=idx[:3]) == -2 and code(mask=torch.zeros(5, dtype=torch.uint8)) == -2
    assert code(mask=torch.zeros(4)) == -1 and code(o=[*o[:2], o[2][:8], *o[3:]]) == -2 and code(X=X[0]) == -2

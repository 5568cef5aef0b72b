"""moe_block_norm and moe_block_norm_grad against the formulas in 64 bits.

Tolerances. u = 2^-24 is the fp32 rounding. A row's sum passes at most 8 NV <= 64
additions in a thread, 6 in a wave and 16 over the waves, so a sum of terms is
within 90 u of its terms' absolute sum, a mean square within 90 u and its
reciprocal root within 50 u; products of up to ten factors and the exponential
(within |g| + 4 units, |g| <= 10 here) add less than 30 u. A value made of one
such sum is therefore within E1 = 200 u of its terms' absolute sum, one made of
two nested ones within E2 = 400 u. A stored 16-bit value adds eps / 2 of itself
and half the smallest step."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
E1, E2 = 200 * U, 400 * U
EPS = 1e-6
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def half_step(dt, v):
    return torch.finfo(dt).eps / 2 * v.abs() + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def sig(g):
    return 1 / (1 + torch.exp(-g))


def rms(v):
    return 1 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)


def forward64(o, r, gate, gp, gn, scale):
    """(y, x, |added|) of the formula."""
    y, added = r, torch.zeros_like(r)
    if o is not None:
        u = o * rms(o) * gp if gp is not None else o
        if gate is not None:
            u = u * sig(gate if gate.dim() == 2 else gate[:, None])
        added = scale * u
        y = r + added
    return y, (y * rms(y) * gn if gn is not None else None), added.abs()


def inputs(T, H, dt, gate, post, nxt, seed=0, std_o=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = {"o": rn(T, H) * std_o, "r": (1.5 * rn(T, H)).to(DT[dt]), "dr_out": rn(T, H).to(DT[dt]), "dx": rn(T, H).to(DT[dt])}
    d["gate"] = {"none": None, "token": rn(T), "full": rn(T, H).to(DT[dt])}[gate]
    d["gp"] = 1 + 0.1 * rn(H) if post else None
    d["gn"] = 1 + 0.1 * rn(H) if nxt else None
    return d


def dbl(d):
    return {k: None if v is None else v.double() for k, v in d.items()}


def run_fwd(d, dt, scale, inplace=False, stream=None, no_o=False):
    M = lib_m()
    r = d["r"].clone()
    r_out = None if no_o else (r if inplace else torch.full_like(r, float("nan")))
    x = None if d["gn"] is None else torch.full_like(r, float("nan"))
    M.moe_block_norm(None if no_o else d["o"], r, M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["gate"], d["gp"], d["gn"],
                     scale, EPS, r_out, x, stream)
    return r_out, x


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


def check_fwd(d, dt, scale, r_out, x, no_o=False):
    D = dbl(d)
    y, xr, added = forward64(None if no_o else D["o"], D["r"], D["gate"], D["gp"], D["gn"], scale)
    dy = E1 * added + 2 * U * y.abs()
    if r_out is not None:
        check(r_out, y, dy + 1.01 * half_step(DT[dt], y), "r_out")
    if x is not None:
        rel = dy.norm(dim=1, keepdim=True) / y.norm(dim=1, keepdim=True).clamp(min=1e-300) + E1
        tol = D["gn"].abs() * rms(y) * dy + rel * xr.abs()
        check(x, xr, tol + 1.01 * half_step(DT[dt], xr), "x")


SHAPES = [(1, 2048), (3, 64), (72, 2816), (129, 4096), (5, 16384), (3, 16448), (2, 65536), (4099, 320)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("gate,post,nxt", [("none", False, True), ("none", True, False), ("token", True, True),
                                           ("full", True, True), ("full", False, True), ("token", False, False)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, gate, post, nxt, dt):
    d = inputs(T, H, dt, gate, post, nxt)
    check_fwd(d, dt, 0.7, *run_fwd(d, dt, 0.7))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 64), (72, 2816), (4099, 320)])
def test_forward_norm_only(T, H):
    d = inputs(T, H, "bf16", "none", False, True)
    _, x = run_fwd(d, "bf16", 1.0, no_o=True)
    check_fwd(d, "bf16", 1.0, None, x, no_o=True)


@pytest.mark.gpu
def test_forward_in_place_and_rows_behind_the_last():
    d = inputs(40, 2048, "f16", "token", True, True)
    M = lib_m()
    want = run_fwd(d, "f16", -0.3)
    r, x = d["r"].clone(), torch.full_like(d["r"], 7.0)
    M.moe_block_norm(d["o"][:33], r[:33], M.MPB_F16, d["gate"][:33], d["gp"], d["gn"], -0.3, EPS, r[:33], x[:33])
    assert torch.equal(r[:33], want[0][:33]) and torch.equal(x[:33], want[1][:33])
    assert torch.equal(r[33:], d["r"][33:]) and bool((x[33:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_forward_extreme_values(dt):
    """Rows of zeros, gates of plus and minus infinity, a row that holds inf or nan: its own row only."""
    T, H = 7, 512
    d = inputs(T, H, dt, "token", True, True, seed=3)
    d["o"][1] = 0
    d["o"][2] = 0
    d["r"][2] = 0
    d["gate"][3], d["gate"][4] = float("inf"), -float("inf")
    d["o"][5, 17] = float("nan")
    d["r"][6, 100] = float("inf")
    r_out, x = run_fwd(d, dt, 0.7)
    keep = [0, 1, 2, 3, 4]
    e = {k: v[keep] if v is not None and v.shape[0] == T else v for k, v in d.items()}
    check_fwd(e, dt, 0.7, r_out[keep], x[keep])
    assert torch.equal(r_out[4], d["r"][4]) and not r_out[2].any() and not x[2].any()
    assert torch.isnan(x[5]).all() and torch.isnan(r_out[5]).all()
    assert torch.isinf(r_out[6, 100]) and torch.isnan(x[6, 100])


# ---------------------------------------------------------------- backward
def run_grad(d, dt, scale, stream=None, ws=None):
    M = lib_m()
    T, H = d["r"].shape
    nan = float("nan")
    out = {"dr": torch.full_like(d["r"], nan), "do": torch.full((T, H), nan, device="cuda"),
           "dgate": None if d["gate"] is None else torch.full_like(d["gate"], nan),
           "dgp": None if d["gp"] is None else torch.full_like(d["gp"], nan),
           "dgn": None if d["gn"] is None else torch.full_like(d["gn"], nan)}
    if ws is None:
        ws = torch.empty(M.moe_block_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    M.moe_block_norm_grad(d["o"], d["r"], M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["gate"], d["gp"], d["gn"], scale,
                          EPS, d["dr_out"], d["dx"] if d["gn"] is not None else None, out["dr"], out["do"],
                          out["dgate"], out["dgp"], out["dgn"], ws, stream)
    return out


def grad64(D, scale):
    """Gradients by 64-bit automatic differentiation of the formula, the stream's
    gradient first: d["r"] is the stream after the block."""
    leaf = {k: D[k].clone().requires_grad_() for k in ("o", "r", "gate", "gp", "gn") if D[k] is not None}
    dy = torch.zeros_like(D["r"]) if D["dr_out"] is None else D["dr_out"].clone()
    g = {}
    if "gn" in leaf:
        y = leaf["r"]
        a, b = torch.autograd.grad((y * rms(y) * leaf["gn"] * D["dx"]).sum(), [y, leaf["gn"]])
        dy, g["dgn"] = dy + a, b
    g["dr"] = dy
    u = leaf["o"] * rms(leaf["o"]) * leaf["gp"] if "gp" in leaf else leaf["o"]
    if "gate" in leaf:
        u = u * sig(leaf["gate"] if D["gate"].dim() == 2 else leaf["gate"][:, None])
    names = [k for k in ("o", "gate", "gp") if k in leaf]
    for k, v in zip(names, torch.autograd.grad((scale * u * dy).sum(), [leaf[k] for k in names])):
        g["d" + k] = v
    return g


def check_grad(d, dt, scale, out):
    D = dbl(d)
    g = grad64(D, scale)
    T, H = D["r"].shape
    A = torch.zeros_like(D["r"]) if D["dr_out"] is None else D["dr_out"].abs()
    if D["gn"] is not None:
        ry = rms(D["r"])
        e, yh = (D["dx"] * D["gn"]).abs(), (D["r"] * ry).abs()
        A = A + ry * (e + yh * (e * yh).mean(1, keepdim=True))
        cols = (E1 + U * (T / 512 + 48)) * (D["dx"].abs() * yh).sum(0)
        check(out["dgn"], g["dgn"], cols + 1e-30, "dgamma_next")
    check(out["dr"], g["dr"], E1 * A + 1.01 * half_step(DT[dt], g["dr"]), "dr")
    s = torch.ones(T, 1, device="cuda", dtype=torch.float64)
    if D["gate"] is not None:
        s = sig(D["gate"] if D["gate"].dim() == 2 else D["gate"][:, None])
    du, oh, w = abs(scale) * s * A, D["o"], 1.0
    ro = 1.0
    if D["gp"] is not None:
        ro, w = rms(D["o"]), D["gp"].abs()
        oh = oh * ro
        cols = (E2 + U * (T / 512 + 48)) * (du * oh.abs()).sum(0)
        check(out["dgp"], g["dgp"], cols + 1e-30, "dgamma_post")
    m = (du * w * oh.abs()).mean(1, keepdim=True) if D["gp"] is not None else 0.0
    check(out["do"], g["do"], E2 * ro * (du * w + oh.abs() * m) + 1e-30, "do")
    if D["gate"] is not None:
        part = du * w * oh.abs() * (1 - s)
        if D["gate"].dim() == 2:
            check(out["dgate"], g["dgate"], E2 * part + 1.01 * half_step(DT[dt], g["dgate"]), "dgate")
        else:
            check(out["dgate"], g["dgate"], E2 * part.sum(1) + 1e-30, "dgate")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("gate,post,nxt", [("none", False, True), ("none", True, False), ("token", True, True),
                                           ("full", True, True), ("full", False, True), ("token", False, False),
                                           ("none", False, False)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_grad(T, H, gate, post, nxt, dt):
    d = inputs(T, H, dt, gate, post, nxt, seed=1)
    check_grad(d, dt, 0.7, run_grad(d, dt, 0.7))


@pytest.mark.gpu
def test_grad_without_stream_gradient_and_repeatable():
    d = inputs(600, 1024, "bf16", "full", True, True, seed=2)
    d["dr_out"] = None
    a, b = run_grad(d, "bf16", 0.7), run_grad(d, "bf16", 0.7)
    check_grad(d, "bf16", 0.7, a)
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.gpu
def test_grad_in_place_and_frozen_weights():
    """dr in place of dr_out, do in place of o, no weight or gate gradients and no workspace."""
    M = lib_m()
    d = inputs(70, 960, "bf16", "token", True, True, seed=4)
    want = run_grad(d, "bf16", 0.7)
    dr, do = d["dr_out"].clone(), d["o"].clone()
    M.moe_block_norm_grad(do, d["r"], M.MPB_BF16, d["gate"], d["gp"], d["gn"], 0.7, EPS, dr, d["dx"], dr, do, None,
                          None, None, None)
    assert torch.equal(dr, want["dr"]) and torch.equal(do, want["do"])
    dr = d["dx"].clone()
    M.moe_block_norm_grad(d["o"], d["r"], M.MPB_BF16, d["gate"], d["gp"], d["gn"], 0.7, EPS, d["dr_out"], dr, dr, None,
                          None, None, None, None)
    assert torch.equal(dr, want["dr"])


@pytest.mark.gpu
@pytest.mark.parametrize("H", [320, 16384, 20480])
def test_grad_in_place_over_many_rows(H):
    """In place with several rows a workgroup, whose loads run ahead."""
    M = lib_m()
    d = inputs(1400, H, "f16", "full", True, True, seed=5)
    want = run_grad(d, "f16", 0.7)
    dr, do = d["dr_out"].clone(), d["o"].clone()
    M.moe_block_norm_grad(do, d["r"], M.MPB_F16, d["gate"], d["gp"], d["gn"], 0.7, EPS, dr, d["dx"], dr, do, None,
                          None, None, None)
    assert torch.equal(dr, want["dr"]) and torch.equal(do, want["do"])


@pytest.mark.gpu
def test_grad_of_an_empty_batch_zeroes_the_weight_gradients():
    M = lib_m()
    z = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(256, device="cuda")
    a, b = torch.full_like(g, 5.0), torch.full_like(g, 5.0)
    ws = torch.empty(M.moe_block_norm_grad_workspace_bytes(0, 256), dtype=torch.uint8, device="cuda")
    M.moe_block_norm_grad(z.float(), z, M.MPB_BF16, None, g, g, 1.0, EPS, z, z, z, z.float(), None, a, b, ws)
    assert not a.any() and not b.any()
    M.moe_block_norm(z.float(), z, M.MPB_BF16, None, g, g, 1.0, EPS, z, z)


@pytest.mark.gpu
def test_stream_and_graph_replays():
    """On another stream, and captured and replayed on changed inputs with eager work between."""
    d, e = (inputs(130, 1408, "bf16", "token", True, True, seed=s) for s in (5, 6))
    want = [(run_fwd(v, "bf16", 0.7), run_grad(v, "bf16", 0.7)) for v in (d, e)]
    M = lib_m()
    st = {k: None if v is None else v.clone() for k, v in d.items()}
    T, H = st["r"].shape
    ws = torch.empty(M.moe_block_norm_grad_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = run_fwd(st, "bf16", 0.7), run_grad(st, "bf16", 0.7, ws=ws)
    s.synchronize()
    assert torch.equal(out[0][0], want[0][0][0]) and torch.equal(out[1]["dgp"], want[0][1]["dgp"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run_fwd(st, "bf16", 0.7), run_grad(st, "bf16", 0.7, ws=ws)
    for k in (0, 1, 0, 1):
        src = (d, e)[k]
        for name, v in st.items():
            if v is not None:
                v.copy_(src[name])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0][0], want[k][0][0]) and torch.equal(out[0][1], want[k][0][1])
        for name in out[1]:
            assert torch.equal(out[1][name], want[k][1][name]), name
        run_grad(e, "bf16", 0.7)


def test_formula_gradients_against_differences():
    """The 64-bit gradients that the kernels are held to, against central differences of the forward formula (CPU)."""
    g = torch.Generator().manual_seed(0)
    T, H, scale = 3, 12, 0.7
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    for gate in (None, rn(T), rn(T, H)):
        v = {"o": rn(T, H), "r": rn(T, H), "gate": gate, "gp": 1 + 0.1 * rn(H), "gn": 1 + 0.1 * rn(H)}
        wr, wx = rn(T, H), rn(T, H)

        def loss(q):
            y, x, _ = forward64(q["o"], q["r"], q["gate"], q["gp"], q["gn"], scale)
            return float((y * wr).sum() + (x * wx).sum())

        y = forward64(v["o"], v["r"], v["gate"], v["gp"], v["gn"], scale)[0]
        got = grad64({**v, "r": y, "dr_out": wr, "dx": wx}, scale)
        for k in v:
            if v[k] is None:
                continue
            way, h = rn(*v[k].shape), 1e-5
            diff = (loss({**v, k: v[k] + h * way}) - loss({**v, k: v[k] - h * way})) / (2 * h)
            want = float((got["d" + k] * way).sum())
            # central differences: h^2 times a third derivative, and rounding over h
            assert abs(diff - want) <= 1e-6 * (1 + abs(want)), k


# ---------------------------------------------------------------- refusals (no GPU needed)
def test_refusals():
    M = lib_m()
    from mixed_precision_bit_amd import _lib
    L = _lib.lib()
    p, odd = ctypes.c_void_p(16), ctypes.c_void_p(8)

    def fwd(o=p, r=p, xd=0, T=4, H=256, gate=None, kind=0, gp=p, gn=p, scale=1.0, eps=1e-6, ro=p, x=p):
        return L.moe_block_norm(o, r, xd, T, H, gate, kind, gp, gn, scale, eps, ro, x, None)

    assert fwd(xd=2) == -1 and "x_dtype" in M.mpb_last_error()
    assert fwd(T=-1) == -1 and fwd(T=(1 << 20) + 1) == -2
    assert fwd(H=0) == -2 and fwd(H=100) == -2 and fwd(H=65600) == -2
    assert fwd(kind=3) == -1 and fwd(kind=1) == -1 and fwd(gate=p) == -1
    assert fwd(scale=float("nan")) == -1 and fwd(eps=0.0) == -1 and fwd(eps=float("inf")) == -1
    assert fwd(r=None) == -1 and fwd(x=None) == -1 and fwd(gn=None) == -1 and fwd(ro=None) == -1 and fwd(o=None) == -1
    assert fwd(o=None, ro=None) == -1                       # gamma_post without o
    assert fwd(o=None, ro=None, gp=None, gn=None, x=None) == -1
    assert fwd(r=odd) == -1 and "aligned" in M.mpb_last_error()
    assert fwd(gate=odd, kind=2) == -1
    assert fwd(T=0, o=None, r=None, ro=None, x=None) == 0

    def bwd(o=p, y=p, xd=0, T=4, H=256, gate=None, kind=0, gp=p, gn=p, dro=p, dx=p, dr=p, do=p, dg=None, dgp=p, dgn=p,
            ws=p, n=1 << 30):
        return L.moe_block_norm_grad(o, y, xd, T, H, gate, kind, gp, gn, 1.0, 1e-6, dro, dx, dr, do, dg, dgp, dgn, ws, n, None)

    assert bwd(xd=-1) == -1 and bwd(H=65) == -2 and bwd(T=-5) == -1
    assert bwd(dx=None) == -1 and bwd(gn=None) == -1 and bwd(gn=None, dx=None) == -1
    assert bwd(gp=None) == -1 and bwd(dg=p) == -1 and bwd(o=None) == -1 and bwd(dr=None) == -1 and bwd(y=None) == -1
    assert bwd(gn=None, dx=None, dgn=None, dro=None) == -1
    assert bwd(ws=None) == -1 and bwd(n=255) == -5 and bwd(do=odd) == -1 and bwd(dgp=odd) == -1
    assert bwd(T=0, dgp=None, dgn=None, ws=None, n=0) == 0
    assert M.moe_block_norm_grad_workspace_bytes(1, 2048) == 2 * 2048 * 4
    assert M.moe_block_norm_grad_workspace_bytes(-1, 2048) == 0 == M.moe_block_norm_grad_workspace_bytes(4, 100)


def test_tensor_refusals():
    """The binding refuses tensors whose type, shape, layout or device the entry would misread."""
    M = lib_m()
    r = torch.zeros(4, 256, dtype=torch.float16)
    o, g = torch.zeros(4, 256), torch.ones(256)

    def code(o=o, r=r, gate=None, gp=g, gn=g, ro=r, x=r, xd=M.MPB_F16):
        with pytest.raises(M.MpbError) as e:
            M.moe_block_norm(o, r, xd, gate, gp, gn, 1.0, 1e-6, ro, x)
        return e.value.code, str(e.value)

    assert "on the CPU" in code()[1]
    assert code(o=o.half())[0] == -1 and code(xd=M.MPB_BF16)[0] == -1 and code(xd=7)[0] == -1
    assert code(o=o[:3])[0] == -2 and code(gp=g[:64])[0] == -2 and code(gate=torch.zeros(5))[0] == -2
    assert "contiguous" in code(o=torch.zeros(256, 4).t())[1]
    assert code(gate=torch.zeros(4, 256))[0] == -1      # a full gate has the activations' type

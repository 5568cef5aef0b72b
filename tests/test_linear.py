"""moe_linear and moe_linear_grad against the formulas in 64 bits.

Tolerances. u = 2^-24 is the fp32 rounding. Products of 16-bit values are exact. A
sum over K terms runs through K / 32 matrix instructions, each of which adds 32
products (within 34 u of their absolute sum, as any order of adding them is), and at
most 16 partial sums of a split reduction: within E(K) = (K / 32 + 64) u of the
terms' absolute sum. An activation has slope at most 1.13 and is itself within
8 u |z| + 16 u |y|: its sigmoid within 6 u, the argument of erfc or of the sigmoid
within 8 u of itself, which changes x f(x) by at most |z| max|x f'(x)| 8 u < 4 u |z|.
Its derivative, a sum of two such terms, is within 32 u (1 + |z|). A value rounded to
a 16-bit type is off by eps / 2 of itself and half the smallest step; dz in one fp16 part by
2^-11 of itself, in two by 2^-22, and by 2^-38 of the largest |dy|, bf16 X and W beside them
by 2^-38 of their largest."""
import math

import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def xd(dt):
    M = lib_m()
    return {"f16": M.MPB_F16, "bf16": M.MPB_BF16, "f32": M.MPB_F32}[dt]


def half_step(dt, v):
    return torch.finfo(dt).eps / 2 * v.abs() + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def E(K):
    return (K / 32 + 64) * U


def act64(z, act):
    """(act, derivative) in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = 2 * math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-a * (z + 0.044715 * z ** 3)))
    return z * s, s + z * s * (1 - s) * a * (1 + 3 * 0.044715 * z * z)


def inputs(T, Kd, N, dt, bias=True, res=None, seed=0, pad=3):
    """Operands of which rows behind the last hold nan: nothing may look at them."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(n, m, std, t):
        v = torch.full((n + pad, m), float("nan"), device="cuda", dtype=t)
        v[:n] = (torch.randn(n, m, generator=g, device="cuda") * std).to(t)
        return v[:n]
    d = {"X": rows(T, Kd, 1.0, DT[dt]), "W": rows(N, Kd, Kd ** -0.5, DT[dt])}
    d["b"] = torch.randn(N, generator=g, device="cuda") if bias else None
    d["res"] = None if res is None else rows(T, N, 1.0, DT[res])
    d["z"], d["g"] = rows(T, N, 1.5, DT[dt]), g
    return d


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


def run_fwd(d, dt, y, act="none", keep=True, stream=None, in_place=False):
    M = lib_m()
    T, Kd, N = *d["X"].shape, d["W"].shape[0]
    big = torch.full((T + 2, N), 7.0, device="cuda", dtype=DT[y])
    z = torch.full((T, N), float("nan"), device="cuda", dtype=DT[dt]) if keep else None
    res = d["res"]
    if in_place:
        big[:T] = res
        res = big[:T]
    ws = torch.empty(M.moe_linear_workspace_bytes(T, Kd, N), dtype=torch.uint8, device="cuda")
    M.moe_linear(d["X"], xd(dt), d["W"], d["b"], ACTS.index(act), res, z, big[:T], ws, stream)
    assert (big[T:] == 7.0).all(), "rows behind the last were written"
    return big[:T], z


def check_fwd(d, dt, y_type, act, y, z):
    X, W = d["X"].double(), d["W"].double()
    ref = X @ W.t()
    tol = E(X.shape[1]) * (X.abs() @ W.abs().t())
    if d["b"] is not None:
        ref = ref + d["b"].double()
        tol = tol + U * (ref.abs() + d["b"].double().abs())
    if z is not None:
        check(z, ref, tol + 1.01 * half_step(DT[dt], ref.abs() + tol), "z")
    a, _ = act64(ref, act)
    if act != "none":
        tol = 1.13 * tol + 8 * U * ref.abs() + 16 * U * a.abs()
    if d["res"] is not None:
        a = a + d["res"].double()
    tol = tol + 2 * U * a.abs()
    check(y, a, tol + (0 if y_type == "f32" else 1.01 * half_step(DT[y_type], a.abs() + tol)), "y")


# few tokens; one tile and edges; split reductions; wide tiles with ragged edges
SHAPES = [(1, 64, 8), (1, 4096, 264), (5, 192, 1000), (16, 2048, 2048), (17, 64, 8), (72, 4096, 520), (129, 320, 264),
          (300, 1024, 136), (1000, 192, 1368), (3001, 128, 4104)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Kd,N", SHAPES)
def test_forward(T, Kd, N, dt):
    d = inputs(T, Kd, N, dt)
    check_fwd(d, dt, dt, "none", *run_fwd(d, dt, dt, keep=False))
    check_fwd(d, dt, "f32", "none", *run_fwd(d, dt, "f32"))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,Kd,N,dt,y", [(3, 128, 72, "f16", "f32"), (200, 1024, 264, "bf16", "bf16"), (3001, 64, 4104, "f16", "f16"),
                                         (300, 64, 520, "bf16", "f32")])
def test_forward_activation_and_residual(T, Kd, N, dt, y, act):
    d = inputs(T, Kd, N, dt, res=y, seed=1)
    d["X"] *= 3  # z up to 12
    check_fwd(d, dt, y, act, *run_fwd(d, dt, y, act))
    a, b = run_fwd(d, dt, y, act), run_fwd(d, dt, y, act, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    d["b"] = None
    check_fwd(d, dt, y, act, *run_fwd(d, dt, y, act, keep=False))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_infinities_stay_in_their_rows(T):
    d = inputs(T, 256, 264, "bf16")
    clean = run_fwd(d, "bf16", "f32")[0].clone()
    d["X"][T - 1, 5] = float("inf")
    d["W"][3, 7] = float("nan")
    y = run_fwd(d, "bf16", "f32")[0]
    assert not y[T - 1].isfinite().any() and y[:, 3].isnan().all()
    keep = [c for c in range(264) if c != 3]
    assert torch.equal(y[:T - 1][:, keep], clean[:T - 1][:, keep])


@pytest.mark.gpu
def test_activations_far_out():
    """Every activation at values up to the type's largest: bias alone, z exact."""
    M = lib_m()
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 6, -6, 13, -13, 30, -30, 90, -90, 3e4, -3e4, 1e18, -1e18, 1e30, -1e30, 3e38, -3e38,
                      1.0, -1.0], device="cuda")
    X, W = torch.zeros(1, 64, device="cuda").bfloat16(), torch.zeros(24, 64, device="cuda").bfloat16()
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    y = torch.empty(1, 24, device="cuda")
    for act in ACTS:
        M.moe_linear(X, M.MPB_BF16, W, z, ACTS.index(act), None, None, y, ws)
        ref = act64(z.double(), act)[0]
        ref = torch.where(ref.isnan(), 0.0, ref)  # -z times e^inf in this formula's 64 bits
        check(y[0], ref, 8 * U * z.double().abs().clamp(max=100) + 64 * U * ref.abs() + 1e-38, act)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ("f16", "bf16"))
def test_gelu_tail(dt):
    """gelu keeps its relative accuracy where Phi is small: the fit 2^-17, fp32's roundings of the
    exponential's argument 2.5 x 2^-24 x a^2 / 2 (below 2^-16 at -12), the result half a step; below the smallest normal number half its last step."""
    M = lib_m()
    N, t = 4096, torch.float16 if dt == "f16" else torch.bfloat16
    z = torch.linspace(-12, 12, N, device="cuda")
    X, W = torch.zeros(1, 64, dtype=t, device="cuda"), torch.zeros(N, 64, dtype=t, device="cuda")
    y = torch.empty(1, N, dtype=t, device="cuda")
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    M.moe_linear(X, xd(dt), W, z, ACTS.index("gelu"), None, None, y, ws)
    ref = act64(z.double().cpu(), "gelu")[0]
    f = torch.finfo(t)
    tol = ref.abs() * (f.eps / 2 + 1.01 * (2.0**-16 + 2.0**-17)) + f.tiny * f.eps / 2
    assert bool(((y[0].double().cpu() - ref).abs() <= tol).all())


# ------------------------------------------------------------------------------------------------ gradients
def run_grad(d, dt, dy, act, stream=None, want=("dX", "dW", "db")):
    M = lib_m()
    T, Kd, N = *d["X"].shape, d["W"].shape[0]
    nan = lambda *s, t=torch.float32: torch.full(s, float("nan"), device="cuda", dtype=t)  # noqa: E731
    big = torch.full((T + 2, Kd), 7.0, device="cuda", dtype=DT[dt])
    out = {"dX": big[:T], "dW": nan(N, Kd), "db": nan(N)}
    out = {k: v if k in want else None for k, v in out.items()}
    dyt = xd("f32" if dy.dtype is torch.float32 else dt)
    ws = torch.empty(M.moe_linear_grad_workspace_bytes(T, Kd, N, ACTS.index(act), dyt), dtype=torch.uint8, device="cuda")
    M.moe_linear_grad(d["X"] if "dW" in want else d["X"], xd(dt), d["W"], ACTS.index(act), None if act == "none" else d["z"], dy,
                      out["dX"], out["dW"], out["db"], ws, stream)
    assert (big[T:] == 7.0).all(), "rows behind the last were written"
    return out


def check_grad(d, dt, dy, act, out):
    X, W = d["X"].double(), d["W"].double()
    T, N = X.shape[0], W.shape[0]
    z = d["z"].double()
    dz = dy.double() * (act64(z, act)[1] if act != "none" else 1)
    own = dy.double().abs() * 32 * U * (1 + z.abs()) if act != "none" else torch.zeros_like(dz)  # dz's own error
    own = own + U * dz.abs()
    formed = act != "none" or dy.dtype is torch.float32
    floor = 2.0 ** -38 * dy.double().abs().max() if formed and T else 0.0
    hi = own + (1.01 * 2.0 ** -11 * dz.abs() + floor if formed else 0)
    both = own + (1.01 * 2.0 ** -22 * dz.abs() + floor if formed else 0)
    x_off, w_off = (2.0 ** -38 * v.abs().max() if formed and dt == "bf16" and T else 0.0 for v in (X, W))
    if out["dX"] is not None:
        ref = dz @ W
        tol = (hi + E(N) * dz.abs()) @ W.abs() + w_off * dz.abs().sum(1)[:, None]
        check(out["dX"], ref, tol + 1.01 * half_step(DT[dt], ref.abs() + tol), "dX")
    if out["dW"] is not None:
        check(out["dW"], dz.t() @ X, (both + E(2 * T) * dz.abs()).t() @ X.abs() + x_off * dz.abs().sum(0)[:, None] + 1e-44, "dW")
    if out["db"] is not None:
        # a group of rows is summed in 4 chains, the groups in 4 chains: T / 4 additions at most, and a few
        check(out["db"], dz.sum(0), (own + (T / 4 + 16) * U * dz.abs()).sum(0) + 1e-44, "db")


GRADS = [(1, 64, 8), (7, 192, 1000), (72, 2048, 264), (200, 2048, 520), (1000, 128, 1368), (3001, 320, 264), (2999, 4160, 2824)]


def gradient_of(T, N, dt, g, std=0.1):
    v = torch.full((T + 3, N), float("nan"), device="cuda", dtype=DT[dt])
    v[:T] = (torch.randn(T, N, generator=g, device="cuda") * std).to(DT[dt])
    return v[:T]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Kd,N", GRADS)
def test_gradients(T, Kd, N, dt):
    d = inputs(T, Kd, N, dt, seed=2)
    dy = gradient_of(T, N, dt, d["g"])
    check_grad(d, dt, dy, "none", run_grad(d, dt, dy, "none"))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,Kd,N,dt,dyt", [(5, 64, 72, "f16", "f16"), (300, 320, 264, "bf16", "bf16"), (1001, 192, 136, "f16", "f32"),
                                           (130, 64, 1000, "bf16", "f32"), (2999, 4160, 2824, "bf16", "bf16")])
def test_gradients_through_an_activation(T, Kd, N, dt, dyt, act):
    d = inputs(T, Kd, N, dt, seed=3)
    dy = gradient_of(T, N, dyt, d["g"])
    check_grad(d, dt, dy, act, run_grad(d, dt, dy, act))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [33, 1025, 2017, 4097])
def test_gradients_of_one_token_past_a_stage(T):
    """Reductions that end one index into a stage of 32, once and in the middle of two parts."""
    for Kd, N in ((128, 264), (4160, 2824)) if T == 4097 else ((128, 264),):
        d = inputs(T, Kd, N, "bf16", seed=12)
        dy = gradient_of(T, N, "bf16", d["g"])
        for act in ("none", "silu"):
            check_grad(d, "bf16", dy, act, run_grad(d, "bf16", dy, act))


@pytest.mark.gpu
@pytest.mark.parametrize("std", [1e-9, 1e-30, 1e5])
def test_gradients_out_of_range_of_fp16(std):
    """fp32 gradients of a mean over a batch, and a large loss scale: dW and dbias keep their bits."""
    d = inputs(333, 128, 264, "f16", seed=4)
    dy = gradient_of(333, 264, "f32", d["g"], std)
    check_grad(d, "f16", dy, "none", run_grad(d, "f16", dy, "none", want=("dW", "db")))
    dy.zero_()
    out = run_grad(d, "f16", dy, "none")
    assert not out["dX"].any() and not out["dW"].any() and not out["db"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("want", [("dX",), ("dW",), ("db",), ("dW", "db")])
def test_single_gradients_match(want):
    d = inputs(150, 128, 264, "bf16", seed=5)
    for act, dyt in (("silu", "bf16"), ("none", "bf16"), ("none", "f32")):
        dy = gradient_of(150, 264, dyt, d["g"])
        whole, part = run_grad(d, "bf16", dy, act), run_grad(d, "bf16", dy, act, want=want)
        for k in want:
            assert torch.equal(whole[k], part[k])


@pytest.mark.gpu
def test_gradients_are_those_of_differences():
    """dX and dW against central differences of the 64-bit loss sum(y * dy)."""
    d = inputs(9, 64, 40, "bf16", seed=6)
    X, W, b = d["X"].double(), d["W"].double(), d["b"].double()
    dy = gradient_of(9, 40, "f32", d["g"], 1.0)
    h = 2.0 ** -12
    for act in ("silu", "gelu", "gelu_tanh"):
        d["z"] = (X @ W.t() + b).bfloat16()
        out = run_grad(d, "bf16", dy, act)
        loss = lambda X, W: float((act64(X @ W.t() + b, act)[0] * dy.double()).sum())  # noqa: E731
        for t, i, k in ((0, 3, "dX"), (8, 63, "dX"), (1, 2, "dW"), (39, 60, "dW")):
            A = (X if k == "dX" else W).clone()
            A[t, i] += h
            up = loss(A, W) if k == "dX" else loss(X, A)
            A[t, i] -= 2 * h
            down = loss(A, W) if k == "dX" else loss(X, A)
            want, got = (up - down) / (2 * h), float(out[k][t, i])
            # z is kept to 8 bits, |act''| < 1.2: up to 2^-9 |z| 1.2 |dy| |w| a term; differences of order h^2
            other = (W[:, i] if k == "dX" else X[:, i]).abs()
            term = (dy.double()[t] if k == "dX" else dy.double()[:, t]).abs() * other
            zt = (d["z"].double()[t] if k == "dX" else d["z"].double()[:, t]).abs()
            tol = float((term * (1.2 * 2 ** -9 * zt + 2 ** -8)).sum()) + 1e-5 + abs(want) * 2 ** -8
            assert abs(got - want) <= tol, (act, k, t, i, got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_operands_of_many_magnitudes(dt):
    """Rows of X, W and dy spread over orders of magnitude: the scales of the fp16 parts follow the largest."""
    d = inputs(200, 256, 264, dt, seed=9)
    spread = lambda n: 10.0 ** torch.linspace(-3, 2 if dt == "f16" else 8, n, device="cuda")[torch.randperm(n, device="cuda")]  # noqa: E731
    d["X"] *= spread(200)[:, None]
    d["W"] *= spread(264)[:, None]
    dy = gradient_of(200, 264, "f32", d["g"], 1.0) * spread(200)[:, None]
    if dt == "f16":
        dy *= 2.0 ** -12  # dX stays in range
    for act in ("none", "silu"):
        check_grad(d, dt, dy, act, run_grad(d, dt, dy, act))


@pytest.mark.gpu
def test_infinite_gradients_reach_what_they_touch_and_no_more():
    d = inputs(150, 128, 264, "bf16", seed=10)
    dy = gradient_of(150, 264, "bf16", d["g"])
    clean = run_grad(d, "bf16", dy, "silu")
    dy = dy.clone()
    dy[7, 9] = float("inf")
    d["z"][7, 9] = 1.0
    out = run_grad(d, "bf16", dy, "silu")
    rows = [t for t in range(150) if t != 7]
    assert not out["dX"][7].isfinite().any() and out["dX"][rows].isfinite().all()
    assert not out["dW"][9].isfinite().any() and out["db"][9] == float("inf")
    cols = [c for c in range(264) if c != 9]
    assert torch.equal(out["dW"][cols], clean["dW"][cols]) and torch.equal(out["dX"][rows], clean["dX"][rows])


@pytest.mark.gpu
def test_raw_bits():
    M = lib_m()
    d = inputs(20, 128, 72, "bf16", seed=11)
    want = run_fwd(d, "bf16", "bf16", "gelu")
    i = torch.int16
    y, z = torch.zeros(20, 72, dtype=i, device="cuda"), torch.zeros(20, 72, dtype=i, device="cuda")
    M.moe_linear(d["X"].view(i), M.MPB_BF16, d["W"].view(i), d["b"], M.MPB_ACT_GELU, None, z, y, torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert torch.equal(y.view(torch.bfloat16), want[0]) and torch.equal(z.view(torch.bfloat16), want[1])


@pytest.mark.gpu
def test_empty_batches():
    M = lib_m()
    d = inputs(0, 128, 72, "f16")
    run_fwd(d, "f16", "f16")
    out = run_grad(d, "f16", gradient_of(0, 72, "f16", d["g"]), "none")
    assert not out["dW"].any() and not out["db"].any()
    out = run_grad(d, "f16", gradient_of(0, 72, "f32", d["g"]), "silu")
    assert not out["dW"].any() and not out["db"].any()
    assert M.moe_linear_workspace_bytes(0, 128, 72) > 0


@pytest.mark.gpu
def test_repeats_are_equal():
    for T, Kd, N in ((72, 4096, 520), (3001, 128, 4104)):
        d = inputs(T, Kd, N, "bf16", seed=7)
        dy = gradient_of(T, N, "bf16", d["g"])
        a, b = run_fwd(d, "bf16", "f32", "silu"), run_fwd(d, "bf16", "f32", "silu")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        a, b = run_grad(d, "bf16", dy, "silu"), run_grad(d, "bf16", dy, "silu")
        assert all(torch.equal(a[k], b[k]) for k in a)


# ------------------------------------------------------------------------------------------------ refusals
def refused(code, f, *args):
    M = lib_m()
    with pytest.raises(M.MpbError) as e:
        f(*args)
    assert e.value.code == code, str(e.value)


def test_refusals():
    M = lib_m()
    h = lambda *s: torch.zeros(*s).bfloat16()  # noqa: E731
    X, W, b, y, ws = h(4, 128), h(16, 128), torch.zeros(16), h(4, 16), torch.zeros(1 << 20, dtype=torch.uint8)
    bf = M.MPB_BF16
    for args in ((None, bf, W, b, 0, None, None, y, ws), (X, bf, None, b, 0, None, None, y, ws), (X, bf, W, b, 0, None, None, None, ws),
                 (X, 5, W, b, 0, None, None, y, ws), (X, M.MPB_F32, W, b, 0, None, None, y, ws), (X, M.MPB_F16, W, b, 0, None, None, y, ws),
                 (X, bf, W, b.double(), 0, None, None, y, ws), (X, bf, W, b, 0, torch.zeros(4, 16), None, y, ws),
                 (X, bf, W, b, 0, None, torch.zeros(4, 16), y, ws), (X.t().contiguous().t(), bf, W, b, 0, None, None, y, ws)):
        refused(-1, M.moe_linear, *args)
    for args in ((h(4, 64), bf, W, b, 0, None, None, y, ws), (X, bf, W, b[:8], 0, None, None, y, ws), (X, bf, W, b, 0, None, None, h(4, 24), ws),
                 (X, bf, h(16, 2, 64), b, 0, None, None, y, ws)):
        refused(-2, M.moe_linear, *args)
    for args in ((None, bf, W, 0, None, y, X, None, None, ws), (X, bf, W, 0, None, None, X, None, None, ws)):
        refused(-1, M.moe_linear_grad, *args)
    refused(-2, M.moe_linear_grad, X, bf, W, 0, None, y, X, torch.zeros(16, 64), None, ws)


def test_refusals_of_the_library():
    """The C entries themselves: validation precedes everything, so no device is needed."""
    M = lib_m()
    L = M._lib.lib()
    p, odd, big = 4096, 4104, 1 << 40
    bf = M.MPB_BF16

    def fwd(X=p, xt=bf, W=p, b=None, act=0, res=None, T=4, Kd=128, N=16, z=None, y=p, yt=bf, ws=p, n=big):
        return L.moe_linear(X, xt, W, b, act, res, T, Kd, N, z, y, yt, ws, n, None)

    def bwd(X=p, xt=bf, W=p, act=0, z=None, dy=p, dt=bf, T=4, Kd=128, N=16, dX=p, dW=p, db=p, ws=p, n=big):
        return L.moe_linear_grad(X, xt, W, act, z, dy, dt, T, Kd, N, dX, dW, db, ws, n, None)
    for f in (fwd, bwd):
        assert f(xt=2) == -1 and f(xt=-1) == -1 and f(act=5) == -1 and f(act=-1) == -1 and f(T=-1) == -1
        assert f(T=(1 << 20) + 1) == -2 and f(Kd=96) == -2 and f(Kd=0) == -2 and f(Kd=65600) == -2
        assert f(N=12) == -2 and f(N=0) == -2 and f(N=524296) == -2
        assert f(X=odd) == -1 and f(W=odd) == -1 and f(ws=None) == -1 and f(ws=odd) == -1
    assert fwd(X=None) == -1 and fwd(W=None) == -1 and fwd(y=None) == -1 and fwd(yt=M.MPB_F16) == -1
    assert fwd(b=odd) == -1 and fwd(res=odd) == -1 and fwd(z=odd) == -1 and fwd(y=odd) == -1
    assert fwd(T=72, Kd=4096, N=16, n=M.moe_linear_workspace_bytes(72, 4096, 16) - 1) == -5
    assert fwd(T=0, X=None, W=None, y=None) == 0
    assert bwd(dX=None, dW=None, db=None) == -1 and bwd(dy=None) == -1 and bwd(W=None) == -1 and bwd(X=None) == -1
    assert bwd(act=2) == -1 and bwd(dt=M.MPB_F16) == -1 and bwd(dX=odd) == -1 and bwd(dW=odd) == -1 and bwd(db=odd) == -1
    assert bwd(n=M.moe_linear_grad_workspace_bytes(4, 128, 16, 0, bf) - 1) == -5
    assert bwd(T=0, dW=None, db=None) == 0
    assert M.moe_linear_workspace_bytes(4, 100, 16) == 0 and M.moe_linear_grad_workspace_bytes(4, 128, 16, 9, bf) == 0
    assert "moe_linear" in M.mpb_last_error()

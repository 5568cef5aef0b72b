"""moe_head_norm and moe_head_norm_grad against the formulas in 64 bits.

Tolerances. u = 2^-24 is the fp32 rounding. A head's sum of squares adds 16 terms in a
lane and at most 5 times over lanes: within 24 u, its reciprocal root within 16 u;
with two products a normed element is within N = 20 u of itself. An angle in turns is
within 2^-25 turns for the positions here, cos and sin then within 8 u (absolute); a
rotated element within |(a, b)| (N + 12 u). Backward: the rotated gradient within R = 12 u
of its pair; the head's mean of products within 60 u of its terms' absolute sum. dgamma
sums T H terms, each within 80 u of its own magnitude, in chains of at most T H / 4 + 100
additions. A stored 16-bit value adds eps / 2 of itself and half the smallest step."""
import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
EPS = 1e-6
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def half_step(dt, v):
    return torch.finfo(dt).eps / 2 * v.abs() + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def inputs(T, Hq, Hk, D, Dr, dt, A=1, norm=True, pairs=0, seed=0, far=1 << 20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = {"qkv": (1.5 * rn(T, Hq + 2 * Hk, D)).to(DT[dt]), "dq": rn(T, Hq, D).to(DT[dt]), "dk": rn(T, Hk, D).to(DT[dt]), "pairs": pairs}
    d["q"], d["k"] = d["qkv"][:, :Hq], d["qkv"][:, Hq:Hq + Hk]
    d["gq"], d["gk"] = (1 + 0.1 * rn(D), 1 + 0.1 * rn(D)) if norm else (None, None)
    d["pos"] = d["axis"] = d["freq"] = None
    if Dr:
        d["pos"] = torch.randint(-far, far, (A, T), generator=g, device="cuda", dtype=torch.int32)
        if T:
            d["pos"][:, 0] = 0
        d["axis"] = torch.randint(0, A, (Dr // 2,), generator=g, device="cuda", dtype=torch.int32) if A > 1 else None
        d["freq"] = (1e4 ** (-torch.arange(Dr // 2, device="cuda") * 2.0 / Dr)).contiguous()
    return d


def angles(d):
    if d["freq"] is None:
        return None
    A = d["pos"].shape[0]
    axis = d["axis"].long() if d["axis"] is not None else torch.zeros(d["freq"].shape[0], dtype=torch.long, device="cuda")
    ok = (axis >= 0) & (axis < A)
    a = d["pos"].double()[axis.clamp(0, A - 1)].t() * d["freq"].double() * ok
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def split(v, d):
    n = d["freq"].shape[0]
    return (v[..., :n], v[..., n:2 * n]) if d["pairs"] == 0 else (v[..., 0:2 * n:2], v[..., 1:2 * n:2])


def put(v, a, b, d):
    n, out = d["freq"].shape[0], v.clone()
    if d["pairs"] == 0:
        out[..., :n], out[..., n:2 * n] = a, b
    else:
        out[..., 0:2 * n:2], out[..., 1:2 * n:2] = a, b
    return out


def turn(v, d, back=False):
    """(rotated, the magnitude of each element's pair)."""
    if d["freq"] is None:
        return v, v.abs()
    c, s = angles(d)
    s = -s if back else s
    a, b = split(v, d)
    m = (a * a + b * b).sqrt()
    return put(v, a * c - b * s, a * s + b * c, d), put(v.abs(), m, m, d)


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


def rot(d):
    return d["pos"], d["axis"], d["freq"], d["pairs"]


def run_fwd(d, dt, q=None, k=None, stream=None):
    M = lib_m()
    T, Hk = d["q"].shape[0], d["k"].shape[1]
    nan = lambda v: torch.full(v.shape, float("nan"), device="cuda", dtype=v.dtype)  # noqa: E731
    q, k = nan(d["q"]) if q is None else q, (nan(d["k"]) if k is None else k) if Hk else None
    M.moe_head_norm(d["q"], d["k"] if Hk else None, M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["gq"], d["gk"], EPS, *rot(d), q, k, stream)
    return q, k


def check_fwd(d, dt, q, k):
    for x, g, got, what in ((d["q"], d["gq"], q, "q"), (d["k"], d["gk"], k, "k")):
        if got is None:
            continue
        x = x.double()
        n = x if g is None else x / (x.square().mean(2, keepdim=True) + EPS).sqrt() * g.double()
        ref, m = turn(n, d)
        tol = m * 32 * U
        check(got, ref, tol + 1.01 * half_step(DT[dt], ref.abs() + tol), what)


# heads of one lane's 16 elements to 512, partial rotations, more heads than a wave holds
SHAPES = [(1, 4, 1, 64, 64), (3, 1, 0, 16, 16), (33, 5, 3, 32, 16), (64, 16, 16, 128, 128), (130, 32, 8, 128, 64), (9, 6, 2, 96, 96),
          (17, 3, 1, 80, 32), (40, 4, 2, 256, 256), (5, 2, 2, 512, 128), (7, 9, 1, 176, 0), (1000, 7, 1, 48, 48), (2500, 3, 2, 64, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("T,Hq,Hk,D,Dr", SHAPES)
def test_forward(T, Hq, Hk, D, Dr, pairs, dt):
    for norm in (True, False):
        d = inputs(T, Hq, Hk, D, Dr, dt, A=3 if Dr > 16 else 1, norm=norm, pairs=pairs)
        check_fwd(d, dt, *run_fwd(d, dt))


@pytest.mark.gpu
def test_forward_in_place_and_strided():
    d = inputs(50, 8, 2, 128, 128, "bf16", A=2)
    want = run_fwd(d, "bf16")
    before = d["qkv"].clone()
    wide = torch.full((50, 9, 128), 7.0, device="cuda").bfloat16()
    q, k = run_fwd(d, "bf16", q=wide[:, :8])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and (wide[:, 8] == 7.0).all()
    run_fwd(d, "bf16", q=d["q"], k=d["k"])  # the packed projection itself, its value heads left as they were
    assert torch.equal(d["q"], want[0]) and torch.equal(d["k"], want[1]) and torch.equal(d["qkv"][:, 10:], before[:, 10:])


@pytest.mark.gpu
def test_one_side_without_norm_and_axes_out_of_range():
    d = inputs(20, 4, 2, 64, 64, "f16", A=2)
    d["gk"] = None
    check_fwd(d, "f16", *run_fwd(d, "f16"))
    d["axis"][3], d["axis"][4] = -1, 2  # these pairs are not turned
    check_fwd(d, "f16", *run_fwd(d, "f16"))


@pytest.mark.gpu
@pytest.mark.parametrize("far", [1 << 24, (1 << 31) - 1])
def test_far_positions(far):
    """Angles of far positions: 64-bit products keep 2^-24 of a turn, 2 pi 2^-24 of the pair's magnitude."""
    d = inputs(64, 2, 1, 64, 64, "f16", far=far)
    q, k = run_fwd(d, "f16")
    for x, g, got in ((d["q"], d["gq"], q), (d["k"], d["gk"], k)):
        x = x.double()
        ref, m = turn(x / (x.square().mean(2, keepdim=True) + EPS).sqrt() * g.double(), d)
        # the reference's own cos reduces an angle rounded at 2^-53 of up to 2^31
        check(got, ref, m * (32 * U + 4 * 6.3 * U) + 1.01 * half_step(DT["f16"], m), "far")


@pytest.mark.gpu
def test_zero_and_infinite_heads():
    d = inputs(4, 4, 1, 64, 64, "bf16")
    d["q"][1, 2] = 0
    clean = run_fwd(d, "bf16")
    assert (clean[0][1, 2] == 0).all()
    d["q"][2, 1, 5] = float("inf")
    q, _ = run_fwd(d, "bf16")
    keep = torch.ones(4, 4, dtype=torch.bool)
    keep[2, 1] = False
    assert torch.equal(q[keep.cuda()], clean[0][keep.cuda()]) and q[2, 1].isnan().any()


# ------------------------------------------------------------------------------------------------ gradients
def run_grad(d, dt, stream=None, in_place=False):
    M = lib_m()
    T, Hq, D = d["q"].shape
    Hk = d["k"].shape[1]
    nan = lambda *s, t=torch.float32: torch.full(s, float("nan"), device="cuda", dtype=t)  # noqa: E731
    dq, dk = (d["dq"].clone(), d["dk"].clone()) if in_place else (nan(T, Hq, D, t=DT[dt]), nan(T, Hk, D, t=DT[dt]))
    gi, gk = (dq, dk) if in_place else (d["dq"], d["dk"])
    out = {"q": dq, "k": dk if Hk else None, "gq": None if d["gq"] is None else nan(D), "gk": None if d["gk"] is None or not Hk else nan(D)}
    ws = torch.empty(M.moe_head_norm_grad_workspace_bytes(T, Hq, Hk, D), dtype=torch.uint8, device="cuda")
    M.moe_head_norm_grad(None if d["gq"] is None else d["q"], None if d["gk"] is None or not Hk else d["k"],
                         M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["gq"], d["gk"], EPS, *rot(d), gi, gk if Hk else None, out["q"], out["k"],
                         out["gq"], out["gk"], ws, stream)
    return out


def check_grad(d, dt, out):
    for x, g, do, got, gg, what in ((d["q"], d["gq"], d["dq"], out["q"], out["gq"], "q"), (d["k"], d["gk"], d["dk"], out["k"], out["gk"], "k")):
        if got is None:
            continue
        x = x.double()
        n, m = turn(do.double(), d, back=True)
        tol = 12 * U * m
        if g is None:
            check(got, n, tol + 1.01 * half_step(DT[dt], n.abs() + tol), "d" + what)
            continue
        g = g.double()
        r = 1 / (x.square().mean(2, keepdim=True) + EPS).sqrt()
        xh, a = x * r, n * g
        ref = r * (a - xh * (a * xh).mean(2, keepdim=True))
        spread = (m * g).abs() + xh.abs() * ((m * g).abs() * xh.abs()).mean(2, keepdim=True)
        tol = r * spread * 100 * U
        check(got, ref, tol + 1.01 * half_step(DT[dt], ref.abs() + tol), "d" + what)
        terms = m * xh.abs()
        n_add = x.shape[0] * x.shape[1] / 4 + 100
        check(gg, (n * xh).sum((0, 1)), (80 + n_add) * U * terms.sum((0, 1)) + 1e-40, "dgamma_" + what)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("T,Hq,Hk,D,Dr", SHAPES)
def test_gradients(T, Hq, Hk, D, Dr, pairs, dt):
    for norm in (True, False):
        d = inputs(T, Hq, Hk, D, Dr, dt, A=2 if Dr > 16 else 1, norm=norm, pairs=pairs, seed=1)
        out = run_grad(d, dt)
        check_grad(d, dt, out)
        again = run_grad(d, dt, in_place=True)
        assert all(torch.equal(out[k], again[k]) for k in out if out[k] is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("side", ["gq", "gk"])
def test_gradients_with_a_norm_on_one_side(side):
    d = inputs(70, 5, 3, 96, 64, "bf16", A=2, seed=4)
    d[side] = None
    out = run_grad(d, "bf16")
    check_grad(d, "bf16", out)
    assert out[side] is None


@pytest.mark.gpu
def test_many_heads_and_raw_bits():
    """1024 query heads, and activations handed over as int16 bits."""
    M = lib_m()
    d = inputs(3, 1024, 1, 32, 32, "f16", seed=5)
    want = run_fwd(d, "f16")
    check_fwd(d, "f16", *want)
    check_grad(d, "f16", run_grad(d, "f16"))
    q, k = torch.zeros(3, 1024, 32, dtype=torch.int16, device="cuda"), torch.zeros(3, 1, 32, dtype=torch.int16, device="cuda")
    M.moe_head_norm(d["q"].view(torch.int16), d["k"].view(torch.int16), M.MPB_F16, d["gq"], d["gk"], EPS, *rot(d), q, k)
    assert torch.equal(q.view(torch.float16), want[0]) and torch.equal(k.view(torch.float16), want[1])


@pytest.mark.gpu
def test_gradients_are_those_of_differences():
    d = inputs(3, 2, 1, 32, 16, "bf16", seed=2)
    out, h = run_grad(d, "bf16"), 2.0 ** -12

    def loss(x, g):
        n = x / (x.square().mean(2, keepdim=True) + EPS).sqrt() * g
        return float((turn(n, d)[0] * d["dq"].double()).sum())
    x, g = d["q"].double(), d["gq"].double()
    for t, hd, i in ((0, 0, 0), (1, 1, 9), (2, 0, 20), (2, 1, 31)):
        a, b = x.clone(), x.clone()
        a[t, hd, i] += h
        b[t, hd, i] -= h
        want = (loss(a, g) - loss(b, g)) / (2 * h)
        assert abs(float(out["q"][t, hd, i]) - want) <= 2 ** -8 * abs(want) + 1e-4
    for i in (0, 7, 31):
        a, b = g.clone(), g.clone()
        a[i] += h
        b[i] -= h
        want = (loss(x, a) - loss(x, b)) / (2 * h)
        assert abs(float(out["gq"][i]) - want) <= 1e-5 * max(1, abs(want))


@pytest.mark.gpu
def test_empty_batch_zeroes_the_gammas():
    d = inputs(0, 4, 2, 64, 64, "f16")
    run_fwd(d, "f16")
    out = run_grad(d, "f16")
    assert not out["gq"].any() and not out["gk"].any()


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals():
    M = lib_m()
    bf, h = M.MPB_BF16, lambda *s: torch.zeros(*s).bfloat16()  # noqa: E731
    q, k, g = h(4, 3, 64), h(4, 1, 64), torch.ones(64)
    pos, freq, ax = torch.zeros(1, 4, dtype=torch.int32), torch.ones(32), torch.zeros(32, dtype=torch.int32)

    def refused(code, *args):
        with pytest.raises(M.MpbError) as e:
            M.moe_head_norm(*args)
        assert e.value.code == code, str(e.value)
    ok = dict(q=q, k=k, t=bf, gq=g, gk=g, eps=EPS, pos=pos, axis=ax, freq=freq, pairs=0, qo=q, ko=k)
    call = lambda **kw: tuple({**ok, **kw}.values())  # noqa: E731
    refused(-1, *call(q=None))
    refused(-1, *call(t=9))
    refused(-1, *call(q=q.float()))
    refused(-1, *call(pos=pos.long()))
    refused(-1, *call(axis=ax.long()))
    refused(-1, *call(q=h(4, 64, 3).transpose(1, 2)))
    refused(-1, *call(q=q[:1].expand(4, 3, 64)))
    refused(-1, *call(freq=None))
    refused(-1, *call(qo=q.float()))
    refused(-2, *call(q=q[0]))
    refused(-2, *call(gq=torch.ones(32)))
    refused(-2, *call(pos=pos[:, :2]))
    refused(-2, *call(pos=None))
    refused(-2, *call(axis=ax[:8]))
    refused(-2, *call(ko=h(4, 2, 64)))
    with pytest.raises(M.MpbError) as e:
        M.moe_head_norm_grad(q, k, bf, g, g, EPS, pos, ax, freq, 0, None, k, q, k, None, None, None)
    assert e.value.code == -1


def test_refusals_of_the_library():
    M = lib_m()
    L = M._lib.lib()
    p, odd = 4096, 4104

    def fwd(q=p, qs=512, k=p, ks=512, xt=1, T=4, Hq=4, Hk=2, D=64, gq=p, gk=p, eps=1e-6, pos=p, A=1, axis=None, freq=p, Dr=64, pairs=0,
            qo=p, qos=512, ko=p, kos=512):
        return L.moe_head_norm(q, qs, k, ks, xt, T, Hq, Hk, D, gq, gk, eps, pos, A, axis, freq, Dr, pairs, qo, qos, ko, kos, None)

    def bwd(q=p, qs=512, k=p, ks=512, xt=1, T=4, Hq=4, Hk=2, D=64, gq=p, gk=p, eps=1e-6, pos=p, A=1, axis=None, freq=p, Dr=64, pairs=0,
            qo=p, qos=512, ko=p, kos=512, dq=p, dqs=512, dk=p, dks=512, dgq=p, dgk=p, ws=p, n=1 << 40):
        return L.moe_head_norm_grad(q, qs, k, ks, xt, T, Hq, Hk, D, gq, gk, eps, pos, A, axis, freq, Dr, pairs, qo, qos, ko, kos, dq, dqs,
                                    dk, dks, dgq, dgk, ws, n, None)
    for f in (fwd, bwd):
        assert f(xt=2) == -1 and f(T=-1) == -1 and f(eps=0.0) == -1 and f(eps=float("nan")) == -1 and f(pairs=2) == -1
        assert f(T=(1 << 20) + 1) == -2 and f(Hq=0) == -2 and f(Hq=1025) == -2 and f(Hk=-1) == -2
        assert f(D=24) == -2 and f(D=528) == -2 and f(Dr=80) == -2 and f(Dr=8) == -2 and f(Dr=-16) == -2 and f(A=0) == -2 and f(A=9) == -2
        assert f(freq=None) == -1 and f(pos=None) == -1 and f(freq=odd) == -1 and f(axis=odd) == -1 and f(gq=odd) == -1
        assert f(qs=248) == -2 and f(qs=257) == -2 and f(ks=120) == -2 and f(qos=100) == -2 and f(kos=0) == -2 and f(qs=1 << 41) == -2
        assert f(q=odd) == -1 and f(k=odd) == -1 and f(qo=odd) == -1 and f(ko=odd) == -1
        assert f(q=None) == -1 and f(k=None) == -1 and f(qo=None) == -1 and f(ko=None) == -1
    assert fwd(T=0, q=None, k=None, qo=None, ko=None, pos=None) == 0
    assert bwd(dq=None) == -1 and bwd(dk=None) == -1 and bwd(dq=odd) == -1 and bwd(dks=8) == -2 and bwd(ws=None) == -1 and bwd(ws=odd) == -1
    assert bwd(gq=None) == -1 and bwd(gk=None) == -1  # a gradient of a gamma that is not there
    assert bwd(n=M.moe_head_norm_grad_workspace_bytes(4, 4, 2, 64) - 1) == -5
    assert bwd(T=0, dgq=None, dgk=None) == 0
    assert M.moe_head_norm_grad_workspace_bytes(4, 4, 2, 60) == 0

"""moe_distill_loss and moe_distill_loss_grad against the formulas in 64 bits.

Tolerances. u = 2^-24 is the fp32 rounding. The exponent (s - max) log2(e) / tau is off by
at most 3 u of itself; terms with an exponent above 24 do not count in an fp32 sum, so
every term that does is within 24 * 3 u ln 2 + 4 u < 60 u of itself, and a sum of up to
400000 terms over 256 threads at least adds at most 1600 terms in one thread, pairs of them 8
at a time: 200 + 8 + 10 + 16 additions, 240 u: the sums are within 300 u, log p within
300 u absolute, and kl, whose sums over the entries are in 64 bits, within 300 u (Q + q_r)
and its own rounding. A gradient element is within (3 u x + 4 u + 300 u) of p_v Q and q_v
each, x = |s - max| / tau."""
import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def sd(dt):
    M = lib_m()
    return {"f16": M.MPB_F16, "bf16": M.MPB_BF16, "f32": M.MPB_F32}[dt]


def half_step(dt, v):
    if dt is torch.float32:
        return 2 * U * v.abs() + 1e-44
    return torch.finfo(dt).eps / 2 * v.abs() + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def inputs(T, V, k, dt, rest, tau=1.0, seed=0, masked=True, stride=0, shift=0):
    """stride: elements between rows beyond V; shift: elements before the first row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = {"ids": torch.stack([torch.randperm(V, generator=g, device="cuda")[:k] for _ in range(T)]).int() if T else torch.zeros(0, k, dtype=torch.int32, device="cuda")}
    d["y"] = 6 + 1.5 * rn(T, k)
    S = 2 * rn(T, V)
    S.scatter_(1, d["ids"].long(), d["y"] + rn(T, k))
    ld = V + stride
    buf = torch.full((T * ld + shift + 64,), float("nan"), device="cuda", dtype=DT[dt])
    d["buf"], d["S"] = buf, torch.as_strided(buf, (T, V), (ld, 1), shift)
    d["S"].copy_(S)
    d["lse"] = torch.logsumexp(d["y"].double() / tau, 1).float() + 0.2 + 0.1 * rn(T).abs() if rest else None
    d["w"] = torch.rand(T, generator=g, device="cuda") + 0.1 if masked else None
    if masked and T > 2:
        d["w"][1] = 0
    d["tau"] = tau
    return d


def like(d):
    v = torch.full_like(d["buf"], 7.0)
    T, V = d["S"].shape
    return v, torch.as_strided(v, (T, V), d["S"].stride(), d["S"].storage_offset())


def outs(T):
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    return nan(T, 4), nan(T), nan(1)


def call(d, dt, dS=None, gloss=None, stream=None):
    M = lib_m()
    stats, kl, loss = outs(d["S"].shape[0])
    M.moe_distill_loss(d["S"], sd(dt), d["ids"], d["y"], d["lse"], d["w"], d["tau"], stats, kl, loss, dS, gloss, stream)
    return stats, kl, loss


def formula(d):
    """(kl, unweighted gradient over tau, p Q, dense q, the student's log probabilities)."""
    S, ids, y, tau = d["S"].double(), d["ids"].long(), d["y"].double(), d["tau"]
    T, V = S.shape
    live = (ids >= 0) & (ids < V)
    y = torch.where(live, y / tau, -torch.inf)
    lse = d["lse"].double()[:, None] if d["lse"] is not None else torch.logsumexp(y, 1, keepdim=True)
    q_e = torch.where(live & (y > -torch.inf), torch.exp(y - lse), 0.0)
    q = torch.zeros(T, V, dtype=torch.float64, device="cuda").scatter_add_(1, ids.clamp(0, V - 1), q_e)
    listed = torch.zeros(T, V, dtype=torch.int32, device="cuda").scatter_add_(1, ids.clamp(0, V - 1), live.int()) > 0
    lp = torch.log_softmax(S / tau, 1)
    kl = torch.where(q > 0, q * (q.log() - lp), 0.0).sum(1)
    Q, p = q.sum(1), torch.exp(lp)
    if d["lse"] is None:
        grad = p * Q[:, None] - q
    else:
        qr = torch.where(listed.all(1), 0.0, (1 - Q).clamp(min=0))
        lpr = torch.logsumexp(torch.where(listed, -torch.inf, lp), 1)
        kl = kl + torch.where(qr > 0, qr * (qr.log() - lpr), 0.0)
        Q = Q + qr
        inside = torch.exp(torch.where(listed, -torch.inf, lp) - lpr[:, None])  # the student's shares of the rest
        grad = torch.where(listed, p * Q[:, None] - q, p * Q[:, None] - torch.where(qr[:, None] > 0, qr[:, None] * inside, 0.0))
        q = torch.where(listed, q, qr[:, None] * inside)
    return kl, grad, p * Q[:, None], q, lp, Q


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


def check_loss(d, kl, loss):
    T = d["S"].shape[0]
    ref, _, _, _, _, Q = formula(d)
    w = d["w"].double() if d["w"] is not None else torch.full((T,), 1.0 / max(T, 1), dtype=torch.float64, device="cuda")
    ref = torch.where(w != 0, ref, 0.0)
    tol = 300 * U * Q + 2 * U * ref.abs()
    check(kl, ref, tol, "kl")
    check(loss[0], d["tau"] ** 2 * (w * ref).sum(), d["tau"] ** 2 * (w.abs() * (tol + 4 * U * ref.abs())).sum() + 1e-44, "loss")


def check_grad(d, dt, dS, gloss=1.0):
    T = d["S"].shape[0]
    _, g, pQ, q, lp, _ = formula(d)
    w = d["w"].double()[:, None] if d["w"] is not None else 1.0 / T
    k = w * d["tau"] * gloss
    x = lp.abs().clamp(max=700) + 1
    tol = (k * (pQ + q) * (3 * U * x + 304 * U)).nan_to_num(0.0) + 1e-44
    ref = torch.where(torch.as_tensor(k != 0, device="cuda"), k * g, 0.0)
    check(dS, ref, tol + 1.01 * half_step(DT[dt], ref.abs() + tol), "dS")


CASES = [(1, 7, 1), (3, 100, 5), (9, 32003, 20), (5, 4096, 256), (4, 151677, 64), (130, 1000, 33), (2, 16, 16), (2, 400000, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T,V,k", CASES)
def test_loss_and_gradient(T, V, k, rest, dt):
    M = lib_m()
    for tau, stride, shift in ((1.0, 0, 0), (2.5, 5, 3)):
        d = inputs(T, V, k, dt, rest, tau, stride=stride, shift=shift)
        stats, kl, loss = call(d, dt)
        check_loss(d, kl, loss)
        buf, dS = like(d)
        gloss = torch.full((1,), 64.0, device="cuda")
        a = call(d, dt, dS, gloss)
        assert torch.equal(a[1], kl) and torch.equal(a[2], loss)  # the same with the gradient
        check_grad(d, dt, dS, 64.0)
        rest_of = buf.clone()
        torch.as_strided(rest_of, dS.shape, dS.stride(), dS.storage_offset()).fill_(7.0)
        assert (rest_of == 7.0).all(), "written outside the rows"
        two_buf, two = like(d)
        M.moe_distill_loss_grad(d["S"], sd(dt), d["ids"], d["y"], d["lse"], d["w"], tau, stats, two, gloss)
        check_grad(d, dt, two, 64.0)
        d2 = {**d, "buf": d["buf"].clone()}
        d2["S"] = torch.as_strided(d2["buf"], d["S"].shape, d["S"].stride(), d["S"].storage_offset())
        call(d2, dt, d2["S"], gloss)  # over the logits
        assert torch.equal(d2["S"], dS)


@pytest.mark.gpu
@pytest.mark.parametrize("rest", [False, True])
def test_entries_that_do_not_count_and_repeated_ones(rest):
    d = inputs(6, 500, 12, "f32", rest, masked=False)
    d["ids"][0, 3], d["ids"][0, 4] = -1, 500
    d["y"][0, 3] = float("nan")
    d["ids"][1, :] = -7           # no entries at all
    d["ids"][2, 5] = d["ids"][2, 2]
    d["ids"][3, :] = 77
    d["y"][4, 0] = -float("inf")
    if rest:
        d["lse"] += 2.5           # the repeated ones stay within 1
    buf, dS = like(d)
    _, kl, loss = call(d, "f32", dS)
    clean = {**d, "y": torch.where((d["ids"] < 0) | (d["ids"] >= 500), 0.0, d["y"])}
    check_loss(clean, kl, loss)
    check_grad(clean, "f32", dS)
    if not rest:
        assert kl[1] == 0 and not dS[1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rest", [False, True])
def test_masked_student_logits(rest, dt):
    """-inf and the type's lowest value where a grammar forbids ids: probability 0, never nan."""
    d = inputs(6, 3000, 9, dt, rest, masked=False)
    low = torch.finfo(DT[dt]).min
    keep = torch.zeros(3000, dtype=torch.bool, device="cuda")
    keep[::3] = True
    for t, v in ((0, -float("inf")), (1, low)):
        d["S"][t, ~keep] = v
        d["ids"][t] = torch.arange(0, 27, 3, device="cuda").int()
    d["S"][2] = -float("inf")     # a row with nothing left
    d["S"][3, d["ids"][3, 0].long()] = -float("inf")  # the teacher gives weight to what is forbidden
    d["S"][4] = low
    d["S"][5] = -float("inf")     # one id left, and not an entry
    d["S"][5, 1] = 3.0
    d["ids"][5, d["ids"][5] == 1] = 2
    buf, dS = like(d)
    stats, kl, loss = call(d, dt, dS)
    one = lambda i: {**d, **{k: d[k][i:i + 1] if d[k] is not None else None for k in ("S", "ids", "y", "lse")}, "w": torch.ones(1, device="cuda")}  # noqa: E731
    for t in (0, 1, 4):
        check(kl[t], formula(one(t))[0][0], 300 * U * 2 + 2 * U * kl[t].double().abs(), f"kl {t}")
        check_grad({**one(t), "w": torch.full((1,), 1 / 6, device="cuda")}, dt, dS[t:t + 1])
    assert kl[2] == 0 and not dS[2].any()
    assert kl[3] == float("inf") and kl[5] == float("inf") and loss == float("inf")
    assert dS[3].isfinite().all() and not dS[5].isnan().any()


@pytest.mark.gpu
def test_nan_and_inf_are_not_hidden_and_stay_in_their_rows():
    d = inputs(5, 2000, 8, "f32", True, masked=False)
    clean = call(d, "f32")[1].clone()
    d["S"][1, 3] = float("nan")
    d["S"][2, 5] = float("inf")
    d["S"][3, d["ids"][3, 1].long()] = float("inf")
    buf, dS = like(d)
    _, kl, loss = call(d, "f32", dS)
    assert kl[1:4].isnan().all() and loss.isnan() and torch.equal(kl[[0, 4]], clean[[0, 4]])
    assert dS[1:4].isnan().any(1).all() and dS[[0, 4]].isfinite().all()


@pytest.mark.gpu
def test_rows_of_weight_zero_are_not_read():
    d = inputs(4, 3001, 8, "bf16", True)
    d["w"] = torch.tensor([0.5, 0.0, 0.25, 0.0], device="cuda")
    d["S"][1], d["y"][3] = float("nan"), float("nan")
    buf, dS = like(d)
    _, kl, loss = call(d, "bf16", dS)
    assert kl.isfinite().all() and loss.isfinite() and kl[1] == 0 and not dS[1].any() and not dS[3].any() and dS[0].any()


@pytest.mark.gpu
def test_rest_far_below_the_entries():
    """The student's rest is 200 below its entries: its probability is below fp32's range, its logarithm is not."""
    d = inputs(3, 5000, 8, "f32", True, masked=False)
    d["S"] -= 200
    d["S"].scatter_(1, d["ids"].long(), d["y"])
    buf, dS = like(d)
    _, kl, loss = call(d, "f32", dS)
    assert kl.isfinite().all()
    ref, g, _, _, _, _ = formula(d)
    check(kl, ref, 300 * U * 2 + 1e-6 * ref, "kl")
    check(dS, g / 3, 400 * U * (g.abs() / 3) + 1e-9, "dS")


@pytest.mark.gpu
def test_gradient_is_that_of_differences():
    for rest in (False, True):
        d = inputs(2, 60, 5, "f32", rest, tau=2.0)
        buf, dS = like(d)
        call(d, "f32", dS)
        S, h = d["S"].double().clone(), 1e-5
        w = d["w"].double()
        for t, v in ((0, int(d["ids"][0, 0])), (0, 11), (1, 59), (1, int(d["ids"][1, 4]))):
            f = []
            for s in (h, -h):
                e = {**d, "S": S.clone()}
                e["S"][t, v] += s
                f.append(float((formula(e)[0] * w).sum()) * 4)
            want = (f[0] - f[1]) / (2 * h)
            assert abs(float(dS[t, v]) - want) <= 1e-5 * abs(want) + 1e-6


@pytest.mark.gpu
def test_empty_batch_and_repeats():
    d = inputs(0, 100, 4, "f32", False, masked=False)
    _, _, loss = call(d, "f32")
    assert loss == 0
    d = inputs(64, 20011, 16, "bf16", True)
    (b1, s1), (b2, s2) = like(d), like(d)
    a, b = call(d, "bf16", s1), call(d, "bf16", s2)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.equal(s1, s2)


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals():
    M = lib_m()
    S, ids, y = torch.zeros(3, 40), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4)
    o = (torch.zeros(3, 4), torch.zeros(3), torch.zeros(1))

    def refused(code, *args):
        with pytest.raises(M.MpbError) as e:
            M.moe_distill_loss(*args)
        assert e.value.code == code, str(e.value)
    f = M.MPB_F32
    for a in ((None, f, ids, y), (S, f, None, y), (S, f, ids, None), (S, 7, ids, y), (S.half(), f, ids, y), (S, f, ids.long(), y),
              (S, f, ids, y.double()), (torch.zeros(40, 3).t(), f, ids, y), (S[:1].expand(3, 40), f, ids, y)):
        refused(-1, *a, None, None, 1.0, *o, None, None)
    refused(-2, S, f, ids[:2], y, None, None, 1.0, *o, None, None)
    refused(-2, S, f, ids, y[:, :3], None, None, 1.0, *o, None, None)
    refused(-2, S, f, ids, y, torch.zeros(4), None, 1.0, *o, None, None)
    refused(-2, S, f, ids, y, None, None, 1.0, torch.zeros(3, 2), *o[1:], None, None)
    refused(-2, S, f, ids, y, None, None, 1.0, *o, S, torch.ones(2))
    refused(-1, S, f, ids, y, None, None, 1.0, *o, torch.zeros(3, 48)[:, :40], None)
    with pytest.raises(M.MpbError) as e:
        M.moe_distill_loss_grad(S, f, None, y, None, None, 1.0, o[0], S, None)
    assert e.value.code == -1


def test_refusals_of_the_library():
    M = lib_m()
    L = M._lib.lib()
    p = 4096

    def fwd(S=p, t=2, ld=50, ids=p, y=p, T=3, V=40, k=4, tau=1.0, st=p, kl=p, loss=p, dS=p):
        return L.moe_distill_loss(S, t, ld, ids, y, None, None, T, V, k, tau, st, kl, loss, dS, None, None)

    def bwd(S=p, t=2, ld=50, ids=p, y=p, T=3, V=40, k=4, tau=1.0, st=p, dS=p):
        return L.moe_distill_loss_grad(S, t, ld, ids, y, None, None, T, V, k, tau, st, dS, None, None)
    for f in (fwd, bwd):
        assert f(t=3) == -1 and f(T=-1) == -1 and f(tau=0.0) == -1 and f(tau=float("nan")) == -1 and f(tau=1e4) == -1 and f(tau=-1.0) == -1
        assert f(T=(1 << 20) + 1) == -2 and f(V=0) == -2 and f(V=400001) == -2 and f(k=0) == -2 and f(k=257) == -2
        assert f(ld=39) == -2 and f(ld=1 << 41) == -2 and f(S=None) == -1 and f(ids=None) == -1 and f(y=None) == -1 and f(st=None) == -1
        assert f(S=4098) == -1 and f(t=1, S=4097) == -1 and f(dS=4100) == -1 and f(st=4100) == -1
    assert fwd(loss=None) == -1 and fwd(kl=None) == -1 and bwd(dS=None) == -1
    assert bwd(T=0, S=None, ids=None, y=None, st=None, dS=None) == 0

"""The router's gradients to fp32 accuracy, from the kernel's own logits.

The reference forms dl in 64 bits from the stored logits, lse and counts, so that
only the gradient calls' own errors are left. u = 2^-24.
dl: exp(l - lse) carries its rounded argument, (|l - lse| + 4) u of itself; the
balance term's weighted mean passes at most 8 + 6 additions and the factors
around it fewer than ten roundings: within (|l - lse| + 40) u of what it is made
of. A slot's weight is such an exponential over a sum of at most 16, and its
gradient's mean one more sum: within (r + 60) u, r the spread of the winning logits.
dX: dl and W are two fp16 halves each, scaled by a power of two per token and per
column that brings the largest into [2^13, 2^14), the second half by 2^11 more.
Each half rounds by at most 2^-11 of what it stands for, so that the pair is
within 2^-22 of the value, or where the second half falls below fp16's smallest
step of 2^-24, within 2^-25 2^-11 of a scaled unit: 2^-49 of the largest. The product of
the second halves (2^-22) is left out: 12 u of the products' absolute sum and
2^-49 of either side's largest times the other's absolute sum. Three matrix
instructions for 32 experts and one addition: n(L) = 4 L / 32 32-fold
sums, each instruction's within 32 additions of its own: 4 L / 32 + 32 more, + 8 for the scales.
dW: dl in three exact bf16 parts, X in one or two; 4 u left out, at most six
instructions for 32 tokens, four waves and up to 256 ranges that are added in turn."""
import math

import pytest

from test_router_loss import DT, U, check, check_fwd, clean, dbl, inputs, run_fwd, run_grad

torch = pytest.importorskip("torch")

ALPHA, BETA = 0.01, 0.001


def gradient(o, d, alpha=ALPHA, beta=BETA, gw=True):
    """(dl, what it is made of, its tolerance) in 64 bits, from the stored logits, lse and counts."""
    D = dbl(d)
    T, E, K = D["X"].shape[0], D["W"].shape[0], D["idx"].shape[1]
    l, lse, counts = o["logits"].double(), o["lse"].double()[:, None], o["counts"].double()
    live = torch.ones(T, 1, dtype=torch.bool, device=l.device) if D["mask"] is None else D["mask"].bool()[:, None]
    N = counts[E].clamp(min=1)
    f = counts[:E] / (K * N)
    p = torch.exp(l - lse) * live
    dot = (p * f).sum(1, keepdim=True)
    a, c = alpha * E / N, 2 * beta / N
    dl = p * (a * (f - dot) + c * lse)
    made = p * (abs(a) * (f + dot) + abs(c) * lse.abs())
    tol = made * U * ((l - lse).abs() + 40)
    if gw:
        idx = D["idx"].long()
        lk = l.gather(1, idx)
        w = torch.softmax(lk, 1) * live
        mean = (w * D["gw"]).sum(1, keepdim=True)
        m = w * (D["gw"].abs() + (w * D["gw"].abs()).sum(1, keepdim=True))
        dl = dl.scatter_add(1, idx, w * (D["gw"] - mean))
        made = made.scatter_add(1, idx, m)
        tol = tol.scatter_add(1, idx, m * U * (60 + lk.amax(1, keepdim=True) - lk.amin(1, keepdim=True)))
    return dl, made, tol


def dx_tol(dl, tol, W):
    """Tolerance of dX = dl W element by element."""
    E = W.shape[0]
    n = 4 * (-(-E // 64) * 64) / 32 + 40
    aw = W.abs()
    return (tol @ aw + (n + 12) * U * (dl.abs() @ aw) + 1e-37
            + 2.0 ** -49 * (dl.abs().amax(1, keepdim=True) * aw.sum(0) + dl.abs().sum(1, keepdim=True) * aw.amax(0)))


def halves_product(dl, W, second):
    """dl W from two fp16 halves of each side, the second scaled by `second`, summed in 64 bits (CPU)."""
    def cut(x, dim):
        m = x.abs().amax(dim, keepdim=True)
        up = torch.exp2(13 - torch.floor(torch.log2(m.clamp(min=1e-300))))
        v = (x * up).float()
        hi = v.half()
        lo = ((v - hi.float()) * second).half()
        return hi.double(), lo.double() / second, 1 / up
    (ah, al, au), (bh, bl, bu) = cut(dl, 1), cut(W, 0)
    return (ah @ bh + ah @ bl + al @ bh) * au * bu


def spread(T, H, E, K, dt, seed=0, device="cuda"):
    """Inputs whose router rows are spread over nine decades, the probabilities the other way: products of about one
    size, each of a value far below its token's or its column's largest."""
    g = torch.Generator(device=device).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    X = rn(T, H).to(DT[dt])
    rows = 9 * torch.rand(E, 1, generator=g, device=device) - 9
    W = rn(E, H) * H ** -0.5 * 10.0 ** rows
    b = rn(E) - math.log(10) * rows[:, 0]
    l = X.float() @ W.t() + b
    idx = torch.topk(l, K, dim=1).indices.int().contiguous()
    return {"X": X, "W": W, "b": b, "idx": idx, "mask": None, "gw": rn(T, K) / T}


def test_the_halves_bound_holds_for_spread_rows():
    """The arithmetic of the bound, on the CPU: second halves scaled by 2^11 stay within it, plain ones do not."""
    d = spread(64, 256, 60, 4, "bf16", seed=1, device="cpu")
    l = d["X"].double() @ d["W"].double().t() + d["b"]
    lse = torch.logsumexp(l, 1)
    counts = torch.cat([torch.bincount(d["idx"].flatten().long(), minlength=60), torch.tensor([64])])
    dl = gradient({"logits": l, "lse": lse, "counts": counts}, d, gw=False)[0]
    dl, W = dl.float().double(), d["W"].double()
    tol = dx_tol(dl, torch.zeros_like(dl), W) - (4 * 64 / 32 + 40) * U * (dl.abs() @ W.abs())
    err = lambda s: float(((halves_product(dl, W, s) - dl @ W).abs() / tol).max())  # noqa: E731
    assert err(2048.0) <= 1.0
    assert err(1.0) > 4.0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("gw", [True, False])
@pytest.mark.parametrize("T,H,E,K", [(70, 256, 60, 4), (300, 512, 128, 8), (130, 192, 300, 8)])
def test_dx_of_spread_rows(T, H, E, K, gw, dt):
    d = spread(T, H, E, K, dt, seed=T)
    o = run_fwd(d, dt)
    dl, made, tol = gradient(o, d, gw=gw)
    W = d["W"].double()
    check(run_grad(d, dt, o, gw=gw, want=("dX",))["dX"], dl @ W, dx_tol(dl, tol, W), "dX")


# ---------------------------------------------------------------- products to fp32 accuracy, by the norm of their errors
def far(n):
    """Tolerance of an error's norm, in units of u and of the norm of what the sums are made of (the root of the sum of
    their terms' squares, or the sum where that is larger). Roundings of u / sqrt(3) each, independent, at partial sums
    that grow to the whole: sqrt(n / 6) of them over n; three times that, and 8 for what each term carries by itself."""
    return (8 + 3 * (n / 6) ** 0.5) * U


def norms(got, terms_sq, ref, n, what):
    """The error's norm over the whole result against far(n)."""
    size = torch.maximum(terms_sq.sqrt(), ref.abs())
    err = float((got.double() - ref).norm() / size.norm())
    assert err <= far(n), f"{what}: error {err / U:.1f} u, tolerance {far(n) / U:.1f} u"


def check_products(d, dt, o, g, gw):
    """Logits from X and W, then dX, dW and dbias from dl of the stored logits: element by element, and in norm."""
    D = clean(dbl(d))
    (T, H), E = D["X"].shape, D["W"].shape[0]
    X, W = D["X"], D["W"]
    ref = X @ W.t()
    b = 0.0 if D["b"] is None else D["b"]
    live = torch.ones(T, dtype=torch.bool, device=X.device) if D["mask"] is None else D["mask"].bool()
    norms(o["logits"][live], ((X * X) @ (W * W).t() + b * b)[live], (ref + b)[live], 6 * H / 32 + 32, "logits")
    dl, made, tol = gradient(o, d, gw=gw)
    made_sq = made * made
    # of what an element is made of, dl keeps (|l - lse| + 40) u at most and a tenth of that as a rule
    n_dx, n_dw = 4 * E / 32 + 40, 6 * T / 32 + 260
    check(g["dX"], dl @ W, dx_tol(dl, tol, W), "dX")
    norms(g["dX"], made_sq @ (W * W), dl @ W, n_dx, "dX")
    ax = X.abs()
    check(g["dW"], dl.t() @ X, tol.t() @ ax + (n_dw + 4) * U * (dl.abs().t() @ ax) + 1e-37, "dW")
    norms(g["dW"], made_sq.t() @ (X * X), dl.t() @ X, n_dw, "dW")
    check(g["db"], dl.sum(0), tol.sum(0) + 34 * U * dl.abs().sum(0) + 1e-37, "dbias")
    norms(g["db"], made_sq.sum(0), dl.sum(0), 64, "dbias")


PRODUCTS = [(1, 2048, 60, 4), (72, 2048, 60, 4), (33, 128, 512, 16), (700, 320, 129, 8), (65, 65536, 4, 2),
            (1000, 2816, 128, 8), (4099, 256, 60, 4)]
# 128-token tiles of the logits (from 8192 tokens) with 64 and 128 experts, whole and ragged, dX over several blocks of
# 256 tokens a workgroup with and without W taken in again between them
LARGE = [(8192, 512, 60, 4), (8209, 512, 128, 8), (8209, 2816, 60, 4), (8209, 2816, 300, 8), (16381, 2048, 128, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,H,E,K", PRODUCTS + LARGE)
def test_products(T, H, E, K, masked, dt):
    d = inputs(T, H, E, K, dt, masked, seed=T + E)
    o = run_fwd(d, dt)
    if T >= 8192:
        check_fwd(d, dt, o)
    for gw in (True, False):
        check_products(d, dt, o, run_grad(d, dt, o, gw=gw), gw)


def parts(x, n):
    """The first n bf16 parts of x, cut off by truncation."""
    x, out = x.float(), 0.0
    for _ in range(n):
        p = (x.view(torch.int32) & -65536).view(torch.float32)
        out, x = out + p.double(), x - p
    return out


@pytest.mark.parametrize("T,H,E,K", [(72, 2048, 60, 4), (700, 320, 129, 8), (300, 2816, 128, 8)])
def test_fewer_parts_are_noticed(T, H, E, K):
    """Planted in the reference's own values, on the CPU: W in two parts for the logits, dl in two parts or rounded to
    bf16 for the gradients, each outside; the whole values are inside."""
    g = torch.Generator().manual_seed(T)
    X = torch.randn(T, H, generator=g).bfloat16()
    W = torch.randn(E, H, generator=g) * H ** -0.5
    d = {"X": X, "W": W, "b": -0.5 * torch.log1p(torch.arange(E).float()), "mask": None, "gw": torch.randn(T, K, generator=g) / T}
    l = X.double() @ W.double().t() + d["b"]
    d["idx"] = torch.topk(l, K, dim=1).indices.int()
    counts = torch.cat([torch.bincount(d["idx"].flatten().long(), minlength=E), torch.tensor([T])])
    o = {"logits": l, "lse": torch.logsumexp(l, 1), "counts": counts}
    for gw in (True, False):
        dl = gradient(o, d, gw=gw)[0]
        grads = lambda q: {"dX": q @ W.double(), "dW": q.t() @ X.double(), "db": q.sum(0)}  # noqa: E731
        check_products(d, "bf16", o, grads(dl.float().double()), gw)
        for q in (dl.bfloat16().double(), parts(dl, 2)):
            for k in ("dX", "dW"):
                with pytest.raises(AssertionError, match=k):
                    check_products(d, "bf16", o, {**grads(dl), k: grads(q)[k]}, gw)
        short = {**o, "logits": X.double() @ parts(W, 2).t() + d["b"]}
        with pytest.raises(AssertionError, match="logits"):
            check_products(d, "bf16", short, grads(dl), gw)

"""moe_adapters keeps A x at fp32 accuracy between its two products.

The norm of the error over the whole result, in units of u = 2^-24 and of the norm
of what the sums are made of (the root of the sum of their terms' squares).
Roundings of u / sqrt(3) each, independent, at partial sums that grow to the whole
make sqrt(n / 6) of them over n; three times that, and 8 for what a term carries by
itself (the scale, the cut parts and the sum with base). n: one instruction for 32
of Kd, up to 16 ranges and 8 waves, and five for 32 ranks."""
import pytest

from test_adapters import DT, U, inputs, run

torch = pytest.importorskip("torch")


def check_norm(d, got):
    (T, Kd), (n, R, _), N = d["X"].shape, d["A"].shape, d["B"].shape[1]
    err = size = 0.0
    for a in range(n):
        rows = (d["adapter"] == a).nonzero()[:, 0]
        r = R if d["ranks"] is None else int(d["ranks"][a])
        X, A, B, s = d["X"][rows].double(), d["A"][a, :r].double(), d["B"][a, :, :r].double(), float(d["scales"][a])
        err += float((got[rows].double() - s * (X @ A.t() @ B.t())).square().sum())
        size += s * s * float(((X * X) @ (A * A).t() @ (B * B).t()).sum())
    tol = (8 + 3 * ((Kd / 32 + 24 + 5 * R / 32) / 6) ** 0.5) * U
    rel = (err / size) ** 0.5
    assert rel <= tol, f"error {rel / U:.1f} u, tolerance {tol / U:.1f} u"


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Kd,N,n,R", [(1, 2048, 2048, 1, 16), (40, 4096, 1024, 5, 32), (128, 4096, 4096, 64, 32),
                                        (1100, 320, 1408, 2, 64), (1700, 2816, 704, 3, 128), (2000, 256, 320, 6, 24)])
def test_products(T, Kd, N, n, R, dt):
    d = {**inputs(T, Kd, N, n, R, dt, seed=T, mixed=False), "base": None}
    if T == 1:
        d["adapter"].zero_()
    check_norm(d, run(d, dt))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_a_rounded_middle_is_noticed(dt):
    """Planted on the CPU: A x in bf16, or in two bf16 parts, is outside; in fp32 it is inside."""
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    T, Kd, N, R = 50, 4096, 256, 32
    d = {"X": rn(T, Kd).to(DT[dt]), "A": (rn(1, R, Kd) * Kd ** -0.5).to(DT[dt]), "B": (rn(1, N, R) * R ** -0.5).to(DT[dt]),
         "ranks": None, "scales": torch.ones(1), "adapter": torch.zeros(T, dtype=torch.int32)}
    z = (d["X"].double() @ d["A"][0].double().t()).float()
    out = lambda q: q.double() @ d["B"][0].double().t()  # noqa: E731
    check_norm(d, out(z))
    first = (z.view(torch.int32) & -65536).view(torch.float32)
    second = ((z - first).view(torch.int32) & -65536).view(torch.float32)
    for q in (z.bfloat16(), first.double() + second.double()):
        with pytest.raises(AssertionError, match="tolerance"):
            check_norm(d, out(q))

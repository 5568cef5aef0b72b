"""moe_adapters against the formula in 64 bits.

Tolerances. u = 2^-24. z = A x is a sum of Kd exact products, one matrix
instruction per 32 of them (within 32 additions) over at most 16 ranges and four
waves: within n1 u of the products' absolute sum, n1 = Kd / 32 + 100. B z takes at
most five instructions per 32 ranks, n2 = 6 (R / 32 + 1) + 100, and the cut parts
leave out less than 4 u. The sum with base rounds twice."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def inputs(T, Kd, N, n, R, dt, seed=0, mixed=True, runs=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    d = {"X": rn(T, Kd).to(DT[dt]), "A": (rn(n, R, Kd) * Kd ** -0.5).to(DT[dt]), "B": (rn(n, N, R) * R ** -0.5).to(DT[dt])}
    d["ranks"] = torch.randint(0, R + 1, (n,), generator=g, device="cuda", dtype=torch.int32) if mixed else None
    d["scales"] = rn(n)
    ad = torch.randint(-1, n + 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    d["adapter"] = torch.sort(ad).values.contiguous() if runs else ad
    d["base"] = rn(T, N)
    return d


def run(d, dt, out=None, stream=None, ws=None):
    M = lib_m()
    (T, Kd), (n, R, _), N = d["X"].shape, d["A"].shape, d["B"].shape[1]
    if out is None:
        out = torch.full((T, N), float("nan"), device="cuda")
    if ws is None:
        ws = torch.full((M.moe_adapters_workspace_bytes(T, Kd, n, R),), 255, dtype=torch.uint8, device="cuda")
    M.moe_adapters(d["X"], M.MPB_BF16 if dt == "bf16" else M.MPB_F16, d["A"], d["B"], d["ranks"], d["scales"], d["adapter"],
                   d["base"], out, ws, stream)
    return out


def formula(d):
    """(out, tolerance), one adapter after another."""
    (T, Kd), (n, R, _), N = d["X"].shape, d["A"].shape, d["B"].shape[1]
    out = torch.zeros(T, N, dtype=torch.float64, device="cuda") if d["base"] is None else d["base"].double()
    tol = 2 * U * out.abs()
    n1, n2 = Kd / 32 + 100, 6 * (R / 32 + 1) + 104
    ids = d["adapter"].tolist()
    for a in sorted(set(ids)):
        r = R if d["ranks"] is None else min(max(int(d["ranks"][a]), 0), R) if 0 <= a < n else 0
        if not 0 <= a < n or r == 0:
            continue
        rows = torch.tensor([t for t, i in enumerate(ids) if i == a], device="cuda")
        X, A, B = d["X"][rows].double(), d["A"][a, :r].double(), d["B"][a, :, :r].double()
        s = 1.0 if d["scales"] is None else float(d["scales"][a])
        z, za = X @ A.t(), X.abs() @ A.abs().t()
        add = s * (z @ B.t())
        out[rows] += add
        tol[rows] += abs(s) * U * (n1 * (za @ B.abs().t()) + n2 * (z.abs() @ B.abs().t())) + 2 * U * add.abs()
    return out, tol


def check(d, got):
    ref, tol = formula(d)
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {float((err / tol).nan_to_num(1e9).max()):.2f} of the tolerance"


SHAPES = [  # T, Kd, N, n, R, runs
    (1, 2048, 2048, 4, 16, False), (1, 64, 64, 1, 8, False), (2, 128, 192, 3, 24, False), (16, 256, 64, 1, 32, True),
    (17, 64, 320, 1, 128, True), (72, 2048, 1408, 60, 16, False), (128, 4096, 256, 64, 32, False), (255, 192, 128, 300, 72, False),
    (64, 320, 704, 2, 64, True), (65, 320, 704, 2, 64, True), (2100, 128, 192, 3, 24, True), (1100, 320, 1408, 2, 64, False),
    (256, 320, 704, 2, 64, True), (257, 320, 704, 2, 64, True), (257, 128, 128, 400, 40, False), (600, 2816, 448, 5, 64, True),
    (4099, 256, 320, 7, 16, False), (4099, 64, 64, 1, 128, True), (1500, 128, 64, 4096, 8, False), (33, 65536, 64, 2, 16, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("T,Kd,N,n,R,runs", SHAPES)
def test_adapters(T, Kd, N, n, R, runs, mixed, dt):
    d = inputs(T, Kd, N, n, R, dt, seed=T + R, mixed=mixed, runs=runs)
    check(d, run(d, dt))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 700, 1700])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_unused_ranks_ids_and_defaults(T, dt):
    """Nan past an adapter's rank, ranks and ids out of range, no base, no scales."""
    d = inputs(T, 256, 192, 6, 40, dt, seed=9)
    d["ranks"] = torch.tensor([0, 1, 13, 32, 99, -4], dtype=torch.int32, device="cuda")
    for a, r in enumerate(d["ranks"].clamp(0, 40).tolist()):
        d["A"][a, r:] = float("nan")
        d["B"][a, :, r:] = float("nan")
    d["adapter"][:4] = torch.tensor([6, 1 << 30, -(1 << 31), -1], dtype=torch.int32)
    check(d, run(d, dt))
    e = {**d, "base": None, "scales": None}
    got = run(e, dt)
    check(e, got)
    assert not got[:4].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 700, 1700])
def test_in_place_and_rows_not_taken(T):
    d = inputs(T, 128, 256, 3, 16, "bf16", seed=10, mixed=False)
    want = run(d, "bf16")
    big = torch.cat([d["base"], torch.full((8, 256), 7.0, device="cuda")])
    e = {**d, "base": big[:T]}
    run(e, "bf16", out=big[:T])
    assert torch.equal(big[:T], want) and bool((big[T:] == 7).all())
    none = (d["adapter"] < 0) | (d["adapter"] >= 3)
    assert none.any() and torch.equal(want[none], d["base"][none])
    d["adapter"].fill_(-1)
    assert torch.equal(run(d, "bf16"), d["base"])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [60, 700, 1700])
def test_a_tokens_result_does_not_depend_on_the_others(T):
    """The same tokens in another order, and with other tokens' inputs infinite: the same bits."""
    d = inputs(T, 256, 128, 5, 32, "f16", seed=11)
    want = run(d, "f16")
    p = torch.randperm(T, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    e = {**d, "X": d["X"][p].contiguous(), "adapter": d["adapter"][p].contiguous(), "base": d["base"][p].contiguous()}
    assert torch.equal(run(e, "f16"), want[p])
    e = {**d, "X": d["X"].clone()}
    e["X"][::3] = float("inf")
    keep = torch.arange(T, device="cuda") % 3 != 0
    assert torch.equal(run(e, "f16")[keep], want[keep])
    assert torch.equal(run(d, "f16"), want)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [50, 500, 2000])
def test_stream_and_graph_replays_with_other_ids(T):
    d, e = (inputs(T, 192, 320, 6, 24, "bf16", seed=s) for s in (12, 13))
    want = [run(v, "bf16") for v in (d, e)]
    st = {k: v.clone() for k, v in d.items()}
    M = lib_m()
    ws = torch.empty(M.moe_adapters_workspace_bytes(T, 192, 6, 24), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, 320, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(st, "bf16", out=out, stream=s, ws=ws)
    s.synchronize()
    assert torch.equal(out, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(st, "bf16", out=out, ws=ws)
    for i in (1, 0, 1, 0):
        for k, v in st.items():
            v.copy_((d, e)[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        run(e, "bf16")


@pytest.mark.gpu
def test_empty_batch():
    d = inputs(4, 128, 64, 2, 8, "bf16")
    e = {k: v[:0].contiguous() if k in ("X", "adapter", "base") else v for k, v in d.items()}
    assert run(e, "bf16").shape == (0, 64)


def test_refusals():
    M = lib_m()
    from mixed_precision_bit_amd import _lib
    L = _lib.lib()
    p, odd = ctypes.c_void_p(16), ctypes.c_void_p(8)

    def f(X=p, xd=0, T=4, Kd=256, A=p, B=p, r=p, s=p, n=2, R=16, N=128, i=p, base=p, out=p, ws=p, nb=1 << 30):
        return L.moe_adapters(X, xd, T, Kd, A, B, r, s, n, R, N, i, base, out, ws, nb, None)

    assert f(xd=2) == -1 and f(T=-1) == -1 and f(T=(1 << 20) + 1) == -2 and f(Kd=100) == -2 and f(Kd=65600) == -2
    assert f(N=0) == -2 and f(N=100) == -2 and f(N=131136) == -2 and f(n=0) == -2 and f(n=4097) == -2
    assert f(R=0) == -2 and f(R=12) == -2 and f(R=136) == -2
    for k in ("X", "A", "B", "i", "out", "ws"):
        assert f(**{k: None}) == -1, k
    for k in ("X", "A", "B", "base", "out", "ws"):
        assert f(**{k: odd}) == -1, k
    assert f(nb=255) == -5 and "workspace" in M.mpb_last_error()
    assert f(T=0, X=None, i=None, base=None, out=None, ws=None, nb=0) == 0
    assert M.moe_adapters_workspace_bytes(4, 256, 2, 12) == 0 == M.moe_adapters_workspace_bytes(4, 250, 2, 16)
    assert M.moe_adapters_workspace_bytes(300, 256, 2, 16) >= 300 * 16 * 4 + 300 * 4


def test_tensor_refusals():
    M = lib_m()
    X, A, B = (torch.zeros(*s, dtype=torch.float16) for s in ((4, 128), (2, 8, 128), (2, 64, 8)))
    ad, out, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 64), torch.zeros(1 << 16, dtype=torch.uint8)

    def code(X=X, A=A, B=B, ranks=None, ad=ad, base=None, out=out):
        with pytest.raises(M.MpbError) as e:
            M.moe_adapters(X, M.MPB_F16, A, B, ranks, None, ad, base, out, ws)
        return e.value.code

    assert code() == -1                                     # on the CPU
    assert code(A=A.float()) == -1 and code(ad=ad.long()) == -1 and code(out=out.half()) == -1
    assert code(B=B[:1]) == -2 and code(A=A[:, :, :64]) == -2 and code(ad=ad[:2]) == -2 and code(base=out[:, :32]) == -2
    assert code(B=B.transpose(1, 2)) == -2 and code(ranks=torch.zeros(3, dtype=torch.int32)) == -2 and code(X=X[0]) == -2

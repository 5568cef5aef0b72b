"""The block's operators where offsets pass 32 bits, and two calls at once."""
import pytest

import test_adapters as TA
import test_block_norm as TN
import test_router_loss as TR

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def rows_of(d, rows):
    return {k: v[rows].contiguous() if v is not None and v.dim() and v.shape[0] == d["T"] else v for k, v in d.items() if k != "T"}


def test_norms_past_2_to_the_32_elements():
    """T x H = 4.6e9: the last rows are held to the formula, and the sums over rows to sums over slices."""
    T, H = (1 << 20) - 5, 4416
    base = TN.inputs(331, H, "bf16", "token", True, True, seed=1)
    pick = torch.arange(T, device="cuda") % 331
    d = {k: (v[pick] if v is not None and v.shape[0] == 331 else v) for k, v in base.items()}
    d["dr_out"] = None
    rows = torch.tensor([0, 1, 486500, T - 2, T - 1], device="cuda")
    small = rows_of({**d, "T": T}, rows)
    r_out, x = TN.run_fwd(d, "bf16", 0.7, inplace=True)
    TN.check_fwd(small, "bf16", 0.7, r_out[rows], x[rows])
    del r_out, x
    g = TN.run_grad(d, "bf16", 0.7)
    one = TN.run_grad(small, "bf16", 0.7)
    for k in ("dr", "do", "dgate"):
        assert torch.equal(g[k][rows], one[k]), k
    # the batch repeats 331 rows: whole repeats and a rest
    many = TN.grad64({**TN.dbl(base), "dr_out": None}, 0.7)
    rest = TN.grad64({**TN.dbl({k: (v[:T % 331] if v is not None and v.shape[0] == 331 else v) for k, v in base.items()}), "dr_out": None}, 0.7)
    for k in ("dgp", "dgn"):
        want = T // 331 * many[k] + rest[k]
        # every row within E2 of its terms, T / 512 + 48 additions (as in the smaller tests); terms are below 40 here
        assert float((g[k].double() - want).abs().max()) <= (TN.E2 + TN.U * (T / 512 + 48)) * 40 * T, k


def test_router_past_2_to_the_32_bytes():
    T, H, E = 600_011, 4096, 6
    base = TR.inputs(997, H, E, 2, "bf16", True, seed=2)
    pick = torch.arange(T, device="cuda") % 997
    d = {k: (v[pick] if v is not None and v.shape[0] == 997 else v) for k, v in base.items()}
    o = TR.run_fwd(d, "bf16")
    rows = torch.tensor([0, 524_300, T - 1], device="cuda")
    small = {k: (v[rows].contiguous() if v is not None and v.shape[0] == T else v) for k, v in d.items()}
    s = TR.run_fwd(small, "bf16")
    # other launch shapes add H in another order: both within the tolerance of a logit
    tol = 2 * TR.logit_tol(TR.clean(TR.dbl(small))) + 1e-30
    assert bool(((o["logits"][rows].double() - s["logits"].double()).abs() <= tol).all())
    counts = torch.bincount(d["idx"][d["mask"].bool()].flatten().long(), minlength=E)
    assert torch.equal(o["counts"][:E].long(), counts) and int(o["counts"][E]) == int(d["mask"].sum())
    gr = TR.run_grad(d, "bf16", o)
    TR.check_grad(small, "bf16", {"dX": gr["dX"][rows]}, counts=o["counts"].long())


def test_adapters_past_2_to_the_32_bytes():
    T, Kd, N = 330_001, 6656, 4096
    base = TA.inputs(1009, Kd, N, 3, 8, "f16", seed=3)
    pick = torch.arange(T, device="cuda") % 1009
    d = {k: (v[pick] if v is not None and v.shape[0] == 1009 else v) for k, v in base.items()}
    out = TA.run(d, "f16", out=d["base"])
    rows = torch.tensor([0, 5, 262_150, T - 3, T - 1], device="cuda")
    small = {k: (v[rows].contiguous() if v is not None and v.shape[0] == T else v) for k, v in d.items()}
    small["base"] = base["base"][pick[rows]]
    TA.check(small, out[rows])


def test_two_calls_at_once():
    """Calls on two streams with a workspace each, and a decode-size call beside a long one: the same bits as alone."""
    a, b = TR.inputs(4096, 1024, 64, 4, "bf16", True, seed=4), TR.inputs(70, 1024, 64, 4, "f16", False, seed=5)
    c, e = TA.inputs(3000, 512, 1024, 5, 16, "bf16", seed=6), TA.inputs(40, 512, 1024, 5, 16, "f16", seed=7)
    n = TN.inputs(3000, 1024, "bf16", "full", True, True, seed=8)

    def one(stream):
        o = TR.run_fwd(a, "bf16", stream=stream)
        return [*o.values(), *TR.run_grad(a, "bf16", o, stream=stream).values(), TA.run(c, "bf16", stream=stream)]

    def two(stream):
        o = TR.run_fwd(b, "f16", stream=stream)
        return [*o.values(), *TR.run_grad(b, "f16", o, stream=stream).values(), TA.run(e, "f16", stream=stream),
                *TN.run_grad(n, "bf16", 0.7, stream=stream).values()]

    want = one(None), two(None)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        # results filled on the current stream before either call begins
        got = []
        for st, f in zip(s, (one, two)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(f(st))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))

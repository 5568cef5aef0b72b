"""moe_adapters on its 64-token tiles, each test certain that its sizes take them."""
import pytest

from test_adapters import check, inputs, lib_m, run

torch = pytest.importorskip("torch")


def workspace(T, Kd, n, R, rows):
    """Bytes of the workspace with tiles of `rows` tokens: partial sums, tokens, tiles."""
    tiles = min(n + 1, T) + T // rows
    ranges = max(1, min((320 if rows == 64 else 512) // tiles, Kd // 128, 16))
    return sum((b + 255) // 256 * 256 for b in (ranges * T * R * 4, tiles * rows * 4, (2 * tiles + 4) * 4))


def assert_wide(T, Kd, n, R):
    got = lib_m().moe_adapters_workspace_bytes(T, Kd, n, R)
    assert got == workspace(T, Kd, n, R, 64) != workspace(T, Kd, n, R, 16)


WIDE = [(1700, 256, 704, 3, 24), (1801, 128, 64, 6, 40), (1100, 192, 1088, 3, 32), (1150, 320, 576, 2, 64),
        (1300, 64, 320, 4, 128), (769, 2816, 192, 2, 96)]


def test_sizes_that_take_wide_tiles():
    for T, Kd, _, n, R in WIDE:
        assert_wide(T, Kd, n, R)
    got = lib_m().moe_adapters_workspace_bytes
    assert got(4093, 2816, 16, 64) == workspace(4093, 2816, 16, 64, 16) and got(9000, 256, 3, 16) == workspace(9000, 256, 3, 16, 16)


def case(T, Kd, N, n, R, dt, seed):
    """An adapter of rank 0, one of an odd rank, ids and ranks out of range, nan past every rank, tokens without an
    adapter, and group sizes that no tile divides."""
    d = inputs(T, Kd, N, n, R, dt, seed=seed)
    r = torch.arange(n, dtype=torch.int32) * 5 % R
    r[1] = R + 7 if n > 2 else R - 3
    r[n - 1] = -4 if n > 4 else R - 1
    d["ranks"] = r.cuda()
    for a, k in enumerate(r.clamp(0, R).tolist()):
        d["A"][a, k:] = float("nan")
        d["B"][a, :, k:] = float("nan")
    d["adapter"][torch.tensor([0, 100, T - 2, T - 1])] = torch.tensor([n, 1 << 30, -(1 << 31), -1], dtype=torch.int32, device="cuda")
    sizes = torch.bincount(d["adapter"].clamp(-1, n).long() + 1, minlength=n + 2)
    assert bool((sizes[1:n + 1] % 64 != 0).any()) and int(sizes[0]) > 0
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Kd,N,n,R", WIDE)
def test_wide_tiles(T, Kd, N, n, R, dt):
    """With and without base, scales and ranks, and in place: rows past a tile's end read their wave's first token again
    and store it again."""
    assert_wide(T, Kd, n, R)
    d = case(T, Kd, N, n, R, dt, seed=T)
    want = run(d, dt)
    check(d, want)
    none = (d["adapter"] < 0) | (d["adapter"] >= n)
    none |= ~none & (d["ranks"][d["adapter"].clamp(0, n - 1).long()] <= 0)
    assert int(none.sum()) > 100 and torch.equal(want[none], d["base"][none])
    e = {**d, "base": None, "scales": None}
    got = run(e, dt)
    check(e, got)
    assert not got[none].any()
    big = torch.cat([d["base"], torch.full((70, N), 7.0, device="cuda")])
    run({**d, "base": big[:T]}, dt, out=big[:T])
    assert torch.equal(big[:T], want) and bool((big[T:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_in_place_replays_on_wide_tiles(dt):
    """In place, captured, replayed with other ids on a fresh base each time."""
    M = lib_m()
    T, Kd, N, n, R = WIDE[0]
    sets = [case(T, Kd, N, n, R, dt, seed=s) for s in (21, 22)]
    want = [run(v, dt) for v in sets]
    st = {k: v.clone() for k, v in sets[0].items()}
    ws = torch.empty(M.moe_adapters_workspace_bytes(T, Kd, n, R), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(st, dt, out=st["base"], ws=ws)
    for i in (1, 0, 1, 0):
        for k, v in st.items():
            v.copy_(sets[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(st["base"], want[i])
        run(sets[1 - i], dt)

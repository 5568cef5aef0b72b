"""Who owns the routing workspace: every call of a layer its own, so that calls on
two streams, and captured calls replayed after larger eager ones, share none."""
import weakref

import pytest

import mpb_synth as S

torch = pytest.importorskip("torch")


@pytest.fixture
def host_layer(monkeypatch):
    """(layer, seen): a layer of config 1's sizes (its logits go through the workspace) whose kernel calls only note
    the workspaces they are given; nothing runs on a GPU."""
    from mixed_precision_bit_amd import _lib as M
    from mixed_precision_bit_amd.layer import DeviceLayer
    c = S.layer_config(1)
    D = object.__new__(DeviceLayer)
    D.H, D.I, D.E, D.S, D.K, D.device = c["H"], c["I"], c["E"], c["S"], c["K"], "cpu"
    D.W_r, D.bias = torch.zeros(D.E, D.H), None
    D.planes_table = D.luts_table = D.q_dev = torch.zeros(1, dtype=torch.int64)
    seen = []
    monkeypatch.setattr(M, "moe_ffn_workspace_bytes", lambda T: 256)
    monkeypatch.setattr(M, "moe_route", lambda X, xd, W, b, K, idx, w, ws, stream=None: seen.append(ws))
    monkeypatch.setattr(M, "moe_ffn", lambda *a: None)
    monkeypatch.setattr(M, "moe_block_norm", lambda *a: None)
    return D, seen


def rows(D, T):
    return torch.zeros(T, D.H, dtype=torch.float16)


def test_calls_share_no_routing_workspace(host_layer):
    """Two calls of one size, and one of fewer tokens, each bring a workspace of their own, of the size they need."""
    from mixed_precision_bit_amd import _lib as M
    D, seen = host_layer
    for T in (64, 64, 16, 2033):
        D.block(rows(D, T), rows(D, T), "f16")
        assert seen[-1].numel() >= M.moe_route_workspace_bytes(T, D.E)
    D.forward(rows(D, 64), "f16")
    idx, w = D.alloc_route(64)
    D.route(rows(D, 64), "f16", idx, w)
    assert len({ws.data_ptr() for ws in seen}) == len(seen) == 6
    mine = torch.empty(M.moe_route_workspace_bytes(64, D.E), dtype=torch.uint8)
    D.route(rows(D, 64), "f16", idx, w, ws=mine)      # a caller's own, where it keeps one
    assert seen[-1] is mine


def test_the_layer_keeps_no_routing_workspace(host_layer):
    """A call's workspace goes back to the allocator's pool that it came from (a stream's, a capture's) with the call."""
    D, seen = host_layer
    D.block(rows(D, 64), rows(D, 64), "f16")
    gone = weakref.ref(seen.pop())
    assert gone() is None


def block_inputs(D, T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D.H, generator=g, device="cuda").half()
    return x, torch.randn(T, D.H, generator=g, device="cuda").half(), torch.ones(D.H, device="cuda")


@pytest.fixture(scope="module")
def layer():
    from mixed_precision_bit_amd import _lib as M
    from mixed_precision_bit_amd.layer import DeviceLayer
    L = S.make_layer(1)
    D = DeviceLayer.from_synth(L)
    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q)
    torch.cuda.synchronize()
    return D


@pytest.mark.gpu
def test_routing_on_two_streams(layer):
    """The router of one layer on two streams at once (moe_ffn itself runs on the bound stream, or captured)."""
    D = layer
    sets = [block_inputs(D, T, T)[0] for T in (64, 200)]

    def route(x, stream=None):
        idx, w = D.alloc_route(x.shape[0])
        D.route(x, "f16", idx, w, stream)
        return idx, w

    want = [route(x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = [route(x, s) for x, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
def test_two_captured_blocks_replayed_at_once(layer):
    """Two graphs of one layer, each replayed on a stream of its own."""
    D = layer
    sets = [block_inputs(D, T, T) for T in (64, 200)]
    want = [D.block(x, r, "f16", None, g) for x, r, g in sets]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x, r, g in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(D.block(x, r, "f16", None, g))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for s, gr in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.gpu
def test_a_captured_block_outlives_larger_eager_calls(layer):
    """Captured without sizing anything first, replayed after larger batches and new tensors have come."""
    D = layer
    a, b = block_inputs(D, 64, 1), block_inputs(D, 64, 2)
    want = [D.block(*v[:2], "f16", None, v[2]) for v in (a, b)]
    x, r, g = (v.clone() for v in a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = D.block(x, r, "f16", None, g)
    for k, T in ((1, 300), (0, 1000), (1, 64), (0, 2033)):
        bx, br, bg = block_inputs(D, T, 3)
        eager = D.block(bx, br, "f16", None, bg)
        keep = [t.clone() for t in eager]
        new = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(16)]
        x.copy_((a, b)[k][0])
        r.copy_((a, b)[k][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want[k]))
        assert all(torch.equal(p, q) for p, q in zip(eager, keep))
        assert all(bool((t == 7).all()) for t in new)

"""moe_head_norm_grad where a wave has several tokens: the gammas' gradients over the whole batch.

Tolerance of dgamma, u = 2^-24, as in test_head_norm but for the chain of additions: up to 768 workgroups of 4 waves take
every (4 x 768)th token, 64 / NL heads at a time (NL lanes of 16 elements hold a head), so a lane adds the tokens of its wave
times their groups of heads; then come the lanes, the 4 waves, and the workgroups' rows in 16 chains."""
import pytest

import test_head_norm as TH
from test_head_norm import DT, EPS, U

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def check_dgamma(d, got_q, got_k, chunk=1 << 24):
    T, Hq, D = d["q"].shape
    nl = 1
    while 16 * nl < D:
        nl *= 2
    for x, do, got, what in ((d["q"], d["dq"], got_q, "q"), (d["k"], d["dk"], got_k, "k")):
        if got is None:
            continue
        H = x.shape[1]
        adds = -(-T // (4 * 768)) * -(-H // (64 // nl)) + 6 + 4 + 48 + 16
        ref = terms = 0.0
        rows = max(1, chunk // (H * D))
        for t in range(0, T, rows):
            part = {**d, "pos": None if d["pos"] is None else d["pos"][:, t:t + rows]}
            xs = x[t:t + rows].double()
            n, m = TH.turn(do[t:t + rows].double(), part, back=True)
            xh = xs / (xs.square().mean(2, keepdim=True) + EPS).sqrt()
            ref, terms = ref + (n * xh).sum((0, 1)), terms + (m * xh.abs()).sum((0, 1))
        TH.check(got, ref, (80 + adds) * U * terms, "dgamma_" + what)


# more tokens than waves; groups of heads that fill a wave, and that do not; lanes past the end of a head
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hk,D,Dr,pairs", [(8191, 5, 3, 96, 64, 0), (8192, 16, 8, 256, 128, 1), (3100, 9, 1, 128, 128, 0),
                                                (6145, 3, 2, 512, 0, 0), (20000, 2, 1, 16, 16, 1), (9217, 33, 5, 32, 32, 0)])
def test_gradients_of_several_tokens_a_wave(T, Hq, Hk, D, Dr, pairs, dt):
    d = TH.inputs(T, Hq, Hk, D, Dr, dt, A=2 if Dr > 16 else 1, pairs=pairs, seed=7)
    out = TH.run_grad(d, dt)
    TH.check_grad(d, dt, out)
    check_dgamma(d, out["gq"], out["gk"])
    again = TH.run_grad(d, dt, in_place=True)
    assert all(torch.equal(out[k], again[k]) for k in out)


def test_gammas_gradients_past_32_bits():
    """4.3e9 elements of queries and keys: both gammas' gradients, summed over the whole batch."""
    T, Hq, Hk, D = 1 << 20, 30, 2, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.empty(T, Hq + Hk, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    dqk = torch.empty(T, Hq + Hk, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    d = {"q": qkv[:, :Hq], "k": qkv[:, Hq:], "dq": dqk[:, :Hq], "dk": dqk[:, Hq:], "axis": None, "pairs": 0,
         "gq": 1 + 0.1 * torch.randn(D, generator=g, device="cuda"), "gk": 1 + 0.1 * torch.randn(D, generator=g, device="cuda"),
         "pos": torch.arange(T, device="cuda", dtype=torch.int32)[None], "freq": 1e4 ** (-torch.arange(64, device="cuda") / 64.0)}
    out = TH.run_grad(d, "bf16")
    check_dgamma(d, out["gq"], out["gk"])
    rows = torch.tensor([0, 555555, T - 2, T - 1], device="cuda")
    at = {**d, "q": d["q"][rows], "k": d["k"][rows], "dq": d["dq"][rows], "dk": d["dk"][rows], "pos": d["pos"][:, rows]}
    few = TH.run_grad(at, "bf16")
    TH.check_grad(at, "bf16", few)
    assert torch.equal(few["q"], out["q"][rows]) and torch.equal(few["k"], out["k"][rows])

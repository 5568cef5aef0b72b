"""moe_distill_loss with more than 512 rows: workgroups of 256 to 1024 threads by the vocabulary, rows that read their
gradient's second time from memory or from the cache. Tolerances as derived in test_distill."""
import pytest

import test_distill as TD

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CASES = [(513, 5000, 7, "bf16"),                               # 256 threads a row
         (600, 9001, 33, "f32"), (700, 9001, 5, "f16"),         # 320
         (600, 20011, 64, "f16"), (513, 48001, 20, "f32"),      # 512
         (513, 50001, 20, "f32"), (520, 100003, 3, "bf16")]     # 1024


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("T,V,k,dt", CASES)
def test_loss_and_gradient_of_many_rows(T, V, k, dt, rest):
    M = TD.lib_m()
    d = TD.inputs(T, V, k, dt, rest, 2.0, stride=3, shift=1)
    stats, kl, loss = TD.call(d, dt)
    TD.check_loss(d, kl, loss)
    gloss = torch.full((1,), 512.0, device="cuda")
    _, dS = TD.like(d)
    a = TD.call(d, dt, dS, gloss)
    # the loss does not depend on whether its gradient is asked for
    assert torch.equal(a[0], stats) and torch.equal(a[1], kl) and torch.equal(a[2], loss)
    TD.check_grad(d, dt, dS, 512.0)
    _, two = TD.like(d)
    M.moe_distill_loss_grad(d["S"], TD.sd(dt), d["ids"], d["y"], d["lse"], d["w"], 2.0, stats, two, gloss)
    TD.check_grad(d, dt, two, 512.0)
    again = TD.call(d, dt)
    assert all(torch.equal(x, y) for x, y in zip(again, (stats, kl, loss)))

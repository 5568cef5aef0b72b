"""The binding's refusals of the block's operators: what is missing or misshapen raises MpbError, as the rest does."""
import pytest

torch = pytest.importorskip("torch")


def lib_m():
    import mixed_precision_bit_amd as M
    return M


def refused(code, f, *args):
    M = lib_m()
    with pytest.raises(M.MpbError) as e:
        f(*args)
    assert e.value.code == code, str(e.value)


def test_missing_tensors():
    M = lib_m()
    h, f = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 128)
    g, ws, W = torch.ones(128), torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(8, 128)
    idx, A, B = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(2, 8, 128).bfloat16(), torch.zeros(2, 64, 8).bfloat16()
    o = [torch.zeros(4, 8), torch.zeros(4), torch.zeros(9, dtype=torch.int32), torch.zeros(8), torch.zeros(3)]
    refused(-1, M.moe_block_norm, f, None, M.MPB_BF16, None, g, g, 1.0, 1e-6, h, h)
    refused(-1, M.moe_block_norm_grad, f, h, M.MPB_BF16, None, g, g, 1.0, 1e-6, h, h, None, f, None, g, g, ws)
    for X, w, i in ((None, W, idx), (h, None, idx), (h, W, None)):
        refused(-1, M.moe_router_loss, X, M.MPB_BF16, w, None, i, None, 0.1, 0.1, *o, ws)
        refused(-1, M.moe_router_loss_grad, X, M.MPB_BF16, w, i, None, *o[:3], 0.1, 0.1, None, None, f, W, None, ws)
    ad = torch.zeros(4, dtype=torch.int32)
    for X, a, b in ((None, A, B), (h, None, B), (h, A, None)):
        refused(-1, M.moe_adapters, X, M.MPB_BF16, a, b, None, None, ad, None, torch.zeros(4, 64), ws)


def test_a_loss_gradient_of_several_values():
    M = lib_m()
    X, W, idx = torch.zeros(4, 128).bfloat16(), torch.zeros(8, 128), torch.zeros(4, 2, dtype=torch.int32)
    o = [torch.zeros(4, 8), torch.zeros(4), torch.zeros(9, dtype=torch.int32)]
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    for gloss in (torch.ones(3), torch.ones(0), torch.ones(2, 1)):
        refused(-2, M.moe_router_loss_grad, X, M.MPB_BF16, W, idx, None, *o, 0.1, 0.1, None, gloss, None, W, None, ws)
    refused(-1, M.moe_router_loss_grad, X, M.MPB_BF16, W, idx, None, *o, 0.1, 0.1, None, torch.ones(1, 1), None, W, None, ws)

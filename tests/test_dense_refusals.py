"""What DeviceLayer.distill refuses comes as the library's error, with the gradient asked for or not."""
import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("what,code", [("columns", -1), ("one row for all", -1), ("rows that overlap", -1), ("every second", -1),
                                       ("batches", -2), ("one row alone", -2)])
def test_logits_that_are_no_rows(what, code, grad):
    from mixed_precision_bit_amd import MpbError
    from mixed_precision_bit_amd.layer import DeviceLayer
    D = DeviceLayer.__new__(DeviceLayer)  # no device is needed to refuse
    D.device = "cpu"
    S = {"columns": torch.zeros(40, 3).t(), "one row for all": torch.zeros(1, 40).expand(3, 40),
         "rows that overlap": torch.as_strided(torch.zeros(200), (3, 40), (20, 1)), "every second": torch.zeros(3, 80)[:, ::2],
         "batches": torch.zeros(3, 4, 5), "one row alone": torch.zeros(3)}[what]
    with pytest.raises(MpbError) as e:
        D.distill(S, torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4), grad=grad)
    assert e.value.code == code, str(e.value)

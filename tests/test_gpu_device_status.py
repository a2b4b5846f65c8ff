"""The status words are read after all work on the device, on streams that do not block on the legacy one too."""
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import uvu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["attention", "plan"])
def test_status_waits_for_other_streams(which):
    plan = uvu.Plan("16x0e+16x1o", "1x0e+1x1o", 1)
    read = uvu.Attention.device_status if which == "attention" else plan.device_status
    assert read() == 0  # loads what the call needs
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # some 100 ms
    assert not side.query()
    assert read() == 0
    assert side.query()

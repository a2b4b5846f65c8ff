"""Limits of the arguments of the operators around a layer, and the optimiser's own checks: these tests need no GPU."""
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import optim, uvu

F32, BF16 = uvu.UVU_F32, uvu.UVU_BF16


def refused(f, *args):
    with pytest.raises(uvu.UVUError) as e:
        f(*args)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("channels, inner, fits", [(1024, 9, True), (4096, 9, True), (1, 36864, True), (8192, 1, True), (4096, 10, False), (1, 36865, False),
                                                   (4097, 2, False), (8193, 1, False), (65536, 65536, False)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_width_of_rms_norm(channels, inner, fits, dtype):
    """A batch without rows passes every check that one with rows does of its sizes, and launches nothing."""
    for call in (lambda: uvu.uvu_rms_norm_fwd(dtype, 0, channels, inner, 1e-5, None, None, None, None, None, None, None),
                 lambda: uvu.uvu_rms_norm_quant(dtype, 0, channels, inner, 1e-5, 128, None, None, None, None, None, None, None)):
        if fits:
            call()
        else:
            status, text = refused(call)
            assert status == 1 and "channels * inner" in text


def test_muon_groups_of_matrices():
    """A group that is added later is held to the same; one that is refused leaves the optimiser as it was."""
    matrix, vector, volume = (torch.zeros(s, requires_grad=True) for s in ((3, 4), (3,), (2, 3, 4, 5)))
    opt = optim.Muon([matrix])
    for bad in (vector, volume):
        with pytest.raises(ValueError, match="matrices"):
            opt.add_param_group({"params": [bad]})
        assert len(opt.param_groups) == 1
    opt.add_param_group({"params": [torch.zeros(2, 3, 4, requires_grad=True)], "lr": 0.1})
    assert [g["lr"] for g in opt.param_groups] == [0.02, 0.1]
    with pytest.raises(ValueError, match="matrices"):
        optim.Muon([{"params": [matrix]}, {"params": [vector]}])

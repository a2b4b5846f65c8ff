"""Edges of the operators around a layer (uvu_embed_*, uvu_rms_norm_*, uvu_orthogonalize, optim.Muon): what test_gpu_layer.py's cases
do not reach.  Tolerances as there, or from the arithmetic beside the test."""
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import uvu
from test_gpu_layer import nan_like, norm_case

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------------------------- RMS norm

@pytest.mark.parametrize("group", [0, 1, 32, 40, 64, 128])
@pytest.mark.parametrize("case", [(100, 16, 4), (9, 1000, 1), (33, 128, 9), (3, 8192, 1), (7, 1100, 1), (20001, 256, 1), (3000, 301, 1), (5000, 1024, 1)],
                         ids=lambda c: "x".join(map(str, c)))
def test_rms_norm_quant_is_the_forward_divided_and_rounded(case, group):
    """In fp32 the forward gives y itself: the scales are max |y| / 448, bit for bit, and the 8-bit values those of y / scale, rounded once
    (an IEEE division on the host, and PyTorch's rounding to e4m3 of values up to 448, which no host arithmetic disturbs)."""
    (x, res, _, _, gamma), _ = norm_case(case, "f32")
    n, width = case[0], case[1] * case[2]
    each = group or width
    groups = -(-width // each)
    q, s, h, y = torch.zeros(case, dtype=torch.float8_e4m3fn, device="cuda"), nan_like((n, groups)), nan_like(case), nan_like(case)
    uvu.rms_norm_quant(x, gamma, q, s, group=group, residual=res, h=h)
    uvu.rms_norm_fwd(x, gamma, y, residual=res, h=h)
    y = torch.nn.functional.pad(y.cpu().view(n, width), (0, groups * each - width)).view(n, groups, each)
    want = y.abs().amax(2) / 448
    assert torch.equal(s.cpu(), want)
    v = torch.where(want[:, :, None] > 0, y / want[:, :, None], 0.0).clamp(-448, 448).view(n, -1)[:, :width]
    assert torch.equal(q.cpu().view(n, width).float(), v.to(torch.float8_e4m3fn).float())

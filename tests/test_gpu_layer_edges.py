"""Edges of the operators around a layer (uvu_embed_*, uvu_rms_norm_*, uvu_orthogonalize, optim.Muon): what test_gpu_layer.py's cases
do not reach.  Tolerances as there, or from the arithmetic beside the test."""
import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import uvu
from oracle import layer
from test_gpu_layer import UNIT, nan_like, norm_case, rounded, values, within

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


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
@pytest.mark.parametrize("width", [24, 33, 512, 1000, 6003, 8192])
def test_rms_norm_of_any_size(width, eps, kind):
    """Rows whose squares leave fp32 at either end, beside others: with eps = 0 each is normalised, with 1e-5 the small ones stay small.

    Relative errors: rstd has the sum's (48 additions to a value, halved by the root) and few roundings, 2^-24 (24 + 8) at most, and so
    have y, with the result's rounding, and t = gamma dy, u = h rstd, mean(t u) in dx = dh + rstd (t - u mean), measured by its terms."""
    sizes = [1.0, 1e-30, 1e-25, 1e-21, 1e-19, 1e-8, 2e17, 1e18, 1e19, 1e30, 3e37]
    rng = np.random.default_rng(width)
    n = 5 * len(sizes)
    size = np.resize(sizes, n)[:, None]
    x, xr = rounded(rng.standard_normal((n, width)) * size, kind)
    dy, dyr = rounded(rng.standard_normal((n, width)), kind)
    gamma, gr = rounded(1 + 0.2 * rng.standard_normal(width), "f32")
    y, rstd, dx, dg = nan_like((n, width), kind), nan_like((n,)), nan_like((n, width), kind), nan_like((width,))
    uvu.rms_norm_fwd(x, gamma, y, rstd, eps=eps)
    ry, rr = layer.rms_norm(xr[:, :, None], gr, eps)
    within(rstd, rr, 32 * 2.0 ** -24 * rr, "rstd")
    within(y, ry[:, :, 0], (32 * 2.0 ** -24 + 1.01 * UNIT[kind]) * np.abs(ry[:, :, 0]) + 2.0 ** -133, "y")
    uvu.rms_norm_bwd(dy, x, gamma, rstd, dx, dg)
    rdx, rdg = layer.rms_norm_vjp(xr[:, :, None], gr, eps, dyr[:, :, None])
    t, u = dyr * gr, xr * rr[:, None]
    terms = rr[:, None] * (np.abs(t) + np.abs(u) * np.mean(np.abs(t * u), axis=1, keepdims=True))
    within(dx, rdx[:, :, 0], 128 * 2.0 ** -24 * terms + 1.01 * UNIT[kind] * np.abs(rdx[:, :, 0]) + 2.0 ** -133, "dx")
    within(dg, rdg, (n + 64) * 2.0 ** -24 * np.abs(dyr * u).sum(0), "dgamma")
    # the same rows to 8 bits: those of the forward in fp32
    if kind == "f32":
        q, s = torch.zeros(n, width, dtype=torch.float8_e4m3fn, device="cuda"), nan_like((n, 1))
        uvu.rms_norm_quant(x, gamma, q, s, group=0, eps=eps)
        want = y.cpu().abs().amax(1, keepdim=True) / 448
        assert torch.equal(s.cpu(), want)
        v = torch.where(want > 0, y.cpu() / want, 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(q.cpu().float(), v.float())


def test_rms_norm_of_any_eps():
    """The largest eps beside the largest rows."""
    x = torch.tensor([[1.0] * 40, [3e38] * 40, [2.0 ** 63] * 40], device="cuda")
    y, rstd = nan_like((3, 40)), nan_like((3,))
    uvu.rms_norm_fwd(x, torch.ones(40, device="cuda"), y, rstd, eps=3e38)
    ref = (values(x[:, :1])[:, 0] ** 2 + float(np.float32(3e38))) ** -0.5
    within(rstd, ref, 2.0 ** -20 * ref)  # the second is below 2^-126: 22 bits
    within(y, values(x) * ref[:, None], 2.0 ** -20 * np.abs(values(x) * ref[:, None]))

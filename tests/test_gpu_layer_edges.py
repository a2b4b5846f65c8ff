"""Edges of the operators around a layer (uvu_embed_*, uvu_rms_norm_*, uvu_orthogonalize, optim.Muon): what test_gpu_layer.py's cases
do not reach.  Tolerances as there, or from the arithmetic beside the test."""
import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import optim, uvu
from gpu_util import check, dev
from oracle import layer
from test_gpu_layer import (KINDS, MUON, TINY, TYPES, UNIT, embed_case, gradient, nan_like, near, near_dx, norm_case, ortho_limit, rounded,
                            values, within)
from test_gpu_layer import test_orthogonalize as orthogonalize_case
from test_gpu_workspace_bounds import Guarded

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------- embedding

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", [(40001, 119, 64, 1, 0), (20000, 300, 512, 1, 0), (9001, 3, 128, 1, 0), (300, 7, 24, 1, 0)], ids=lambda c: "x".join(map(str, c)))
def test_embedding_gradient_wherever_it_lies(case, kind):
    """Tensors that begin off 16 bytes give the same bits: the order of the sums does not depend on where they lie."""
    tokens, rows, c, _, _ = case
    _, ix, _, _, dout, _ = embed_case(case, kind)
    dout = dout.view(tokens, c)
    want = nan_like((rows, c), kind)
    uvu.embed_bwd(ix, dout, want)
    flat, out = torch.cat([dout.flatten()[:1], dout.flatten()]), nan_like((rows * c + 1,), kind)
    for d, o in ((flat[1:].view(tokens, c), nan_like((rows, c), kind)), (dout, out[1:].view(rows, c)), (flat[1:].view(tokens, c), out[1:].view(rows, c))):
        uvu.embed_bwd(ix, d, o)
        assert torch.equal(o, want)


@pytest.mark.parametrize("tokens", [500, 20000])
def test_embedding_of_many_rows(tokens):
    """A table of more than 2^24 rows, whose tokens are sorted in four passes, in one block and in several."""
    rows = 2 ** 24 + 77
    rng = np.random.default_rng(tokens)
    index = rng.integers(0, rows, size=tokens).astype(np.int32)
    index[:5], index[5:8] = rows - 1, (-1, rows, 2 ** 24)
    index[tokens // 2:] = index[:tokens - tokens // 2]
    ix, dout = dev(index), torch.randn(tokens, 2, device="cuda")
    dtable = nan_like((rows, 2))
    uvu.embed_bwd(ix, dout, dtable)
    keep = (index >= 0) & (index < rows)
    used, which = np.unique(index[keep], return_inverse=True)
    ref, size, count = layer.embed_vjp(which.astype(np.int32), values(dout)[keep][:, :, None], len(used), 1.0, 0)
    within(dtable[dev(used.astype(np.int64))], ref, (np.maximum(count, 1)[:, None] + 2) * 2.0 ** -24 * size)
    assert not dtable.index_fill_(0, dev(used.astype(np.int64)), 0.0).any()
    out = nan_like((tokens, 2))
    table = dtable
    table[:, 0] = torch.arange(rows, device="cuda") % 1000
    uvu.embed_fwd(ix, table, out)
    assert torch.equal(out[:, 0].cpu(), torch.from_numpy(np.where(keep, index % 1000, 0)).float()) and not out[:, 1].any()


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


@pytest.mark.parametrize("group", [0, 1, 32, 40, 64])
@pytest.mark.parametrize("case", [(40, 24, 1), (40, 33, 1), (40, 300, 1), (40, 512, 1), (40, 1000, 1), (40, 2003, 3), (40, 1024, 9)],
                         ids=lambda c: "x".join(map(str, c)))
def test_rms_norm_quant_of_any_size(case, group):
    """Scales of all sizes, of groups of zeros and of NaN, beside usual ones: those of the forward, and its values divided by them.  (Scales
    of y below 448 2^-126 are subnormal, and so are their quotients' remainders: the division is the card's there.)"""
    n, c, inner = case
    width = c * inner
    rng = np.random.default_rng(width)
    size = np.resize([1.0, 1e-22, 1e-30, 1e-36, 1e-44, 0.0, 1.0, np.nan], n)[:, None, None]
    x, _ = rounded(rng.standard_normal(case) * size, "f32")
    gamma, _ = rounded((1 + 0.2 * rng.standard_normal(c)) * np.resize([1.0] * 40 + [0.0] * 45 + [1e34] * 7, c), "f32")
    each = group or width
    groups = -(-width // each)
    q, s, y = torch.zeros(case, dtype=torch.float8_e4m3fn, device="cuda"), nan_like((n, groups)), nan_like(case)
    uvu.rms_norm_quant(x, gamma, q, s, group=group, eps=1e-5)
    uvu.rms_norm_fwd(x, gamma, y, eps=1e-5)
    y = torch.nn.functional.pad(y.cpu().view(n, width), (0, groups * each - width)).view(n, groups, each)
    want = y.abs().amax(2) / 448
    assert torch.equal(s.cpu().nan_to_num(-1.0), want.nan_to_num(-1.0))
    v = torch.where(want[:, :, None] == 0, 0.0, y / want[:, :, None]).clamp(-448, 448).view(n, -1)[:, :width]
    assert torch.equal(q.cpu().view(n, width).float().nan_to_num(-999.0), v.to(torch.float8_e4m3fn).float().nan_to_num(-999.0))


def test_rms_norm_of_any_eps():
    """The largest eps beside the largest rows."""
    x = torch.tensor([[1.0] * 40, [3e38] * 40, [2.0 ** 63] * 40], device="cuda")
    y, rstd = nan_like((3, 40)), nan_like((3,))
    uvu.rms_norm_fwd(x, torch.ones(40, device="cuda"), y, rstd, eps=3e38)
    ref = (values(x[:, :1])[:, 0] ** 2 + float(np.float32(3e38))) ** -0.5
    within(rstd, ref, 2.0 ** -20 * ref)  # the second is below 2^-126: 22 bits
    within(y, values(x) * ref[:, None], 2.0 ** -20 * np.abs(values(x) * ref[:, None]))


WIDE = [(5, 1024, 9), (1, 4096, 9), (3, 2731, 3), (7, 4000, 4), (700, 1024, 9), (2, 1, 8193), (4, 1000, 12)]  # rows of more than 8192 values


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("case", WIDE, ids=lambda c: "x".join(map(str, c)))
def test_rms_norm_wide(case, residual, kind):
    """Values and gradients; tensors that begin off 16 bytes, and results over operands, are the same within rounding; repeats bit for bit."""
    (x, res, dy, dh, gamma), (xr, rr, dyr, dhr, gr) = norm_case(case, kind)
    shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
    n = case[0]
    runs = []
    for move in (lambda t: t, lambda t: t.clone(), shift):
        a, b, c, d = (move(t) for t in (x, res, dy, dh))
        y, h, dx = (move(nan_like(case, kind)) for _ in range(3))
        rstd, dg = nan_like((n,)), nan_like(case[1:2])
        uvu.rms_norm_fwd(a, gamma, y, rstd, **(dict(residual=b, h=h) if residual else {}))
        h = h if residual else a
        uvu.rms_norm_bwd(c, h, gamma, rstd, dx, dg, dh=d if residual else None)
        hr = values(h)
        within(h, xr + rr if residual else xr, UNIT[kind] * np.abs(xr + rr) + TINY[kind], "h")
        ry, rrstd = layer.rms_norm(hr, gr, 1e-5)
        near(y, ry, kind, "y")
        near(rstd, rrstd, "f32", "rstd")
        rdx, rdg = layer.rms_norm_vjp(hr, gr, 1e-5, dyr, dhr if residual else None)
        near_dx(dx, rdx, hr, gr, dyr, dhr if residual else np.zeros_like(dhr), kind)
        near(dg, rdg, "f32", "dgamma")
        runs.append((y, h, rstd, dx, dg))
    assert all(torch.equal(p, q) for p, q in zip(runs[0], runs[1]))
    if residual:  # h over x, y over the residual; dx over dy
        xi, ri, di, dg, rstd = x.clone(), res.clone(), dy.clone(), nan_like(case[1:2]), nan_like((n,))
        uvu.rms_norm_fwd(xi, gamma, ri, rstd, residual=ri, h=xi)
        uvu.rms_norm_bwd(di, xi, gamma, rstd, di, dg, dh=dh)
        assert all(torch.equal(p, q) for p, q in zip(runs[0], (ri, xi, rstd, di, dg)))


@pytest.mark.parametrize("group", [0, 1, 40, 128, 512])
@pytest.mark.parametrize("case", [c for c in WIDE if c[0] < 100], ids=lambda c: "x".join(map(str, c)))
def test_rms_norm_wide_quant(case, group):
    test_rms_norm_quant_is_the_forward_divided_and_rounded(case, group)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shifted", [False, True])
def test_rms_norm_wide_quant_of_16_bits(shifted, kind):
    """Bytes of rows of 8193 and 9216 values, on and off the vectors' alignment, nothing written before or behind them."""
    for case in ((3, 2731, 3), (5, 1024, 9)):
        (x, res, _, _, gamma), _ = norm_case(case, kind)
        n, width = case[0], case[1] * case[2]
        at = 33 if shifted else 32
        flat = torch.full((n * width + 64,), 0x55, dtype=torch.uint8, device="cuda")
        q, s, h = flat[at:at + n * width].view(case), nan_like((n, -(-width // 96))), nan_like(case, kind)
        uvu.rms_norm_quant(x, gamma, q, s, group=96, residual=res, h=h)
        y = layer.rms_norm(values(h), values(gamma), 1e-5)[0].reshape(n, width)
        ref = layer.scales(y, 96)
        np.testing.assert_allclose(values(s), ref, rtol=2.0 ** -20)
        v = y / np.repeat(ref, 96, axis=1)[:, :width]
        got = q.view(torch.float8_e4m3fn).float().view(n, width)
        within(got, v, 0.5 * layer.e4m3_step(np.minimum(np.abs(v) * (1 + 2.0 ** -19), 448)) + 2.0 ** -19 * np.abs(v))
        assert (flat[:at] == 0x55).all() and (flat[at + n * width:] == 0x55).all()


def test_rms_norm_wide_of_any_size():
    """As test_rms_norm_of_any_size, for rows of 9216 values."""
    sizes = np.array([1.0, 1e-30, 1e-21, 2e17, 1e30, 3e37])
    x, xr = rounded(np.random.default_rng(3).standard_normal((6, 1024, 9)) * sizes[:, None, None], "f32")
    gamma, y, rstd, dx, dg = torch.ones(1024, device="cuda"), nan_like(x.shape), nan_like((6,)), nan_like(x.shape), nan_like((1024,))
    uvu.rms_norm_fwd(x, gamma, y, rstd, eps=0.0)
    ry, rr = layer.rms_norm(xr, np.ones(1024), 0.0)
    within(rstd, rr, 64 * 2.0 ** -24 * rr)
    within(y, ry, 64 * 2.0 ** -24 * np.abs(ry) + 2.0 ** -149)
    dy, dyr = rounded(np.random.default_rng(4).standard_normal(x.shape), "f32")
    uvu.rms_norm_bwd(dy, x, gamma, rstd, dx, dg)
    rdx, rdg = layer.rms_norm_vjp(xr, np.ones(1024), 0.0, dyr)
    u = xr * rr[:, None, None]
    terms = rr[:, None, None] * (np.abs(dyr) + np.abs(u) * np.mean(np.abs(dyr * u), axis=(1, 2), keepdims=True))
    within(dx, rdx, 128 * 2.0 ** -24 * terms + 2.0 ** -149)
    within(dg, rdg, 128 * 2.0 ** -24 * np.abs(dyr * u).sum((0, 2)))


# ----------------------------------------------------------------------------------- Newton-Schulz

CLUSTERS = [(2, 128, 512), (3, 40, 300), (1, 500, 100), (2, 40, 1800), (1, 113, 2000), (1, 1030, 17), (9, 128, 2048), (2, 31, 700)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", CLUSTERS, ids=lambda c: "x".join(map(str, c)))
def test_orthogonalize_clusters(case, kind):
    """Clusters of 2, 4 and 8 blocks, with rows that they share evenly and not."""
    orthogonalize_case(case, kind)


@pytest.mark.parametrize("eps", [0.0, 1e38])
@pytest.mark.parametrize("size", [1e36, 3e38])
@pytest.mark.parametrize("shape", [(30, 50), (300, 200)], ids=str)
def test_orthogonalize_largest_norms(shape, size, eps):
    """1 / (|G| + eps) below 2^-126.  Without steps each value has the norm's error (of 36 additions to a value, in fp32, halved by the root),
    the factor's rounding and the product's: 24 roundings of 2^-24 at most."""
    g, gr = rounded(np.random.default_rng(7).uniform(-1, 1, shape) * size, "f32")
    out = nan_like(shape)
    uvu.orthogonalize(g, out, steps=0, eps=eps)
    ref = gr / (np.linalg.norm(gr / size) * size + float(np.float32(eps)))
    within(out, ref, 24 * 2.0 ** -24 * np.abs(ref) + 2.0 ** -149)
    # with steps: the limit of test_orthogonalize_any_size, at this size
    uvu.orthogonalize(g, out, eps=0.0)
    check(values(out), layer.newton_schulz(gr / size, 5, MUON, 0.0)[-1], False)


@pytest.mark.parametrize("norm", [1e-9, 1e-11, 1e-13])
@pytest.mark.parametrize("shape", [(96, 160), (300, 200), (60, 2000)], ids=str)
def test_orthogonalize_far_below_eps(shape, norm):
    """Gradients whose norm is far below eps: X has values that two fp16 terms hold to 2^-44 at least.  Each of the steps writes X with that error
    and stretches what was there before by at most a, beside the products' errors of ortho_limit."""
    rng = np.random.default_rng(8)
    a = gradient(shape, rng)
    g, gr = rounded(a * (norm / np.linalg.norm(a)), "f32")
    out = nan_like(shape)
    uvu.orthogonalize(g, out, eps=1e-7)
    xs = layer.newton_schulz(gr, 5, MUON, 1e-7)
    held = 2.0 ** -44 * g.numel() ** 0.5 * sum(MUON[0] ** k for k in range(1, 6))
    assert np.linalg.norm(values(out) - xs[-1]) <= ortho_limit(xs, "f32") + held


@pytest.mark.parametrize("shape", [(30, 50), (300, 200)], ids=str)
def test_orthogonalize_beyond_its_range(shape):
    """a I + b P + c P P beyond 250 is not held: NaN, not wrong values."""
    g = torch.randn(shape, device="cuda")
    out = torch.zeros(shape, device="cuda")
    uvu.orthogonalize(g, out, steps=1, coefficients=(300.0, 0.0, 0.0))
    assert torch.isnan(out).all()


# --------------------------------------------------------------------------------------------- Muon

def muon_reference(start, grads, lr, momentum, nesterov, decay):
    """Parameters and momentum after the gradients, in fp64."""
    p, buf = start.copy(), np.zeros_like(start)
    for g in grads:
        buf = momentum * buf + (1 - momentum) * g
        u = ((1 - momentum) * g + momentum * buf if nesterov else buf).reshape(-1, *p.shape[-2:])
        o = np.stack([layer.newton_schulz(a, 5, MUON, 1e-7)[-1] for a in u]).reshape(p.shape)
        p = p * (1 - lr * decay) - lr * max(1, p.shape[-2] / p.shape[-1]) ** 0.5 * o
    return p, buf


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("nesterov", [True, False])
def test_muon_of_any_type(kind, nesterov):
    """Matrices, batches and a transposed parameter whose gradient is transposed too.  The momentum is fp32: each step rounds it three times
    at most.  A parameter has two roundings a step, of at most its largest value on the way, beside what gpu_util.check allows of an update."""
    rng = np.random.default_rng(13)
    steps, shapes = 12, [(3, 20, 12), (20, 12), (30, 44)]
    first = [rounded(rng.standard_normal(s), kind) for s in shapes]
    params = [t.clone().requires_grad_(True) for t, _ in first]
    params[2] = first[2][0].t().contiguous().t().requires_grad_(True)
    assert not params[2].is_contiguous()
    grads = [[rounded(0.5 + rng.standard_normal(s), kind) for s in shapes] for _ in range(steps)]
    opt = optim.Muon(params, lr=0.05, momentum=0.9, nesterov=nesterov, weight_decay=0.01)
    for step in grads:
        for p, (g, _) in zip(params, step):
            p.grad = g.clone()
        params[2].grad = step[2][0].t().contiguous().t()
        opt.step()
    for i, p in enumerate(params):
        ref, buf = muon_reference(first[i][1], [g[i][1] for g in grads], 0.05, 0.9, nesterov, 0.01)
        got = opt.state[p]["momentum"]
        assert got.dtype == torch.float32 and p.dtype == first[i][0].dtype
        within(got, buf, 3 * steps * 2.0 ** -24 * max(np.abs(g[i][1]).max() for g in grads), "momentum")
        largest = max(np.abs(first[i][1]).max(), np.abs(ref).max()) + 0.05 * steps
        within(p.detach(), ref, 2 * steps * UNIT[kind] * largest * (kind != "f32") + 1e-4 * (1 + np.abs(ref)), "parameter")


@pytest.mark.parametrize("kind", KINDS)
def test_muon_goes_on_from_a_saved_state(kind):
    rng = np.random.default_rng(14)
    start, _ = rounded(rng.standard_normal((24, 40)), kind)
    grads = [rounded(rng.standard_normal((24, 40)), kind)[0] for _ in range(3)]
    a, b = (start.clone().requires_grad_(True) for _ in range(2))
    opt = optim.Muon([a])
    for g in grads[:2]:
        a.grad = g
        opt.step()
    again = optim.Muon([b], lr=0.5)
    again.load_state_dict(opt.state_dict())
    b.data.copy_(a.data)
    assert again.state[b]["momentum"].dtype == torch.float32 and torch.equal(again.state[b]["momentum"], opt.state[a]["momentum"])
    for p, o in ((a, opt), (b, again)):
        p.grad = grads[2]
        o.step()
    assert torch.equal(a, b) and torch.equal(again.state[b]["momentum"], opt.state[a]["momentum"])


def test_muon_of_many_matrices():
    """More matrices of one size than a call takes."""
    n = 70_000
    g = torch.randn(n, 2, 3, device="cuda")
    p = torch.zeros(n, 2, 3, device="cuda", requires_grad=True)
    p.grad = g
    optim.Muon([p], lr=1.0, momentum=0.0).step()
    for part in (slice(0, 50), slice(65530, 65540), slice(n - 50, n)):
        want = torch.empty_like(g[part])
        uvu.orthogonalize(g[part].contiguous(), want)
        assert torch.equal(p.detach()[part], -want)


# --------------------------------------------------------------------------------- as they are used

def test_graphs_of_every_sort():
    """The sort in several blocks, and the one beside which a large table is zeroed, on a side stream and in two captured graphs."""
    rng = np.random.default_rng(15)
    cases = []
    for tokens, rows in ((20000, 3000), (3000, 70000), (40000, 70000)):
        cases.append((dev(rng.integers(-1, rows, size=tokens).astype(np.int32)), torch.randn(tokens, 32, device="cuda"), rows))

    def new():
        return [nan_like((rows, 32)) for _, _, rows in cases]

    def step(out, **kw):
        for (ix, dout, _), o in zip(cases, out):
            uvu.embed_bwd(ix, dout, o, **kw)

    want, got, side = new(), new(), torch.cuda.Stream()
    step(want)
    side.wait_stream(torch.cuda.current_stream())
    step(got, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs, graphs = [new(), new()], []
    for o in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(o)
    for _ in range(2):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("off", [0, 1], ids=["aligned", "off"])
def test_workspaces_hold_what_they_are_asked_for(kind, off):
    """Workspaces of exactly the bytes that are asked for, of gradients on and off 16 bytes: nothing is written behind them, nor behind results."""
    g = Guarded()

    def at(t):
        return torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape) if off else t

    for case in ((300, 119, 64, 1, 0), (40001, 119, 64, 1, 0), (20000, 70000, 24, 1, 0), (5000, 9, 33, 4, 2), (9, 3, 7, 1, 0)):
        tokens, rows, c, inner, column = case
        _, ix, _, _, dout, _ = embed_case(case, kind)
        dout, dtable = at(dout), g.out(rows, c, dtype=TYPES[kind])
        uvu.embed_bwd(ix, dout, dtable, column=column, workspace=g.ws(uvu.embed_workspace_bytes(dout, dtable)))
    for case in ((5000, 128, 4), (3, 8191, 1), (70001, 5, 1), (6001, 427, 1), (1, 3, 1), (700, 1024, 9), (3, 2731, 3)):
        x, _, dy, dh, gamma = norm_case(case, kind)[0]
        x, dy, dh = at(x), at(dy), at(dh)
        y, rstd = torch.empty_like(x), g.out(case[0])
        uvu.rms_norm_fwd(x, gamma, y, rstd)
        uvu.rms_norm_bwd(dy, x, gamma, rstd, g.out(*case, dtype=TYPES[kind]), g.out(case[1]), dh=dh, workspace=g.ws(uvu.rms_norm_workspace_bytes(x)))
    for case in ((2, 128, 512), (12, 40, 1800), (3, 129, 127), (2, 256, 256), (1, 700, 301), (1, 1, 1)):
        a = at(torch.randn(case, device="cuda").to(TYPES[kind]))
        need = uvu.orthogonalize_workspace_bytes(a)
        for steps in (0, 1, 5):
            uvu.orthogonalize(a, g.out(*case, dtype=TYPES[kind]), steps=steps, workspace=g.ws(need))
    g.check()
    assert uvu.orthogonalize_device_status() == 0

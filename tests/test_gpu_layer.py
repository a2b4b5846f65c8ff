"""GPU parity of the operators around a layer (uvu_embed_*, uvu_rms_norm_*, uvu_orthogonalize) with the fp64 oracle
(oracle.layer), their edges, and a training step that uses them together.

Tolerances, from the arithmetic.  u: half a step of the result's type.  Embedding: one fp32 product (2^-24) and the result's
rounding; its gradient: n - 1 fp32 additions of a row's n terms (2^-24 of the terms' magnitudes each), a product and the rounding.
RMS norm: fp32 results as gpu_util.check has them; 16-bit results u of the value beside 1e-4 (1 + |ref|) for fp32's arithmetic.
8 bits: half a step at the value of y / s, and what 2^-20 of y moves.  Newton-Schulz: see ortho_limit."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import autograd, optim, uvu
from gpu_util import check, dev
from oracle import layer

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}  # the smallest magnitude
KINDS = list(TYPES)
MUON = uvu.MUON


def rounded(a, kind):
    """A device tensor of the type, and the fp64 values that it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TYPES[kind])
    return t.cuda(), t.double().numpy()


def values(t):
    return t.double().cpu().numpy()


def within(got, ref, bound, what=""):
    got = values(got)
    assert got.shape == ref.shape, what
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{what}: {(~(over <= 0)).sum()} elements beyond their bound, by up to {over.max():.3e}"


def near(got, ref, kind, what=""):
    if kind == "f32":
        return check(values(got), ref, False, what)
    within(got, ref, UNIT[kind] * np.abs(ref) + 1e-4 * (1 + np.abs(ref)), what)


def nan_like(shape, kind="f32"):
    return torch.full(shape, float("nan"), dtype=TYPES[kind], device="cuda")


# ------------------------------------------------------------------------------------- embedding

# tokens, rows, channels, inner, column
EMBEDS = [(1, 1, 1, 1, 0), (1, 70000, 8, 1, 0), (61, 10, 128, 4, 0), (61, 10, 128, 4, 3), (5, 3, 7, 9, 4), (33, 300, 40, 1, 0),
          (1000, 1, 24, 1, 0), (1000, 5, 33, 1, 0), (257, 256, 16, 1, 0), (3000, 255, 12, 2, 1), (2049, 66000, 9, 1, 0), (9001, 89, 128, 4, 0),
          (20000, 3, 1100, 1, 0), (40001, 119, 64, 1, 0), (300, 100, 5, 1, 0), (70000, 2000, 20, 1, 0), (12000, 65536, 256, 1, 0),
          (16384, 7, 40, 1, 0), (16385, 70000, 8, 1, 0), (30000, 4, 16, 9, 2)]


def embed_case(case, kind, pad=True):
    tokens, rows, c, inner, column = case
    rng = np.random.default_rng(tokens * 31 + rows)
    index = np.minimum((rng.random(tokens) ** 3 * rows).astype(np.int32), rows - 1)
    if pad and tokens > 4:
        index[rng.random(tokens) < 0.1] = -1
        index[1], index[3] = rows, 2 ** 31 - 1
    table, tr = rounded(rng.standard_normal((rows, c)), kind)
    dout, dr = rounded(rng.standard_normal((tokens, c, inner)), kind)
    return index, dev(index), table, tr, dout, dr


def embed_bound(ref, kind):
    return (UNIT[kind] * 1.001 + 2.0 ** -24) * np.abs(ref) + TINY[kind]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", EMBEDS, ids=lambda c: "x".join(map(str, c)))
def test_embedding(case, kind):
    tokens, rows, c, inner, column = case
    index, ix, table, tr, dout, dr = embed_case(case, kind)
    scale = float(np.float32(c ** 0.5))
    out, dtable = nan_like((tokens, c, inner), kind), nan_like((rows, c), kind)
    uvu.embed_fwd(ix, table, out, scale=scale, column=column)
    uvu.embed_bwd(ix, dout, dtable, scale=scale, column=column)
    ref = layer.embed(index, tr, scale, inner, column)
    within(out, ref, embed_bound(ref, kind), "out")
    ref, size, count = layer.embed_vjp(index, dr, rows, scale, column)
    within(dtable, ref, embed_bound(ref, kind) + np.maximum(count, 1)[:, None] * 2.0 ** -24 * size, "dtable")
    empty = torch.from_numpy(count == 0).cuda()
    assert not dtable[empty].any()


def test_embedding_sums_are_not_lost():
    """300,000 equal values of one row: a running fp32 sum in one go would be off by more than the check allows."""
    n = 300_001
    index, dout = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n, 8), 0.1, device="cuda")
    dtable = nan_like((2, 8))
    uvu.embed_bwd(index, dout, dtable)
    ref = n * float(np.float32(0.1))
    assert (values(dtable[0]) / ref - 1 < 1e-5).all() and (1 - values(dtable[0]) / ref < 1e-5).all() and not dtable[1].any()


@pytest.mark.parametrize("kind", KINDS)
def test_embedding_gradient_keeps_infinities(kind):
    """Rows whose tokens lie in one piece, a few, and many: an infinity's sum is that infinity, a NaN's and that of both signs NaN."""
    counts = (3, 96, 1536, 9216)  # halves of them are values of every type
    index = torch.repeat_interleave(torch.arange(4, dtype=torch.int32), torch.tensor(counts))
    dout = torch.full((len(index), 5), 0.5)
    for first, n in zip(np.cumsum((0,) + counts), counts):
        dout[first + n // 2, 0] = dout[first, 3] = float("inf")
        dout[first + n - 1, 1] = dout[first + 1, 3] = -float("inf")
        dout[first, 2] = float("nan")
    dtable = nan_like((4, 5), kind)
    uvu.embed_bwd(index.cuda(), dout.to(dtable.dtype).cuda(), dtable)
    inf = np.inf
    np.testing.assert_array_equal(values(dtable), [[inf, -inf, np.nan, np.nan, n / 2] for n in counts])


@pytest.mark.parametrize("kind", KINDS)
def test_embedding_views_and_padding(kind):
    """Tensors that begin off a 16-byte boundary; a batch of padding alone; NaN in rows and cotangents that nothing picks."""
    index, ix, table, tr, dout, dr = embed_case((500, 40, 64, 1, 0), kind)
    flat = nan_like((40 * 64 + 1,), kind)
    flat[1:] = table.flatten()
    out, dflat = nan_like((500 * 64 + 1,), kind), nan_like((500 * 64 + 1,), kind)
    dflat[1:] = dout.flatten()
    dflat[1:].view(500, 64)[ix < 0] = float("nan")
    for tb, o, d in ((flat[1:].view(40, 64), out[1:].view(500, 64), dflat[1:].view(500, 64)),):
        uvu.embed_fwd(ix, tb, o)
        ref = layer.embed(index, tr, 1.0, 1, 0)[:, :, 0]
        within(o, ref, embed_bound(ref, kind))
        dt = nan_like((40 * 64 + 1,), kind)
        uvu.embed_bwd(ix, d, dt[1:].view(40, 64))
        ref, size, count = layer.embed_vjp(index, dr, 40, 1.0, 0)
        within(dt[1:].view(40, 64), ref, embed_bound(ref, kind) + np.maximum(count, 1)[:, None] * 2.0 ** -24 * size)
        assert torch.isnan(dt[0]) and torch.isnan(out[0])
    none, dt, o = torch.full((7,), -1, dtype=torch.int32, device="cuda"), nan_like((40, 64), kind), nan_like((7, 64), kind)
    uvu.embed_fwd(none, nan_like((40, 64), kind), o)
    uvu.embed_bwd(none, nan_like((7, 64), kind), dt)
    assert not o.any() and not dt.any()


def test_embedding_of_no_tokens():
    none, dt = torch.empty(0, dtype=torch.int32, device="cuda"), nan_like((9, 4))
    uvu.embed_fwd(none, dt, torch.empty(0, 4, device="cuda"))
    uvu.embed_bwd(none, torch.empty(0, 4, device="cuda"), dt)
    assert (dt == 0).all()


def test_embedding_repeats_bit_for_bit():
    for case in ((40001, 119, 64, 1, 0), (9001, 5000, 100, 1, 0), (700, 20, 32, 4, 0)):
        _, ix, table, _, dout, _ = embed_case(case, "f32")
        runs = [nan_like(tuple(table.shape)) for _ in range(3)]
        for r in runs:
            uvu.embed_bwd(ix, dout, r)
        assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


# -------------------------------------------------------------------------------------- RMS norm

# rows, channels, inner
NORMS = [(1, 1, 1), (100, 16, 4), (7, 24, 1), (33, 7, 9), (5, 40, 1), (300, 128, 4), (17, 512, 1), (64, 100, 1), (9, 1000, 1), (3, 1024, 1),
         (5, 1025, 1), (2, 333, 9), (11, 2048, 1), (3, 8192, 1), (4, 8190, 1), (3, 8191, 1), (20011, 96, 1), (3000, 513, 1), (70001, 4, 1), (9001, 1024, 1), (30001, 512, 1), (2500, 2048, 1), (20000, 33, 9)]


def norm_case(case, kind):
    rng = np.random.default_rng(sum(case))
    x, xr = rounded(rng.standard_normal(case) * 1.5 + 0.4, kind)
    res, rr = rounded(2 * rng.standard_normal(case), kind)
    dy, dyr = rounded(rng.standard_normal(case), kind)
    dh, dhr = rounded(rng.standard_normal(case), kind)
    gamma, gr = rounded(1 + 0.2 * rng.standard_normal(case[1]), "f32")
    return (x, res, dy, dh, gamma), (xr, rr, dyr, dhr, gr)


def near_dx(got, ref, h, gamma, dy, dh, kind):
    """dx = dh + r (t - u m), m = mean(t u), cancels in rows of few values (one value: t - u^2 t, all but nothing), so its error
    is measured by its terms: t has one rounding, r and u = h r three each (a sum's error halved by the root, the root, the
    quotient), m at most 48 additions to a value (32 in a thread, 16 over threads), so r 2^-24 (8 |t| + 64 |u| mean|t u|)
    and a rounding of the sum with dh covers them."""
    rstd = layer.rms_norm(h, gamma, 1e-5)[1][:, None, None]
    t, u = dy * gamma[None, :, None], h * rstd
    terms = rstd * (8 * np.abs(t) + 64 * np.abs(u) * np.mean(np.abs(t * u), axis=(1, 2), keepdims=True))
    within(got, ref, 2.0 ** -24 * (terms + np.abs(ref)) + UNIT[kind] * (np.abs(ref) + 2.0 ** -24 * terms) + TINY[kind], "dx")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("case", NORMS, ids=lambda c: "x".join(map(str, c)))
def test_rms_norm(case, residual, kind):
    (x, res, dy, dh, gamma), (xr, rr, dyr, dhr, gr) = norm_case(case, kind)
    y, rstd, dx, dg = nan_like(case, kind), nan_like(case[:1]), nan_like(case, kind), nan_like(case[1:2])
    h, hr = x, xr
    if residual:
        h = nan_like(case, kind)
        uvu.rms_norm_fwd(x, gamma, y, rstd, residual=res, h=h)
        within(h, xr + rr, UNIT[kind] * np.abs(xr + rr) + TINY[kind], "h")
        hr = values(h)
    else:
        uvu.rms_norm_fwd(x, gamma, y, rstd)
    uvu.rms_norm_bwd(dy, h, gamma, rstd, dx, dg, dh=dh if residual else None)
    ry, rrstd = layer.rms_norm(hr, gr, 1e-5)
    near(y, ry, kind, "y")
    near(rstd, rrstd, "f32", "rstd")
    rdx, rdg = layer.rms_norm_vjp(hr, gr, 1e-5, dyr, dhr if residual else None)
    near_dx(dx, rdx, hr, gr, dyr, dhr, kind)
    near(dg, rdg, "f32", "dgamma")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("width", [64, 66, 4100])
def test_rms_norm_views_and_in_place(kind, width):
    """Tensors off a 16-byte boundary, and results over operands, are those of separate ones bit for bit where the threads' columns
    are the same, else within rounding."""
    case = (50, width, 1)
    (x, res, dy, dh, gamma), (xr, rr, dyr, dhr, gr) = norm_case(case, kind)
    shift = lambda t: torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape)  # noqa: E731
    x1, r1, d1, e1 = (shift(t) for t in (x, res, dy, dh))
    assert x1.data_ptr() % 16
    y, h, rstd = shift(x), shift(x), nan_like((50,))
    uvu.rms_norm_fwd(x1, gamma, y, rstd, residual=r1, h=h)
    hr = values(h)
    within(h, xr + rr, UNIT[kind] * np.abs(xr + rr) + TINY[kind])
    near(y, layer.rms_norm(hr, gr, 1e-5)[0], kind)
    dx, dg = shift(x), nan_like((width,))
    uvu.rms_norm_bwd(d1, h, gamma, rstd, dx, dg, dh=e1)
    ref = layer.rms_norm_vjp(hr, gr, 1e-5, dyr, dhr)
    near(dx, ref[0], kind)
    near(dg, ref[1], "f32")
    # h over x, y over the residual; dx over dy
    want_y, want_h = nan_like(case, kind), nan_like(case, kind)
    uvu.rms_norm_fwd(x, gamma, want_y, rstd, residual=res, h=want_h)
    want_dx = nan_like(case, kind)
    uvu.rms_norm_bwd(dy, want_h, gamma, rstd, want_dx, dg, dh=dh)
    xi, ri, di = x.clone(), res.clone(), dy.clone()
    uvu.rms_norm_fwd(xi, gamma, ri, rstd, residual=ri, h=xi)
    uvu.rms_norm_bwd(di, xi, gamma, rstd, di, dg, dh=dh)
    assert torch.equal(xi, want_h) and torch.equal(ri, want_y) and torch.equal(di, want_dx)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", [(1, 3, 1), (2, 3, 1), (3, 521, 1), (4001, 521, 1), (2003, 1021, 1), (1001, 333, 3), (70001, 5, 1), (6001, 427, 1)],
                         ids=lambda c: "x".join(map(str, c)))
def test_rms_norm_odd_rows(case, kind):
    """Rows of odd length, whose words begin a value off in every other one: values and gradients, nothing written before, between
    or behind them, results over operands, and the same bits again."""
    (x, res, dy, dh, gamma), (xr, rr, dyr, dhr, gr) = norm_case(case, kind)
    n, count = case[0], x.numel()

    def framed(t=None):
        f = nan_like((count + 16,), kind)
        if t is not None:
            f[8:-8] = t.flatten()
        return f, f[8:-8].view(case)

    (fy, y), (fh, h), (fx, dx), rstd, dg = framed(), framed(), framed(), nan_like((n,)), nan_like(case[1:2])
    uvu.rms_norm_fwd(x, gamma, y, rstd, residual=res, h=h)
    uvu.rms_norm_bwd(dy, h, gamma, rstd, dx, dg, dh=dh)
    hr = values(h)
    within(h, xr + rr, UNIT[kind] * np.abs(xr + rr) + TINY[kind], "h")
    near(y, layer.rms_norm(hr, gr, 1e-5)[0], kind, "y")
    rdx, rdg = layer.rms_norm_vjp(hr, gr, 1e-5, dyr, dhr)
    near_dx(dx, rdx, hr, gr, dyr, dhr, kind)
    near(dg, rdg, "f32", "dgamma")
    for f in (fy, fh, fx):
        assert torch.isnan(f[:8]).all() and torch.isnan(f[-8:]).all()
    (_, xi), (_, ri), (_, di), dg2 = framed(x), framed(res), framed(dy), nan_like(case[1:2])
    uvu.rms_norm_fwd(xi, gamma, ri, rstd, residual=ri, h=xi)
    uvu.rms_norm_bwd(di, xi, gamma, rstd, di, dg2, dh=dh)
    assert torch.equal(xi, h) and torch.equal(ri, y) and torch.equal(di, dx) and torch.equal(dg2, dg)


def test_rms_norm_rows_apart():
    """A row of NaN, of an infinity and of zeros leaves the others as they are; a sum over many equal rows keeps its bits."""
    x = torch.randn(9, 48, device="cuda")
    gamma = torch.ones(48, device="cuda")
    clean, y = nan_like((9, 48)), nan_like((9, 48))
    uvu.rms_norm_fwd(x, gamma, clean)
    x[2], x[4, 3], x[6] = float("nan"), float("inf"), 0
    uvu.rms_norm_fwd(x, gamma, y)
    others = [0, 1, 3, 5, 7, 8]
    assert torch.equal(y[others], clean[others]) and torch.isnan(y[2]).all() and (y[6] == 0).all() and torch.isnan(y[4, 3])
    n = 400_000
    h, dy, rstd = torch.ones(n, 8, device="cuda"), torch.full((n, 8), 0.1, device="cuda"), torch.ones(n, device="cuda")
    dx, dg = nan_like((n, 8)), nan_like((8,))
    uvu.rms_norm_bwd(dy, h, torch.ones(8, device="cuda"), rstd, dx, dg)
    assert np.abs(values(dg) / (n * float(np.float32(0.1))) - 1).max() < 1e-5


def test_rms_norm_of_no_rows_and_repeats():
    dg, none = nan_like((8,)), torch.empty(0, 8, device="cuda")
    uvu.rms_norm_fwd(none, torch.ones(8, device="cuda"), none)
    uvu.rms_norm_bwd(none, none, torch.ones(8, device="cuda"), torch.empty(0, device="cuda"), none, dg)
    assert (dg == 0).all()
    (x, _, dy, dh, gamma), _ = norm_case((5000, 100, 1), "bf16")
    runs = []
    for _ in range(2):
        y, rstd, dx, dg = nan_like(x.shape, "bf16"), nan_like((5000,)), nan_like(x.shape, "bf16"), nan_like((100,))
        uvu.rms_norm_fwd(x, gamma, y, rstd)
        uvu.rms_norm_bwd(dy, x, gamma, rstd, dx, dg, dh=dh)
        runs.append((y, rstd, dx, dg))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [0, 1, 32, 40, 64, 128])
@pytest.mark.parametrize("case", [(1, 1, 1), (100, 16, 4), (9, 1000, 1), (5, 129, 1), (33, 128, 9), (3, 8192, 1), (7, 1100, 1), (301, 256, 1), (20001, 256, 1), (3000, 301, 1), (2, 7, 1), (2001, 777, 1)],
                         ids=lambda c: "x".join(map(str, c)))
def test_rms_norm_quant(case, group, kind):
    (x, res, _, _, gamma), (xr, rr, _, _, gr) = norm_case(case, kind)
    n, width = case[0], case[1] * case[2]
    groups = -(-width // group) if group else 1
    q, s, h = torch.zeros(case, dtype=torch.float8_e4m3fn, device="cuda"), nan_like((n, groups)), nan_like(case, kind)
    uvu.rms_norm_quant(x, gamma, q, s, group=group, residual=res, h=h)
    within(h, xr + rr, UNIT[kind] * np.abs(xr + rr) + TINY[kind])
    y = layer.rms_norm(values(h), gr, 1e-5)[0].reshape(n, width)
    ref = layer.scales(y, group)
    np.testing.assert_allclose(values(s), ref, rtol=2.0 ** -20)  # y: a sum's fp32 error halved by the root, three products
    each = np.repeat(ref, group or width, axis=1)[:, :width]
    v = np.divide(y, each, out=np.zeros_like(y), where=each > 0)
    # half a step at the value; where 2^-19 of it crosses into the next binade, that one's
    within(q.float().view(n, width), v, 0.5 * layer.e4m3_step(np.minimum(np.abs(v) * (1 + 2.0 ** -19), 448)) + 2.0 ** -19 * np.abs(v))


def test_rms_norm_quant_edges():
    x = torch.randn(6, 64, device="cuda")
    x[1], x[2, 40], x[3] = 0, float("nan"), 1e-30
    q, s = torch.full((6, 64), 1.0, device="cuda").to(torch.float8_e4m3fn), nan_like((6, 2))
    uvu.rms_norm_quant(x, torch.ones(64, device="cuda"), q, s, group=32, eps=1e-5)
    assert (q[1].float() == 0).all() and (s[1] == 0).all()
    assert torch.isnan(q[2].float()).all() and torch.isnan(s[2]).all()  # the norm is of the row
    assert torch.isfinite(q[3].float()).all() and (q[3].float().abs() == 448).all()
    as_bytes = torch.zeros(6, 64, dtype=torch.uint8, device="cuda")
    uvu.rms_norm_quant(x, torch.ones(64, device="cuda"), as_bytes, s, group=32)
    assert torch.equal(as_bytes, q.view(torch.uint8))


# ----------------------------------------------------------------------------------- Newton-Schulz

def ortho_limit(xs, kind):
    """Of the Frobenius error of X_n.  A step's products are of fp32 accuracy, 2^-22 of their factors' norms at most (the terms'
    roundings and the sums'): P, P P and the product with X move X_(k+1) by (|a| + 3 |b| + 5 |c|) 2^-22 |X_k|_F at most, as
    |P| < 1.7 in the spectral norm.  The steps after it stretch a difference by at most a each (the slope of the polynomial is
    largest at zero).  16-bit results add their rounding."""
    a, b, c = (abs(v) for v in MUON)
    n = len(xs) - 1
    moved = 2.0 ** -22 * np.linalg.norm(xs[0]) * a ** n
    moved += sum((a + 3 * b + 5 * c) * 2.0 ** -22 * np.linalg.norm(xs[k]) * a ** (n - 1 - k) for k in range(n))
    return moved + (0 if kind == "f32" else UNIT[kind] * np.linalg.norm(xs[-1]) + TINY[kind] * xs[-1].size ** 0.5)


def gradient(shape, rng, few=None):
    m, n = shape
    few = few or max(1, min(m, n) // 8)
    return 1e-3 * (rng.standard_normal((m, few)) @ rng.standard_normal((few, n)) / few ** 0.5 + 0.3 * rng.standard_normal((m, n)))


ORTHOS = [(1, 1, 1), (2, 1, 40), (1, 40, 1), (3, 5, 7), (13, 128, 128), (2, 64, 1664), (1, 1664, 64), (4, 100, 130), (3, 129, 127), (1, 17, 3000),
          (2, 256, 256), (1, 300, 700), (1, 700, 301), (1, 513, 640), (1, 128, 4100), (12, 40, 1800), (2, 127, 2049), (1, 1000, 1000), (40, 24, 16)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", ORTHOS, ids=lambda c: "x".join(map(str, c)))
def test_orthogonalize(case, kind):
    rng = np.random.default_rng(sum(case))
    g, gr = rounded(np.stack([gradient(case[1:], rng) for _ in range(case[0])]), kind)
    out = nan_like(case, kind)
    uvu.orthogonalize(g, out)
    for i in range(case[0]):
        xs = layer.newton_schulz(gr[i], 5, MUON, 1e-7)
        err, most = np.linalg.norm(values(out[i]) - xs[-1]), ortho_limit(xs, kind)
        assert err <= most, f"matrix {i}: {err:.3e} > {most:.3e} (norm {np.linalg.norm(xs[-1]):.3e})"
    if kind == "f32" and case != (1, 1, 1):
        # what the limit cannot see: each value against fp32's usual error, with the steps' stretching of it
        check(values(out), np.stack([layer.newton_schulz(a, 5, MUON, 1e-7)[-1] for a in gr]), False)


@pytest.mark.parametrize("shape", [(640, 650), (650, 600)], ids=str)
def test_orthogonalize_many_large(shape):
    """Enough matrices that the widest tiles are taken, of an odd number of row blocks: copies give the same results."""
    rng = np.random.default_rng(12)
    g, gr = rounded(gradient(shape, rng), "f32")
    out = nan_like((16, *shape))
    uvu.orthogonalize(g.expand(16, -1, -1), out)
    check(values(out[0]), layer.newton_schulz(gr, 5, MUON, 1e-7)[-1], False)
    assert all(torch.equal(out[0], o) for o in out)


@pytest.mark.parametrize("steps, coefficients, eps, scale", [(0, MUON, 1e-7, 2.0), (1, (2.0, -1.5, 0.5), 0.0, 1.0), (9, (1.875, -1.25, 0.375), 1e-3, -0.5)],
                         ids=["none", "one", "nine"])
@pytest.mark.parametrize("shape", [(24, 60), (200, 150)], ids=str)
def test_orthogonalize_options(shape, steps, coefficients, eps, scale):
    rng = np.random.default_rng(5)
    g, gr = rounded(rng.standard_normal(shape), "f32")
    out = nan_like(shape)
    uvu.orthogonalize(g, out, steps=steps, coefficients=coefficients, eps=eps, scale=scale)
    check(values(out), scale * layer.newton_schulz(gr, steps, coefficients, eps)[-1], False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [(20, 33), (128, 128), (260, 140), (65, 600)], ids=str)
def test_orthogonalize_views_and_in_place(shape, kind):
    """Strides, views off a 16-byte boundary, out over g; the values beside a view stay as they were."""
    rng = np.random.default_rng(6)
    m, n = shape
    g, gr = rounded(np.stack([gradient(shape, rng) for _ in range(2)]), kind)
    want = nan_like((2, m, n), kind)
    uvu.orthogonalize(g, want)
    big = torch.full((4, m + 1, n + 5), 7.0, device="cuda").to(TYPES[kind])
    view = big[::2, 1:, 3:n + 3]
    view.copy_(g)
    out = torch.full((2, m, n + 3), 9.0, device="cuda").to(TYPES[kind])
    uvu.orthogonalize(view, out[:, :, 1:n + 1])
    assert torch.equal(out[:, :, 1:n + 1], want) and (out[:, :, 0] == 9).all() and (out[:, :, n + 1:] == 9).all()
    uvu.orthogonalize(view, view)
    assert torch.equal(view, want)
    view.fill_(7)
    assert (big == 7).all()
    single = nan_like((m, n), kind)
    uvu.orthogonalize(g[1], single)
    assert torch.equal(single, want[1])


@pytest.mark.parametrize("size", [1e-30, 1e-19, 1.0, 1e18, 1e30])
@pytest.mark.parametrize("shape", [(30, 50), (300, 200)], ids=str)
def test_orthogonalize_any_size(shape, size):
    """The norm of values whose squares leave fp32, eps = 0."""
    rng = np.random.default_rng(7)
    g, gr = rounded(rng.standard_normal(shape) * size, "f32")
    out = nan_like(shape)
    uvu.orthogonalize(g, out, eps=0.0)
    check(values(out), layer.newton_schulz(gr, 5, MUON, 0.0)[-1], False)


@pytest.mark.parametrize("shape", [(30, 50), (300, 200)], ids=str)
def test_orthogonalize_matrices_apart(shape):
    rng = np.random.default_rng(8)
    g, _ = rounded(rng.standard_normal((5, *shape)), "f32")
    clean, out = nan_like(g.shape), nan_like(g.shape)
    uvu.orthogonalize(g, clean)
    g[1, 3, 4], g[2], g[4, 0, 0] = float("nan"), 0, float("inf")
    uvu.orthogonalize(g, out)
    assert torch.equal(out[[0, 3]], clean[[0, 3]]) and (out[2] == 0).all()
    assert not torch.isfinite(out[1]).any() and torch.isnan(out[4]).any()


# --------------------------------------------------------------------------------- as they are used

def test_streams_and_graphs():
    """Two captured graphs and eager calls on a side stream, with workspaces of their own, give the results of plain calls."""
    rng = np.random.default_rng(9)
    ix = dev(rng.integers(-1, 40, size=3000).astype(np.int32))
    dout, x, dy = (torch.randn(3000, 64, device="cuda") for _ in range(3))
    gamma = torch.rand(64, device="cuda")
    gs = [dev(rng.standard_normal(s).astype(np.float32)) for s in ((3, 96, 160), (300, 200))]

    def new():
        return [nan_like((40, 64)), nan_like((3000, 64)), nan_like((3000,)), nan_like((3000, 64)), nan_like((64,)),
                *(nan_like(tuple(g.shape)) for g in gs)]

    def step(o, **kw):
        uvu.embed_bwd(ix, dout, o[0], **kw)
        uvu.rms_norm_fwd(x, gamma, o[1], o[2], **kw)
        uvu.rms_norm_bwd(dy, x, gamma, o[2], o[3], o[4], **kw)
        for g, out in zip(gs, o[5:]):
            uvu.orthogonalize(g, out, **kw)

    want = new()
    step(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = new()
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
    assert uvu.orthogonalize_device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
def test_autograd(kind):
    """The autograd forms against the formulas in fp64 autograd, with each gradient alone and the stream's cotangent missing."""
    rng = np.random.default_rng(10)
    index = np.array([3, 0, -1, 3, 9, 2, 2, 2], np.int32)
    table, tr = rounded(rng.standard_normal((5, 16)), kind)
    gamma, gr = rounded(1 + 0.2 * rng.standard_normal(16), "f32")
    cy, cyr = rounded(rng.standard_normal((8, 16, 4)), kind)
    ch, chr_ = rounded(rng.standard_normal((8, 16, 4)), kind)
    table.requires_grad_(True)
    gamma.requires_grad_(True)
    x = autograd.embedding(dev(index), table, scale=0.5, inner=4)
    res, rr = rounded(rng.standard_normal((8, 16, 4)), kind)
    res.requires_grad_(True)
    y, h = autograd.rms_norm(x, gamma, residual=res)
    got = torch.autograd.grad([y, h], [table, gamma, res], [cy, ch], retain_graph=True)
    hr = values(h.detach())
    rdx, rdg = layer.rms_norm_vjp(hr, gr, 1e-5, cyr, chr_)
    near(got[2], rdx, kind, "dres")
    near(got[1], rdg, "f32", "dgamma")
    ref, size, count = layer.embed_vjp(index, values(got[2]), 5, 0.5, 0)
    within(got[0], ref, embed_bound(ref, kind) + np.maximum(count, 1)[:, None] * 2.0 ** -24 * size, "dtable")
    (only,) = torch.autograd.grad(y, [res], [cy], retain_graph=True)
    near(only, layer.rms_norm_vjp(hr, gr, 1e-5, cyr)[0], kind)
    (only, dg) = torch.autograd.grad(h, [res, gamma], [ch], retain_graph=True)
    assert torch.equal(only, ch) and not dg.any()
    # a broadcast residual and a transposed cotangent
    row = torch.randn(1, 16, 4, device="cuda").to(TYPES[kind]).requires_grad_(True)
    y1, h1 = autograd.rms_norm(x.detach(), gamma, residual=row.expand(8, -1, -1))
    (drow,) = torch.autograd.grad(y1, [row], [cy.transpose(0, 1).contiguous().transpose(0, 1)])
    full = layer.rms_norm_vjp(values(h1.detach()), gr, 1e-5, cyr)[0]
    within(drow, full.sum(0, keepdims=True), 9 * UNIT[kind] * np.abs(full).sum(0, keepdims=True) + 1e-4 * (1 + np.abs(full).sum(0, keepdims=True)))
    plain = autograd.embedding(dev(index), table)
    assert plain.shape == (8, 16) and not plain[2].any() and not plain[4].any()
    alone = autograd.rms_norm(plain, gamma)
    (dt,) = torch.autograd.grad(alone.float().square().sum(), [table])
    assert torch.isfinite(dt).all()


def test_muon_step():
    """Two steps of the optimiser on matrices of three sizes, against the same in fp64."""
    rng = np.random.default_rng(11)
    shapes = [(4, 40, 24), (40, 24), (30, 70), (200, 150)]
    start, grads = [rng.standard_normal(s) for s in shapes], [[rng.standard_normal(s) for s in shapes] for _ in range(2)]
    params = [dev(a.astype(np.float32)).requires_grad_(True) for a in start]
    opt = optim.Muon(params, lr=0.1, momentum=0.9, weight_decay=0.01)
    ref = [p.detach().double().cpu().numpy() for p in params]
    buf = [np.zeros(s) for s in shapes]
    for step in grads:
        for p, g in zip(params, step):
            p.grad = dev(g.astype(np.float32))
        opt.step()
        for i, g in enumerate(step):
            g = g.astype(np.float32).astype(np.float64)
            buf[i] = 0.9 * buf[i] + 0.1 * g
            u = (0.1 * g + 0.9 * buf[i]).reshape(-1, *shapes[i][-2:])
            o = np.stack([layer.newton_schulz(a, 5, MUON, 1e-7)[-1] for a in u]).reshape(shapes[i])
            ref[i] = ref[i] * (1 - 0.1 * 0.01) - 0.1 * max(1, shapes[i][-2] / shapes[i][-1]) ** 0.5 * o
    for p, r in zip(params, ref):
        check(values(p.detach()), r, False)


def test_example_runs():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "species_model.py")
    spec = importlib.util.spec_from_file_location("species_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, params = example.train(n_molecules=8, steps=3)
    assert np.isfinite(losses).all() and all(torch.isfinite(p).all() and torch.isfinite(p.grad).all() and p.grad.any() for p in params)

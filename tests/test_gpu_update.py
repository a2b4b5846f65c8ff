"""GPU parity of the node-update operators (uvu_group_norm_*, uvu_attn_*, uvu_dropout_*) with the fp64
oracle (oracle.update), their edge cases, their refusals, and one training block that chains them to
a convolution.

Tolerances, from the arithmetic.  fp32 results: gpu_util.check (relative Frobenius 1e-5, elements
1e-4 (1 + |ref|)).  16-bit results: one rounding of the result to p bits is at most u |ref| with
u = 2^-p; attention also rounds P and dS to p bits before the products and takes delta from the
rounded output, whose first-order elementwise effect the oracle returns; the remainder, fp32
arithmetic and the 16-bit types' smallest magnitudes, is below 1e-4 (1 + |ref|)."""
import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import uvu
from gpu_util import check
from oracle import update

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def rounded(a, kind):
    """A device tensor of the type, and the fp64 values that it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TYPES[kind])
    return t.cuda(), t.double().numpy()


def near(got, ref, kind, extra=0.0, what=""):
    got = got.double().cpu().numpy()
    if kind == "f32":
        return check(got, ref, False, what)
    assert got.shape == ref.shape, what
    bound = UNIT[kind] * np.abs(ref) + extra + 1e-4 * (1 + np.abs(ref))
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), f"{what}: {(over > 0).sum()} elements beyond their bound, by up to {over.max():.3e}"


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def nan_like(shape, kind="f32"):
    return torch.full(shape, float("nan"), dtype=TYPES[kind], device="cuda")


# ------------------------------------------------------------------------------------ group norm

NORMS = [  # lengths, channels, groups
    ([1], 1, 1), ([100], 16, 4), ([3, 0, 1, 17, 64], 24, 3), ([0, 0, 5], 40, 40), ([33, 2], 7, 7), ([33, 2], 7, 1),
    ([129, 300, 1], 128, 8), ([1000], 512, 32), ([41] * 30, 64, 2), ([2500, 7], 320, 8), ([20, 3], 2056, 1), ([9], 8192, 4),
    ([5000], 96, 3), ([70000, 3], 128, 16)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", NORMS, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}-{c[2]}")
@pytest.mark.parametrize("act", ["silu", "none"])
def test_group_norm(case, kind, act):
    lengths, c, groups = case
    rng = np.random.default_rng(sum(lengths) + c)
    off, n, b = offsets(lengths), sum(lengths), len(lengths)
    x, xr = rounded(rng.standard_normal((n, c)) * 1.5 + 0.4, kind)
    dy, dyr = rounded(rng.standard_normal((n, c)), kind)
    gamma, gr = rounded(1 + 0.2 * rng.standard_normal(c), "f32")
    beta, br = rounded(0.2 * rng.standard_normal(c), "f32")
    code = uvu.UVU_ACT_SILU if act == "silu" else uvu.UVU_ACT_NONE
    mean, rstd = nan_like((b, groups)), nan_like((b, groups))
    y, dx, dg, db = nan_like((n, c), kind), nan_like((n, c), kind), nan_like((c,)), nan_like((c,))
    longest = max(lengths)
    uvu.group_norm_fwd(x, gamma, beta, i32(off), groups, y, mean, rstd, act=code, max_rows=longest)
    uvu.group_norm_bwd(dy, x, gamma, beta, i32(off), groups, mean, rstd, dx, dg, db, act=code, max_rows=longest)
    ry, rm, rr = update.group_norm(xr, gr, br, off, groups, act == "silu", 1e-5)
    rdx, rdg, rdb = update.group_norm_vjp(xr, gr, br, off, groups, act == "silu", 1e-5, dyr)
    for name, got, ref, k in (("y", y, ry, kind), ("mean", mean, rm, "f32"), ("rstd", rstd, rr, "f32"), ("dx", dx, rdx, kind),
                              ("dgamma", dg, rdg, "f32"), ("dbeta", db, rdb, "f32")):
        near(got, ref, k, what=name)


@pytest.mark.parametrize("kind", list(TYPES))
def test_group_norm_wrong_max_rows_and_views(kind):
    """A max_rows below the longest graph, and tensors that begin off a 16-byte boundary, change nothing but time."""
    rng = np.random.default_rng(8)
    off, n, c, groups = offsets([700, 0, 3, 41]), 744, 64, 4
    flat, _ = rounded(rng.standard_normal(n * c + 1), kind)
    x = flat[1:].view(n, c)
    xr = x.double().cpu().numpy()
    dy, dyr = rounded(rng.standard_normal((n, c)), kind)
    gamma, beta = nan_like((c,)).fill_(1.25), nan_like((c,)).fill_(-0.5)
    for most in (1, 50, None):
        mean, rstd = nan_like((4, groups)), nan_like((4, groups))
        y = nan_like((n * c + 1,), kind)[1:].view(n, c)
        dx, dg, db = nan_like((n, c), kind), nan_like((c,)), nan_like((c,))
        uvu.group_norm_fwd(x, gamma, beta, i32(off), groups, y, mean, rstd, max_rows=most)
        uvu.group_norm_bwd(dy, x, gamma, beta, i32(off), groups, mean, rstd, dx, dg, db, max_rows=most)
        g, b = np.full(c, 1.25), np.full(c, -0.5)
        near(y, update.group_norm(xr, g, b, off, groups, True, 1e-5)[0], kind, what="y")
        for got, ref, k in zip((dx, dg, db), update.group_norm_vjp(xr, g, b, off, groups, True, 1e-5, dyr), (kind, "f32", "f32")):
            near(got, ref, k)


@pytest.mark.parametrize("lengths", [[400], [60000]], ids=["short", "long"])
def test_group_norm_far_from_zero(lengths):
    """Values of 1000 +- 1: a variance formed as E[x^2] - mean^2 would be lost."""
    rng = np.random.default_rng(9)
    n = sum(lengths)
    x, xr = rounded(rng.standard_normal((n, 32)) + 1000, "f32")
    one, zero = torch.ones(32, device="cuda"), torch.zeros(32, device="cuda")
    y, mean, rstd = nan_like((n, 32)), nan_like((1, 4)), nan_like((1, 4))
    uvu.group_norm_fwd(x, one, zero, i32(offsets(lengths)), 4, y, mean, rstd, act=uvu.UVU_ACT_NONE, max_rows=n)
    ref, _, rr = update.group_norm(xr, np.ones(32), np.zeros(32), offsets(lengths), 4, False, 1e-5)
    # the mean of values near 1000 is known to 1000 * 2^-24 = 6e-5 in fp32, which y shows
    assert np.abs(y.double().cpu().numpy() - ref).max() <= 4e-4
    np.testing.assert_allclose(rstd.cpu().numpy(), rr, rtol=1e-5)


def test_group_norm_repeats_bit_for_bit():
    rng = np.random.default_rng(10)
    off = i32(offsets([900, 1, 350, 2000]))
    x, _ = rounded(rng.standard_normal((3251, 256)), "bf16")
    gamma, beta = torch.rand(256, device="cuda"), torch.rand(256, device="cuda")
    runs = []
    for _ in range(2):
        mean, rstd, y = nan_like((4, 8)), nan_like((4, 8)), nan_like(x.shape, "bf16")
        dx, dg, db = nan_like(x.shape, "bf16"), nan_like((256,)), nan_like((256,))
        uvu.group_norm_fwd(x, gamma, beta, off, 8, y, mean, rstd, max_rows=2000)
        uvu.group_norm_bwd(y, x, gamma, beta, off, 8, mean, rstd, dx, dg, db, max_rows=2000)
        runs.append((y, mean, rstd, dx, dg, db))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_group_norm_of_no_rows():
    mean, rstd = nan_like((2, 2)), nan_like((2, 2))
    x, one = torch.empty(0, 8, device="cuda"), torch.ones(8, device="cuda")
    dg, db = nan_like((8,)), nan_like((8,))
    uvu.group_norm_fwd(x, one, one, i32([0, 0, 0]), 2, x, mean, rstd, eps=0.25)
    uvu.group_norm_bwd(x, x, one, one, i32([0, 0, 0]), 2, mean, rstd, x, dg, db)
    assert (mean == 0).all() and (rstd == 2).all() and (dg == 0).all() and (db == 0).all()


# --------------------------------------------------------------------------------------- dropout

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", [(1, 1), (7, 1), (8, 1), (4099, 1), (131072, 1), (1000, 4), (333, 9), (50, 3), (3, 1000)],
                         ids=lambda c: f"{c[0]}x{c[1]}")
@pytest.mark.parametrize("view", [0, 1])
def test_dropout(case, kind, view):
    draws, inner = case
    rng = np.random.default_rng(draws + inner)
    n = draws * inner
    x, xr = rounded(rng.standard_normal(n + view), kind)
    res, rr = rounded(rng.standard_normal(n + view), kind)
    x, res, xr, rr = x[view:], res[view:], xr[view:], rr[view:]
    for p, seed, off in ((0.1, 5, 0), (0.5, 2 ** 63 + 11, 2 ** 40 + 3), (0.9, 77, 2 ** 32 - 2)):
        keep, scale = update.keep_mask(draws, p, seed, off)
        m = np.repeat(keep, inner) * scale
        y = nan_like((n + view,), kind)[view:]
        uvu.dropout_fwd(x, p, seed, y, offset=off, inner=inner, residual=res)
        near(y, rr + xr * m, kind, what="y")
        uvu.dropout_fwd(x, p, seed, y, offset=off, inner=inner)
        near(y, xr * m, kind, what="y without residual")
        assert np.array_equal(y.cpu().float().numpy() != 0, (np.repeat(keep, inner)) & (xr != 0))
        uvu.dropout_bwd(res, p, seed, y, offset=off, inner=inner)
        near(y, rr * m, kind, what="dx")


@pytest.mark.parametrize("kind", list(TYPES))
def test_dropout_limits(kind):
    """p = 0 keeps everything unscaled, p = 1 nothing; dropped values are not used; in place works."""
    x, xr = rounded(np.random.default_rng(1).standard_normal(1001), kind)
    y = nan_like((1001,), kind)
    uvu.dropout_fwd(x, 0.0, 3, y)
    assert torch.equal(x, y)
    bad = x.clone()
    bad[::2], bad[1::2] = float("nan"), float("inf")
    uvu.dropout_fwd(bad, 1.0, 3, y, residual=x)
    assert torch.equal(x, y)
    keep, scale = update.keep_mask(1001, 0.5, 4, 0)
    bad = x.clone()
    bad[torch.from_numpy(~keep).cuda()] = float("nan")
    uvu.dropout_fwd(bad, 0.5, 4, bad)
    near(bad, xr * keep * scale, kind)
    e = torch.empty(0, device="cuda")
    uvu.dropout_fwd(e, 0.5, 4, e)


# ------------------------------------------------------------------------------------- attention

ATTN = [  # q lengths, k lengths, q heads, kv heads, head dim, kept share (None: no mask)
    ([1], [1], 1, 1, 1, None), ([1], [1], 2, 1, 16, 0.0), ([3, 0, 5], [0, 7, 9], 2, 2, 8, None),
    ([1] * 5, [1, 130, 700, 0, 64], 8, 2, 64, 0.7), ([1, 1], [3000, 4001], 4, 4, 128, None), ([1, 1], [2500, 1], 28, 4, 32, 0.9),
    ([130, 1, 257], [300, 129, 5], 4, 4, 128, 0.9), ([64, 128], [64, 128], 3, 1, 64, None), ([200, 77], [500, 33], 6, 2, 40, 0.5),
    ([61], [1000], 7, 7, 24, None), ([513], [2], 2, 1, 96, None), ([300], [300], 1, 1, 80, 0.02), ([20], [45], 2, 2, 33, 0.8),
    ([1, 2, 3, 4], [5, 6, 7, 8], 5, 1, 7, None), ([700], [640], 2, 2, 112, 0.6)]


def attn_problem(case, kind, seed=0):
    ql, kl, hq, hk, d, share = case
    rng = np.random.default_rng(sum(ql) * 7 + sum(kl) + d + seed)
    nq, nk = sum(ql), sum(kl)
    P = {n: rounded(rng.standard_normal(s), kind) for n, s in (("q", (nq, hq, d)), ("k", (nk, hk, d)), ("v", (nk, hk, d)),
                                                              ("do", (nq, hq, d)))}
    keep = None if share is None else (rng.random(nk) < share).astype(np.uint8)
    at = uvu.Attention(hq, hk, d, i32(offsets(ql)), i32(offsets(kl)), max(ql), max(kl))
    return P, keep, at, offsets(ql), offsets(kl)


def attn_run(at, q, k, v, do, keep, kind):
    out, lse = nan_like(q.shape, kind), nan_like(q.shape[:2])
    g = [nan_like(t.shape, kind) for t in (q, k, v)]
    kd = None if keep is None else torch.from_numpy(keep).cuda()
    at.fwd(q, k, v, out, lse, keep=kd)
    at.bwd(q, k, v, out, lse, do, *g, keep=kd)
    return [out, lse] + g


def attn_compare(got, P, keep, at, qo, ko, kind):
    q, k, v, do = (P[n][1] for n in ("q", "k", "v", "do"))
    out, lse, mag = update.attention(q, k, v, qo, ko, at.scale, keep)
    grads, err = update.attention_vjp(q, k, v, qo, ko, at.scale, do, keep, UNIT[kind])
    near(got[0], out, kind, 2 * UNIT[kind] * mag, "out")
    a, b = got[1].double().cpu().numpy(), lse
    assert np.array_equal(np.isneginf(a), np.isneginf(b)), "lse of empty rows"
    near(torch.from_numpy(np.where(np.isneginf(a), 0, a)), np.where(np.isneginf(b), 0, b), "f32", what="lse")
    for name, x, ref, e in zip(("dq", "dk", "dv"), got[2:], grads, err):
        near(x, ref, kind, e, name)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"q{max(c[0])}-k{max(c[1])}-h{c[2]}.{c[3]}-d{c[4]}-{c[5]}")
def test_attention(case, kind):
    P, keep, at, qo, ko = attn_problem(case, kind)
    got = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, kind)
    attn_compare(got, P, keep, at, qo, ko, kind)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", [64, 20])
def test_attention_strided_views(kind, d):
    """k and v as halves of one projection, q and out as slices of wider rows, and a base off the 16-byte boundary."""
    case = ([70, 5], [90, 133], 4, 2, d, 0.8)
    P, keep, at, qo, ko = attn_problem(case, kind)
    kv = nan_like((sum(case[1]), 2, 2, d), kind)
    kv[:, 0], kv[:, 1] = P["k"][0], P["v"][0]
    wide = nan_like((75, 4, d + 3), kind)
    q = wide[:, :, 1:d + 1]
    q.copy_(P["q"][0])
    out, do = nan_like((75, 4, d + 3), kind)[:, :, 3:], nan_like((75, 4, d + 3), kind)[:, :, 3:]
    do.copy_(P["do"][0])
    lse, kd = nan_like((75, 4)), torch.from_numpy(keep).cuda()
    g = [nan_like(P[n][0].shape, kind) for n in ("q", "k", "v")]
    at.fwd(q, kv[:, 0], kv[:, 1], out, lse, keep=kd)
    at.bwd(q, kv[:, 0], kv[:, 1], out, lse, do, *g, keep=kd)
    attn_compare([out, lse] + g, P, keep, at, qo, ko, kind)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows", [1, 150])
def test_attention_ignores_masked_values(kind, rows):
    """NaN and infinities in masked states, and in the states of the graph behind, reach no result."""
    case = ([rows, rows], [200, 300], 2, 1, 64, 0.7)
    P, keep, at, qo, ko = attn_problem(case, kind)
    keep[150:260] = 0  # the end of one graph and the beginning of the next
    k, v = P["k"][0].clone(), P["v"][0].clone()
    off = torch.from_numpy(keep == 0).cuda()
    k[off], v[off] = float("nan"), float("inf")
    k[155:160], v[157] = float("-inf"), float("nan")
    got = attn_run(at, P["q"][0], k, v, P["do"][0], keep, kind)
    attn_compare(got, P, keep, at, qo, ko, kind)
    assert (got[3][off] == 0).all() and (got[4][off] == 0).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_attention_does_not_leak_between_graphs(kind):
    """A graph full of NaN changes nothing in its neighbours."""
    case = ([60, 90, 33], [100, 50, 70], 2, 2, 32, None)
    P, keep, at, qo, ko = attn_problem(case, kind)
    t = {n: P[n][0].clone() for n in P}
    for n, o in (("q", qo), ("k", ko), ("v", ko), ("do", qo)):
        t[n][o[1]:o[2]] = float("nan")
    got = attn_run(at, t["q"], t["k"], t["v"], t["do"], keep, kind)
    want = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, kind)
    for a, b, o in zip(got, want, (qo, qo, qo, ko, ko)):
        assert torch.equal(a[:o[1]], b[:o[1]]) and torch.equal(a[o[2]:], b[o[2]:])
        assert torch.isnan(a[o[1]:o[2]]).all()


@pytest.mark.parametrize("kind", list(TYPES))
def test_attention_large_scores(kind):
    """Scores in the thousands, rising along the states: the running maximum moves in every tile."""
    d, nk, nq = 32, 900, 140
    rng = np.random.default_rng(2)
    ramp = np.linspace(-1, 1, nk)[:, None, None] * np.ones((nk, 1, d)) * 4
    P = {n: rounded(a, kind) for n, a in (("q", 2 + rng.random((nq, 1, d))), ("k", ramp + 0.01 * rng.standard_normal((nk, 1, d))),
                                          ("v", rng.standard_normal((nk, 1, d))), ("do", rng.standard_normal((nq, 1, d))))}
    at = uvu.Attention(1, 1, d, i32([0, nq]), i32([0, nk]), scale=8.0)
    got = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), None, kind)
    q, k, v = (P[n][1] for n in ("q", "k", "v"))
    out, lse, mag = update.attention(q, k, v, [0, nq], [0, nk], 8.0)
    # scores reach 2600: fp32 holds them to 2^-13 (about 20 roundings of 2^-24 relative), and P to that much more
    near(got[0], out, "bf16" if kind == "f32" else kind, 2 * UNIT[kind] * mag + 2e-3 * mag, "out")
    np.testing.assert_allclose(got[1].cpu().numpy(), lse, rtol=2e-6)


@pytest.mark.parametrize("kind", list(TYPES))
def test_attention_gradient_against_differences(kind):
    """A directional difference of the kernel's own forward against its gradient (fp32), and the 16-bit gradients
    against the fp32 ones on the same values."""
    case = ([40, 9], [70, 30], 4, 2, 16, 0.9)
    P, keep, at, qo, ko = attn_problem(case, kind)
    exactly = {n: P[n][0].float() for n in P}
    g32 = attn_run(at, *(exactly[n] for n in ("q", "k", "v", "do")), keep, "f32")[2:]
    if kind != "f32":
        _, err = update.attention_vjp(*(P[n][1] for n in ("q", "k", "v")), qo, ko, at.scale, P["do"][1], keep, UNIT[kind])
        got = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, kind)[2:]
        for a, b, e in zip(got, g32, err):
            near(a, b.double().cpu().numpy(), kind, e)
        return
    rng = np.random.default_rng(12)
    kd, h = torch.from_numpy(keep).cuda(), 2.0 ** -6
    for i, n in enumerate(("q", "k", "v")):
        d = torch.from_numpy(rng.standard_normal(P[n][0].shape).astype(np.float32)).cuda()
        d = d / d.norm()
        val = []
        for s in (h, -h, 2 * h, -2 * h):
            t = dict(exactly)
            t[n] = t[n] + s * d
            out, lse = nan_like(t["q"].shape), nan_like(t["q"].shape[:2])
            at.fwd(t["q"], t["k"], t["v"], out, lse, keep=kd)
            val.append((out.double() * exactly["do"].double()).sum().item())
        want = (8 * (val[0] - val[1]) - (val[2] - val[3])) / (12 * h)
        have = (g32[i].double() * d.double()).sum().item()
        # fourth-order differences: h^4 = 6e-8, and outputs of size 1 rounded at 2^-24 over 4 h and 800 values: 3e-5
        assert abs(want - have) <= 2e-4 * (1 + abs(want)), (n, want, have)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", [32, 64, 128])
def test_attention_long_walks(kind, d):
    """Many tiles in both directions, where the roles of a block run ahead of one another: no wait gives up, and rows and
    states picked at random agree with the oracle."""
    nq, nk, hq, hk = 3100, 2900, 4, 2
    P, keep, at, qo, ko = attn_problem(([nq, nq], [nk, nk], hq, hk, d, 0.9), kind)
    uvu.Attention.device_status()
    got = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, kind)
    torch.cuda.synchronize()
    assert uvu.Attention.device_status() == 0
    q, k, v, do = (P[n][1] for n in ("q", "k", "v", "do"))
    rows = np.sort(np.random.default_rng(3).choice(nq, 40, replace=False))
    out, lse, mag = update.attention(q[rows], k[:nk], v[:nk], [0, 40], [0, nk], at.scale, keep[:nk])
    grads, err = update.attention_vjp(q[rows], k[:nk], v[:nk], [0, 40], [0, nk], at.scale, do[rows], keep[:nk], UNIT[kind])
    at_rows = torch.from_numpy(rows).cuda()
    near(got[0][at_rows], out, kind, 2 * UNIT[kind] * mag, "out")
    near(got[1][at_rows], lse, "f32", what="lse")
    near(got[2][at_rows], grads[0], kind, err[0], "dq")
    # dk and dv of the second graph, one kv head, from all of its rows
    second = slice(nq, 2 * nq)
    grads, err = update.attention_vjp(q[second, :2], k[nk:, :1], v[nk:, :1], [0, nq], [0, nk], at.scale, do[second, :2], keep[nk:],
                                      UNIT[kind])
    for g, ref, e, name in ((got[3], grads[1], err[1], "dk"), (got[4], grads[2], err[2], "dv")):
        near(g[nk:, :1], ref, kind, e, name)


def test_attention_repeats_bit_for_bit():
    for kind in TYPES:
        P, keep, at, qo, ko = attn_problem(([300, 4], [700, 900], 8, 2, 64, 0.9), kind)
        a, b = (attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, kind) for _ in range(2))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attention_wrong_bounds_on_lengths():
    """max_q and max_k below the longest graph change nothing but time."""
    case = ([90, 200], [400, 17], 4, 2, 64, 0.9)
    for kind in ("f32", "bf16"):
        P, keep, at, qo, ko = attn_problem(case, kind)
        at.max_q, at.max_k = 1, 1
        got = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, kind)
        attn_compare(got, P, keep, at, qo, ko, kind)


def test_attention_offsets_beyond_32_bits():
    """Rows whose elements lie past 2^32 (a view with a long row stride)."""
    d, nk = 64, 5
    store = torch.zeros(nk, 2 ** 30, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(13)
    P = {n: rounded(rng.standard_normal((m, 1, d)), "bf16") for n, m in (("q", 3), ("k", nk), ("v", nk), ("do", 3))}
    k, v = store[:, :d].unflatten(1, (1, d)), store[:, d:2 * d].unflatten(1, (1, d))
    k.copy_(P["k"][0]), v.copy_(P["v"][0])
    at = uvu.Attention(1, 1, d, i32([0, 3]), i32([0, nk]))
    got = attn_run(at, P["q"][0], k, v, P["do"][0], None, "bf16")
    attn_compare(got, P, None, at, [0, 3], [0, nk], "bf16")


def test_operators_on_another_stream():
    """Work on a side stream, ordered by events alone."""
    case = ([100, 30], [200, 90], 4, 2, 64, 0.9)
    P, keep, at, qo, ko = attn_problem(case, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = attn_run(at, *(P[n][0] for n in ("q", "k", "v", "do")), keep, "bf16")
    torch.cuda.current_stream().wait_stream(side)
    attn_compare(got, P, keep, at, qo, ko, "bf16")


def test_operators_in_a_graph():
    """The calls are launches alone: a captured sequence replays on new values."""
    P, keep, at, qo, ko = attn_problem(([50, 31], [64, 200], 4, 4, 32, 0.9), "bf16")
    q, k, v, do = (P[n][0].clone() for n in ("q", "k", "v", "do"))
    kd = torch.from_numpy(keep).cuda()
    out, lse = nan_like(q.shape, "bf16"), nan_like(q.shape[:2])
    g = [nan_like(t.shape, "bf16") for t in (q, k, v)]
    ws = torch.empty(max(16, *at.workspace_bytes(q, k)), dtype=torch.uint8, device="cuda")
    x, y = q.reshape(81, -1), nan_like((81, 128), "bf16")
    gamma = torch.ones(128, device="cuda")
    mean, rstd, off = nan_like((2, 4)), nan_like((2, 4)), i32(qo)
    nws = torch.empty(max(16, *uvu.group_norm_workspace_bytes(x, 2, 4)), dtype=torch.uint8, device="cuda")

    def calls():
        at.fwd(q, k, v, out, lse, keep=kd, workspace=ws)
        at.bwd(q, k, v, out, lse, do, *g, keep=kd, workspace=ws)
        uvu.group_norm_fwd(x, gamma, gamma, off, 4, y, mean, rstd, workspace=nws)
        uvu.dropout_fwd(y, 0.25, 7, y, residual=x)

    calls()
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        calls()
    P2 = attn_problem(([50, 31], [64, 200], 4, 4, 32, 0.9), "bf16", seed=1)[0]
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (do, "do")):
        t.copy_(P2[n][0])
    cg.replay()
    torch.cuda.synchronize()
    attn_compare([out, lse] + g, P2, keep, at, qo, ko, "bf16")


# -------------------------------------------------------------------------------------- refusals

def refuses(status, f, *args, **kw):
    with pytest.raises(uvu.UVUError) as e:
        f(*args, **kw)
    assert e.value.status == status, e.value


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    w, off = torch.ones(8, device="cuda"), i32([0, 4])
    m = torch.zeros(1, 3, device="cuda")
    refuses(1, uvu.group_norm_fwd, x, w, w, off, 3, x.clone(), m, m.clone())  # 8 channels in 3 groups
    m = torch.zeros(1, 2, device="cuda")
    for bad in (-1.0, float("nan"), float("inf")):
        refuses(1, uvu.group_norm_fwd, x, w, w, off, 2, x.clone(), m, m.clone(), eps=bad)
    refuses(1, uvu.group_norm_fwd, x, w, w, off, 2, x.clone(), m, m.clone(), act=7)
    refuses(2, uvu.dropout_fwd, x.double(), 0.1, 1, x.double())
    for p in (-0.1, 1.5, float("nan")):
        refuses(1, uvu.dropout_fwd, x, p, 1, x.clone())
    with pytest.raises(ValueError):
        uvu.dropout_fwd(x, 0.1, 1, x.clone(), inner=5)
    with pytest.raises(ValueError):
        uvu.dropout_fwd(x.t(), 0.1, 1, x.clone())
    with pytest.raises(TypeError):
        uvu.dropout_fwd(x, 0.1, 1, x.half())
    with pytest.raises(TypeError):
        uvu.dropout_fwd(x.int(), 0.1, 1, x.int())
    with pytest.raises(ValueError):
        uvu.group_norm_fwd(x, w.half(), w, off, 2, x.clone(), m, m.clone())
    with pytest.raises(ValueError):
        uvu.group_norm_fwd(x, w, w, off.long(), 2, x.clone(), m, m.clone())
    q = torch.zeros(4, 2, 130, device="cuda")
    lse = torch.zeros(4, 2, device="cuda")
    refuses(2, uvu.Attention(2, 2, 130, off, off).fwd, q, q, q, q.clone(), lse)
    q = torch.zeros(4, 3, 8, device="cuda")
    refuses(1, uvu.Attention(3, 2, 8, off, off).fwd, q, q[:, :2], q[:, :2], q.clone(), torch.zeros(4, 3, device="cuda"))
    q = torch.zeros(4, 2, 8, device="cuda")
    refuses(1, uvu.Attention(2, 2, 8, off, off, scale=float("inf")).fwd, q, q, q, q.clone(), lse)
    refuses(2, uvu.Attention(2, 2, 8, off, off).fwd, q.double(), q.double(), q.double(), q.double(), lse)
    at = uvu.Attention(2, 2, 8, off, off)
    refuses(1, at.bwd, q, q, q, q.clone(), lse, q, dk=q.clone())  # dk without dv
    refuses(1, at.bwd, q, q, q, q.clone(), lse, q, dq=q.clone(), workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    for wrong in (q[:, :1], q.half(), q.transpose(0, 2)):
        with pytest.raises((ValueError, TypeError)):
            at.fwd(q, wrong, q, q.clone(), lse)
    with pytest.raises(ValueError):
        at.fwd(q, q, q, q.clone(), lse, keep=torch.ones(3, dtype=torch.uint8, device="cuda"))

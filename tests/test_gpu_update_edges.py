"""Calls of the node-update operators at the edges of their contracts: unusual strides, empty batches, rows whose mask leaves
nothing, small cotangents, and the kernels that only large batches choose."""
import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import autograd, uvu
from gpu_util import check
from oracle import update
from update_limits import TYPES, gradient_limit, output_limit, relative, unit, values

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows, heads", [(5, 1), (1, 4)])
def test_gradient_of_a_heads_first_consumer(rows, heads, kind):
    """With one head, or one row, the cotangent of the transposed output counts as contiguous with strides of its own."""
    at = uvu.Attention(heads, 1, 8, i32([0, rows]), i32([0, 20]))
    q, k, v = (rand(i, n, h, 8, dtype=TYPES[kind]).requires_grad_(True) for i, (n, h) in enumerate(((rows, heads), (20, 1), (20, 1))))
    g = rand(3, heads, rows, 8, dtype=TYPES[kind])
    got = torch.autograd.grad(autograd.cross_attention(q, k, v, at).transpose(0, 1), (q, k, v), g)
    want = torch.autograd.grad(autograd.cross_attention(q, k, v, at), (q, k, v), torch.empty_like(q).copy_(g.transpose(0, 1)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------- small and large 16-bit cotangents

def gradients(q, k, v, do, at, keep=None):
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    at.fwd(q, k, v, out, lse, keep=keep)
    g = [torch.empty_like(t) for t in (q, k, v)]
    at.bwd(q, k, v, out, lse, do, *g, keep=keep)
    return g


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("states", [4096, 16384])
def test_gradients_of_small_cotangents(states, size, kind):
    """P (dP - delta) of many states and a small cotangent lies far below f16's smallest normal number."""
    dtype, nq, off = TYPES[kind], 40, ([0, 40], [0, states])
    at = uvu.Attention(2, 1, 64, i32(off[0]), i32(off[1]))
    q, k, v = rand(1, nq, 2, 64, dtype=dtype), rand(2, states, 1, 64, dtype=dtype), rand(3, states, 1, 64, dtype=dtype)
    do = (rand(4, nq, 2, 64) * size).to(dtype)
    ref, _ = update.attention_vjp(*map(values, (q, k, v)), *off, at.scale, values(do))
    for name, got, r in zip(("dq", "dk", "dv"), gradients(q, k, v, do, at), ref):
        assert relative(got, r) <= gradient_limit(r, dtype), (name, relative(got, r), gradient_limit(r, dtype))


def test_gradients_of_large_cotangents():
    """dP beyond f16's range, gradients within it."""
    off = ([0, 6, 30], [0, 2, 33])
    at = uvu.Attention(1, 1, 64, i32(off[0]), i32(off[1]))
    q, k, v = (rand(i, n, 1, 64, dtype=torch.float16) for i, n in ((1, 30), (2, 33), (3, 33)))
    do = (rand(4, 30, 1, 64) * 1e4).to(torch.float16)
    k, v = k * 0.25, v * 4
    ref, _ = update.attention_vjp(*map(values, (q, k, v)), *off, at.scale, values(do))
    assert np.abs(values(do)[:6, 0] @ values(v)[:2, 0].T).max() > 2 * 65504 and max(np.abs(r).max() for r in ref[:2]) < 65504
    for name, got, r in list(zip(("dq", "dk"), gradients(q, k, v, do, at), ref)):
        assert relative(got, r) <= gradient_limit(r, torch.float16), (name, relative(got, r), gradient_limit(r, torch.float16))


def test_gradients_of_cotangents_of_many_sizes():
    """Graphs, heads and rows whose cotangents differ by orders of magnitude: each graph's and kv head's dk and dv, and each row's dq,
    as if alone.  Masked states hold infinities, which no scale may follow."""
    off, dtype = ([0, 70, 70, 200], [0, 3000, 3000, 5100]), torch.float16
    at = uvu.Attention(4, 2, 64, i32(off[0]), i32(off[1]), 130, 3000)
    q, k, v = rand(1, 200, 4, 64, dtype=dtype), rand(2, 5100, 2, 64, dtype=dtype), rand(3, 5100, 2, 64, dtype=dtype)
    size = torch.ones(200, 4, 1, device="cuda")
    size[:70] *= 1e-3
    size[:, 2:] *= 0.1
    size[70::2] *= 1e-2  # every other row of the last graph
    do = (rand(4, 200, 4, 64) * size).to(dtype)
    keep = (rand(5, 5100) < 1.3).to(torch.uint8)
    v[keep == 0] = float("inf")
    host = [values(t) for t in (q, k, v)]
    host[2][keep.cpu().numpy() == 0] = 0
    ref, _ = update.attention_vjp(*host, *off, at.scale, values(do), keep.cpu().numpy())
    dq, dk, dv = gradients(q, k, v, do, at, keep)
    for a, b in ((0, 70), (70, 200)):
        for h in range(4):
            for part in (slice(a, b, 2), slice(a + 1, b, 2)):
                r = ref[0][part, h]
                assert relative(dq[part, h], r) <= gradient_limit(r, dtype), (a, h)
    for a, b in ((0, 3000), (3000, 5100)):
        for h in range(2):
            for got, r in ((dk, ref[1]), (dv, ref[2])):
                assert relative(got[a:b, h], r[a:b, h]) <= gradient_limit(r[a:b, h], dtype), (a, h)


# ------------------------------------------------------------------- rows whose mask leaves nothing

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("rows, states", [(1, 70), (150, 300), (1, 6000)])
def test_rows_without_a_kept_state(rows, states, d, kind):
    """Zeros, lse -inf and zero gradients, as for a graph without states, whatever q and d_out hold; the other graph's rows, whose
    NaN meet kept states, are NaN."""
    dtype, n = TYPES[kind], 3 * rows
    at = uvu.Attention(2, 1, d, i32([0, rows, 2 * rows, n]), i32([0, states, states, 2 * states]), rows, states)
    q, k, v, do = (rand(i, m, h, d, dtype=dtype) for i, (m, h) in enumerate(((n, 2), (2 * states, 1), (2 * states, 1), (n, 2))))
    q[:rows, 0], q[0, 1, 0], do[:rows, :, 0] = float("nan"), float("inf"), float("nan")
    q[rows], do[rows] = float("nan"), float("inf")
    q[2 * rows, 0] = float("nan")
    keep = torch.ones(2 * states, dtype=torch.uint8, device="cuda")
    keep[:states] = 0
    keep[states + states // 2:] = 0  # pieces of the last graph are masked, too
    out, lse = torch.empty_like(q), torch.empty(n, 2, device="cuda")
    at.fwd(q, k, v, out, lse, keep=keep)
    g = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    at.bwd(q, k, v, out, lse, do, *g, keep=keep)
    assert (out[:2 * rows] == 0).all() and torch.isneginf(lse[:2 * rows]).all() and (g[0][:2 * rows] == 0).all()
    assert (g[1][:states] == 0).all() and (g[2][:states] == 0).all()
    assert torch.isnan(out[2 * rows, 0]).all() and torch.isnan(lse[2 * rows, 0]) and torch.isnan(g[0][2 * rows, 0]).all()
    assert torch.isfinite(out[2 * rows, 1]).all() and torch.isfinite(lse[2 * rows, 1])


# ------------------------------------------------------------------------------------ empty batches

@pytest.mark.parametrize("nodes, states", [(0, 0), (0, 5), (6, 0)])
def test_node_update_of_empty_sides(nodes, states):
    """A batch without nodes, or whose encoder has no states: finite outputs and gradients of the right shapes."""
    at = uvu.Attention(4, 2, 16, i32([0, 0, nodes]), i32([0, 0, states]))
    m, ctx = rand(1, nodes, 64, 4).requires_grad_(True), rand(2, states, 24).requires_grad_(True)
    weights = [rand(3 + i, *s).requires_grad_(True) for i, s in enumerate(((64,), (64,), (64, 64), (24, 32), (24, 32), (64, 64)))]
    s, h = autograd.node_update(m, at.q_offsets, ctx, at, weights, 8, p=0.25, seed=3)
    assert s.shape == (nodes, 64) and h.shape == (nodes, 64, 4)
    g = torch.autograd.grad(s.sum() + h.sum(), (m, ctx, *weights))
    assert all(torch.isfinite(t).all() for t in (s, h, *g))
    if states == 0:  # nothing is attended to
        assert all((t == 0).all() for t in (g[1], *g[4:]))


# ----------------------------------------------------------- norms of 16-bit results, two row tiles a block

NORMED = [  # q lengths, k lengths, q heads, kv heads, head dim, kept share (None: no mask)
    ([40, 0, 200], [900, 5, 333], 4, 2, 64, 0.9), ([300], [1500], 2, 2, 16, None), ([129, 7], [700, 90], 6, 2, 33, 0.6),
    ([1] * 6, [800] * 6, 8, 2, 128, None), ([500], [1100], 2, 1, 128, 0.9), ([2000], [2600], 2, 1, 32, None), ([1500], [1500], 1, 1, 96, 0.5)]


def of_case(case, dtype, view=0):
    ql, kl, hq, hk, d, share = case
    qo, ko = (np.concatenate([[0], np.cumsum(n)]) for n in (ql, kl))
    # `view` values into a row, so that no row begins on 16 bytes
    t = [rand(i, n, h, d + view, dtype=dtype)[:, :, view:] for i, (n, h) in enumerate(((qo[-1], hq), (ko[-1], hk), (ko[-1], hk), (qo[-1], hq)))]
    t[2] += 0.25  # a mean, as encodings have, gives delta its weight
    g = torch.Generator(device="cuda").manual_seed(5)
    keep = None if share is None else (torch.rand(int(ko[-1]), generator=g, device="cuda") < share).to(torch.uint8)
    return t, keep, qo, ko, uvu.Attention(hq, hk, d, i32(qo), i32(ko), max(ql), max(kl))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("case", NORMED, ids=lambda c: f"q{max(c[0])}-k{max(c[1])}-h{c[2]}.{c[3]}-d{c[4]}-{c[5]}")
def test_norms_of_16_bit_results(case, kind):
    """The elementwise bounds of long rows exceed the gradients themselves; their norms see a lost term or a wrong factor."""
    dtype = TYPES[kind]
    (q, k, v, do), keep, qo, ko, at = of_case(case, dtype)
    host = None if keep is None else keep.cpu().numpy()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    at.fwd(q, k, v, out, lse, keep=keep)
    ref = update.attention(*map(values, (q, k, v)), qo, ko, at.scale, host)[0]
    assert relative(out, ref) <= output_limit(ref, dtype), relative(out, ref)
    ref, _ = update.attention_vjp(*map(values, (q, k, v)), qo, ko, at.scale, values(do), host)
    for name, got, r in zip(("dq", "dk", "dv"), gradients(q, k, v, do, at, keep), ref):
        assert relative(got, r) <= gradient_limit(r, dtype), (name, relative(got, r), gradient_limit(r, dtype))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("share", [None, 0.8])
@pytest.mark.parametrize("d, view", [(16, 0), (30, 0), (32, 0), (64, 0), (64, 1), (96, 0), (128, 0), (128, 1)])
def test_two_row_tiles_a_block(d, view, share, kind):
    """The forward that takes 256 rows a block, which it does once they fill the SMs: all classes of head dimensions, with
    and without a mask, operands off the 16-byte grid, walks longer than the ring of masks, graphs whose second tile is empty."""
    dtype, hk = TYPES[kind], 8
    case = ([4000, 129, 1, 0, 900], [1300, 70, 257, 3, 0], hk, hk, d, share)
    assert ((5030 // 256 + 5) * hk) >= torch.cuda.get_device_properties(0).multi_processor_count
    (q, k, v, _), keep, qo, ko, at = of_case(case, dtype, view)
    out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:2], float("nan"), device="cuda")
    at.fwd(q, k, v, out, lse, keep=keep)
    ref, ref_lse, mag = update.attention(*map(values, (q, k, v)), qo, ko, at.scale, None if keep is None else keep.cpu().numpy())
    got = values(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref_lse))
    kept = ~np.isneginf(ref_lse)
    assert np.abs(got[kept] - ref_lse[kept]).max() <= 1e-4
    assert (np.abs(values(out) - ref) <= 3 * unit(dtype) * (np.abs(ref) + mag) + 1e-4).all()
    for a, b in ((0, 4000), (4000, 4129), (4129, 4130)):
        for h in range(hk):
            assert relative(out[a:b, h], ref[a:b, h]) <= output_limit(ref[a:b, h], dtype), (a, h)
    assert (out[4130:] == 0).all()
    assert uvu.Attention.device_status() == 0


# ---------------------------------------------------------------- group norm of graphs longer than promised

@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("most", [1, None])
def test_group_norm_of_a_long_graph_with_a_mean(most, kind):
    """Values of 5 +- 1.5 over 140000 rows, also with a max_rows that promised one, element by element (no row begins on 16 bytes):
    the statistics keep fp32's accuracy whatever the length, so mean, rstd, dgamma and dbeta meet the fp32 tolerance."""
    n, c, groups, dtype = 140000, 96, 2, TYPES[kind]
    flat, dy = (rand(1, n * c + 1) * 1.5 + 5).to(dtype), rand(2, n, c, dtype=dtype)
    x, off = flat[1:].view(n, c), i32([0, n])
    gamma, beta = 1 + 0.2 * rand(3, c), 0.2 * rand(4, c)
    y, dx, mean, rstd, dg, db = (torch.full(s, float("nan"), dtype=t, device="cuda") for s, t in
                                 (((n, c), dtype), ((n, c), dtype), ((1, groups), torch.float32), ((1, groups), torch.float32),
                                  ((c,), torch.float32), ((c,), torch.float32)))
    uvu.group_norm_fwd(x, gamma, beta, off, groups, y, mean, rstd, max_rows=most)
    uvu.group_norm_bwd(dy, x, gamma, beta, off, groups, mean, rstd, dx, dg, db, max_rows=most)
    host = [values(t) for t in (x, gamma, beta)]
    _, rm, rr = update.group_norm(*host, [0, n], groups, True, 1e-5)
    _, rg, rb = update.group_norm_vjp(*host, [0, n], groups, True, 1e-5, values(dy))
    for got, ref, what in ((mean, rm, "mean"), (rstd, rr, "rstd"), (dg, rg, "dgamma"), (db, rb, "dbeta")):
        check(values(got), ref, False, what)
    # 5 +- 1.5 is known to 5 * 2^-24 in fp32; a sum of 48 n values may cost a few of these, not a hundred
    assert np.abs(values(mean) - rm).max() <= 8 * 5 * 2.0 ** -24


# ------------------------------------------------------------------------------ sums over very long walks

def exact_rows(q, k, v, scale, rows):
    """out and lse of some rows of one head, in fp64 on the device."""
    s = q[rows, 0].double() @ k[:, 0].double().T * scale
    lse = torch.logsumexp(s, 1)
    return torch.exp(s - lse[:, None]) @ v[:, 0].double(), lse


def long_walk(kind, nq, nk, d):
    """Values of one sign, whose sums show every loss: relative Frobenius errors of out (some rows) and lse, and out's values."""
    dtype = TYPES[kind]
    q, k, v = rand(1, nq, 1, d, dtype=dtype), rand(2, nk, 1, d, dtype=dtype), (rand(3, nk, 1, d) * 0.1 + 1).to(dtype)
    at = uvu.Attention(1, 1, d, i32([0, nq]), i32([0, nk]))
    out, lse = torch.empty_like(q), torch.empty(nq, 1, device="cuda")
    at.fwd(q, k, v, out, lse)
    rows = torch.arange(0, nq, max(1, nq // 31), device="cuda")
    ref, ref_lse = exact_rows(q, k, v, at.scale, rows)
    assert (lse[rows, 0].double() - ref_lse).abs().max() <= 1e-5
    return out[rows, 0], values(ref)


@pytest.mark.parametrize("nq, d", [(24576, 64), (24576, 20), (24576, 128), (100, 64)])
def test_sums_of_long_walks_f32(nq, d):
    """2^20 states in one walk, or in pieces: the fp32 tolerance holds."""
    got, ref = long_walk("f32", nq, 2 ** 20, d)
    check(values(got), ref, False, "out")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq, nk, d", [(24576, 2 ** 20, 64), (40000, 2 ** 20, 64), (40000, 2 ** 20, 20), (40000, 2 ** 20, 128), (16, 2 ** 23, 64)])
def test_sums_of_long_walks(nq, nk, d, kind):
    """A sum in tensor memory loses up to 2^-23 of itself with every 16 states: longer walks do without."""
    got, ref = long_walk(kind, nq, nk, d)
    assert relative(got, ref) <= output_limit(ref, TYPES[kind]), relative(got, ref)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq", [24576, 40000])
@pytest.mark.parametrize("d", [32, 33, 128])
def test_long_walks_with_a_rising_maximum(nq, d, kind):
    """Scores that rise along the states, with the first ones masked: what a walk holds is taken over at every reference."""
    dtype, nk = TYPES[kind], 200000
    rise = torch.linspace(-1, 1, nk, device="cuda")[:, None, None]
    q = (1 + 0.3 * rand(1, nq, 1, d)).to(dtype)
    k, v = (rise * 24 / d + 0.02 * rand(2, nk, 1, d)).to(dtype), (rand(3, nk, 1, d) + rise).to(dtype)
    keep = (rand(4, nk) < 0.5).to(torch.uint8)
    keep[:70000] = 0
    at = uvu.Attention(1, 1, d, i32([0, nq]), i32([0, nk]), scale=1.0)
    out, lse = torch.empty_like(q), torch.empty(nq, 1, device="cuda")
    at.fwd(q, k, v, out, lse, keep=keep)
    rows = torch.arange(0, nq, max(1, nq // 31), device="cuda")
    j = keep != 0
    ref, ref_lse = exact_rows(q, k[j], v[j], 1.0, rows)
    assert (lse[rows, 0].double() - ref_lse).abs().max() <= 1e-4
    assert relative(out[rows, 0], values(ref)) <= output_limit(values(ref), dtype)


def one_sign(dtype, nq, nk, hq, hk, d):
    """Operands whose gradients' terms are mostly of one sign: v follows k, q and d_out have a mean."""
    q, k = (rand(1, nq, hq, d) * 0.1 + 0.3).to(dtype), rand(2, nk, hk, d, dtype=dtype)
    return q, k, (k.float() + 0.1 * rand(3, nk, hk, d)).to(dtype), (rand(4, nq, hq, d) * 0.1 + 1).to(dtype)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 36])
def test_gradient_sums_over_many_states(d, kind):
    """dq over 2^21 states, unsplit."""
    nq, nk, dtype = 20480, 2 ** 21, TYPES[kind]
    q, k, v, do = one_sign(dtype, nq, nk, 1, 1, d)
    at = uvu.Attention(1, 1, d, i32([0, nq]), i32([0, nk]))
    got = gradients(q, k, v, do, at)[0]
    rows = torch.arange(0, nq, 2000, device="cuda")
    s = q[rows, 0].double() @ k[:, 0].double().T * at.scale
    p = torch.softmax(s, 1)
    dp = do[rows, 0].double() @ v[:, 0].double().T
    ref = (p * (dp - (p * dp).sum(1, keepdim=True)) * at.scale) @ k[:, 0].double()
    assert relative(got[rows, 0], values(ref)) <= gradient_limit(values(ref), dtype), relative(got[rows, 0], values(ref))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("masked", [False, True])
def test_gradient_sums_over_many_rows(masked, kind):
    """dk and dv of states that 2^19 packed rows attend to, unsplit (152 tiles of states), some of them masked."""
    nq, nk, hk, group, d, dtype = 2 ** 16, 2432, 8, 8, 64, TYPES[kind]
    q, k, v, do = one_sign(dtype, nq, nk, hk * group, hk, d)
    keep = (rand(5, nk) < 1).to(torch.uint8) if masked else None
    at = uvu.Attention(hk * group, hk, d, i32([0, nq]), i32([0, nk]))
    dk, dv = gradients(q, k, v, do, at, keep)[1:]
    j = torch.arange(nk, device="cuda") if keep is None else torch.nonzero(keep)[:, 0]
    h, some = 5, j[::100]
    K, V = k[j, h].double(), v[j, h].double()
    r_dk = r_dv = 0
    for c in range(0, nq, 4096):
        Q, dO = (t[c:c + 4096, h * group:(h + 1) * group].reshape(-1, d).double() for t in (q, do))
        p = torch.softmax(Q @ K.T * at.scale, 1)
        delta = ((p @ V) * dO).sum(1, keepdim=True)
        p = p[:, ::100]
        r_dv = r_dv + p.T @ dO
        r_dk = r_dk + (p * (dO @ V[::100].T - delta) * at.scale).T @ Q
    for name, got, ref in (("dk", dk, r_dk), ("dv", dv, r_dv)):
        assert relative(got[some, h], values(ref)) <= gradient_limit(values(ref), dtype), (name, relative(got[some, h], values(ref)))
    if masked:
        assert (dk[keep == 0] == 0).all() and (dv[keep == 0] == 0).all()

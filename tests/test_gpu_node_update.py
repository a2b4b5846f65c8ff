"""autograd.group_norm, cross_attention, dropout and node_update: the operators as a training step uses
them, against a plain fp64 PyTorch formula of the same block and the oracle's convolution.

Tolerances: the block is a chain of five fp32 stages each way (convolution, norm, products, attention,
products), each of which its own tests hold to a relative Frobenius error of 1e-5, so outputs are held to
5e-5 and gradients, which pass the chain twice, to 1e-4."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import autograd, uvu, workloads
from gpu_util import Problem, dev
from oracle import conv, update

pytestmark = pytest.mark.gpu


def near(got, ref, tol, what):
    got, ref = got.detach().double().cpu(), torch.as_tensor(ref, dtype=torch.float64)
    assert got.shape == ref.shape, what
    err = float((got - ref).norm() / ref.norm())
    assert err <= tol, f"{what}: relative Frobenius error {err:.2e} > {tol}"


def plain_block(m, off, ctx, c_off, weights, groups, hq, hkv, d, p, seed, offset, keep):
    """node_update by its formulas, in fp64."""
    gamma, beta, w_q, w_k, w_v, w_o = weights
    n, u, dim = m.shape
    s = []
    for a, b in zip(off[:-1], off[1:]):
        if a == b:
            continue
        t = m[a:b, :, 0].reshape(b - a, groups, u // groups)
        mean = t.mean((0, 2), keepdim=True)
        var = (t - mean).square().mean((0, 2), keepdim=True)
        z = ((t - mean) / (var + 1e-5).sqrt()).reshape(b - a, u) * gamma + beta
        s.append(z * torch.sigmoid(z))
    s = torch.cat(s)
    q, k, v = (s @ w_q).view(n, hq, d), (ctx @ w_k).view(-1, hkv, d), (ctx @ w_v).view(-1, hkv, d)
    rows = []
    for g in range(len(off) - 1):
        pick = [i for i in range(c_off[g], c_off[g + 1]) if keep[i]]
        for i in range(off[g], off[g + 1]):
            if not pick:
                rows.append(torch.zeros(hq, d, dtype=torch.float64))
                continue
            kk, vv = (t[pick].repeat_interleave(hq // hkv, 1) for t in (k, v))
            prob = torch.softmax(torch.einsum("hd,khd->hk", q[i], kk) * d ** -0.5, 1)
            rows.append(torch.einsum("hk,khd->hd", prob, vv))
    a = torch.stack(rows).reshape(n, -1) @ w_o

    def drop(t, at):
        k, scale = update.keep_mask(n * u, p, seed, at)
        k = torch.from_numpy(k.reshape(n, u)) * scale
        return t * (k if t.dim() == 2 else k[:, :, None])

    s = s + drop(a, offset)
    return s, drop(m * torch.sigmoid(s)[:, :, None], offset + (n * u + 7) // 8)


def test_block_after_a_convolution():
    rng = np.random.default_rng(31)
    off, c_off = np.array([0, 7, 7, 19, 40], np.int32), np.array([0, 33, 40, 40, 71], np.int32)
    N, U, F, hq, hkv, d, groups = 40, 64, 24, 4, 2, 16, 8
    spec = workloads.custom_spec(720, N, "64x0e+64x1o", "1x0e+1x1o+1x2e", 2, "float32")
    recv, src = workloads.random_degree_graph(N, rng.integers(1, 9, size=N), rng)
    Y = workloads.sh_inputs(workloads.unit_vectors(src.size, rng), 2).astype(np.float32)
    P = Problem(spec, recv, src, rng.standard_normal((N, U, 4)).astype(np.float32), Y, N)
    D = P.plan.info.dim_out
    keep = rng.random(71) < 0.8
    ctx = rng.standard_normal((71, F)).astype(np.float32)
    shapes = [(U,), (U,), (U, hq * d), (F, hkv * d), (F, hkv * d), (hq * d, U)]
    weights = [rng.standard_normal(s).astype(np.float32) * (s[0] ** -0.5 if len(s) == 2 else 1) for s in shapes]
    c_s, c_h = rng.standard_normal((N, U)).astype(np.float32), rng.standard_normal((N, U, D)).astype(np.float32)
    p, seed, at = 0.25, 12345, 1000

    x, Yt, w, ct, *wt = (dev(a).requires_grad_(True) for a in (P.x, P.Y, P.w, ctx, *weights))
    attention = uvu.Attention(hq, hkv, d, dev(off), dev(c_off), max_q=21, max_k=33)
    m = autograd.uvu_conv(x, Yt, w, P.plan, P.G)
    s, h = autograd.node_update(m, dev(off), ct, attention, wt, groups, p=p, seed=seed, offset=at, keep=dev(keep), max_rows=21)
    got = torch.autograd.grad((s * dev(c_s)).sum() + (h * dev(c_h)).sum(), (x, Yt, w, ct, *wt))

    m64 = torch.from_numpy(conv.fwd(P.lay, P.off_host, P.src, P.x, P.Y, P.w)).requires_grad_(True)
    c64, *w64 = (torch.from_numpy(a).double().requires_grad_(True) for a in (ctx, *weights))
    r_s, r_h = plain_block(m64, off, c64, c_off, w64, groups, hq, hkv, d, p, seed, at, keep)
    near(s, r_s.detach(), 5e-5, "s")
    near(h, r_h.detach(), 5e-5, "h")
    g_m, *g_rest = torch.autograd.grad((r_s * torch.from_numpy(c_s)).sum() + (r_h * torch.from_numpy(c_h)).sum(), (m64, c64, *w64))
    r_dY, r_dw = conv.bwd_edges(P.lay, P.off_host, P.src, P.x, P.Y, P.w, g_m.numpy())
    ref = [conv.bwd_dx(P.lay, P.off_host, P.src, P.Y, P.w, g_m.numpy(), N), r_dY, r_dw, *g_rest]
    for g, r, what in zip(got, ref, ("dx", "dY", "dw", "dcontext", "dgamma", "dbeta", "dw_q", "dw_k", "dw_v", "dw_o")):
        near(g, r, 1e-4, what)
    # dropped channels are dropped whole, and the masks are the counters' own
    k, _ = update.keep_mask(N * U, p, seed, at + N * U // 8)
    assert torch.equal((h != 0).any(2).cpu(), torch.from_numpy(k.reshape(N, U)))
    assert P.status_ok() and uvu.Attention.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16], ids=["f32", "bf16", "f16"])
def test_operators_give_the_library_results(dtype):
    """The autograd forms return what the entry points return, bit for bit, on views and shared heads too."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    off, c_off = dev(np.array([0, 5, 30], np.int32)), dev(np.array([0, 40, 41], np.int32))
    at = uvu.Attention(4, 2, 24, off, c_off)
    q = rand(30, 4, 24).requires_grad_(True)
    kv = rand(41, 2, 2, 24).requires_grad_(True)
    out = autograd.cross_attention(q, kv[:, 0], kv[:, 1], at)
    do = rand(30, 4, 24)
    dq, dkv = torch.autograd.grad(out, (q, kv), do)
    r, lse = torch.empty_like(do), torch.empty(30, 4, device="cuda")
    k, v = kv[:, 0].detach().contiguous(), kv[:, 1].detach().contiguous()
    at.fwd(q.detach(), k, v, r, lse)
    rq, rk, rv = torch.empty_like(r), torch.empty_like(k), torch.empty_like(v)
    at.bwd(q.detach(), k, v, r, lse, do, dq=rq, dk=rk, dv=rv)
    assert torch.equal(out, r) and torch.equal(dq, rq) and torch.equal(dkv, torch.stack([rk, rv], 1))
    # only one side asked for; one kv head broadcast to two
    (only,) = torch.autograd.grad(autograd.cross_attention(q, k, v, at), (q,), do)
    assert torch.equal(only, rq)
    one = rand(41, 1, 24).requires_grad_(True)
    (d_one,) = torch.autograd.grad(autograd.cross_attention(q, one.expand(-1, 2, -1), v, at), (one,), do)
    at.fwd(q.detach(), one.detach().expand(-1, 2, -1).contiguous(), v, r, lse)
    at.bwd(q.detach(), one.detach().expand(-1, 2, -1).contiguous(), v, r, lse, do, dk=rk, dv=rv)
    assert torch.equal(d_one, rk.sum(1, keepdim=True))

    x, res = rand(30, 16).requires_grad_(True), rand(30, 16).requires_grad_(True)
    gamma, beta = torch.rand(16, device="cuda").requires_grad_(True), torch.rand(16, device="cuda").requires_grad_(True)
    y = autograd.group_norm(x, gamma, beta, off, 4)
    z = autograd.dropout(y, 0.5, 7, offset=3, residual=res)
    dz = rand(30, 16)
    dx, dg, db, dres = torch.autograd.grad(z, (x, gamma, beta, res), dz)
    ry, mean, rstd = torch.empty_like(dz), torch.empty(2, 4, device="cuda"), torch.empty(2, 4, device="cuda")
    xd, gd, bd = x.detach(), gamma.detach(), beta.detach()
    uvu.group_norm_fwd(xd, gd, bd, off, 4, ry, mean, rstd)
    rz, rdy, rdx, rg, rb = torch.empty_like(dz), torch.empty_like(dz), torch.empty_like(dz), torch.empty_like(gd), torch.empty_like(gd)
    uvu.dropout_fwd(ry, 0.5, 7, rz, offset=3, residual=res.detach())
    uvu.dropout_bwd(dz, 0.5, 7, rdy, offset=3)
    uvu.group_norm_bwd(rdy, xd, gd, bd, off, 4, mean, rstd, rdx, rg, rb)
    assert torch.equal(z, rz) and torch.equal(dx, rdx) and torch.equal(dg, rg) and torch.equal(db, rb) and torch.equal(dres, dz)


def test_example_trains():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "node_update.py")
    spec = importlib.util.spec_from_file_location("node_update_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    first, last = example.train(n_molecules=16, steps=60)
    assert np.isfinite(last) and last < 0.5 * first, (first, last)

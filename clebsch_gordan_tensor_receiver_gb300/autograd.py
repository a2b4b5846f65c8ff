"""PyTorch autograd for the UVU convolution, through the library's C ABI only.

`uvu_conv(x, Y, w, plan, graph)` returns out [N][U][D_out].  Its backward is the VJP
(uvu_conv_bwd: dx, dY, dw), and the VJP's own backward is the double backward (uvu_conv_hvp), so
`torch.autograd.grad(..., create_graph=True)` followed by a second `grad` (forces in training, as
in "Receiver-streaming convolutions for channel-wise UVU tensor products", results table: HVP
column) runs on the library's kernels.  Third derivatives are not provided.

`group_norm`, `cross_attention` and `dropout` are the node-update operators with first derivatives,
and `node_update` chains them after a convolution.  `embedding` and `rms_norm` are the lookup of first features
and the norm between layers, with first derivatives.

Every tensor is a contiguous CUDA tensor of the plan's dtype in the layouts of include/uvu.h;
`graph` is a `uvu.Graph` (receiver CSR and transposed CSR) of the same edges.  This module only
marshals arguments: every step runs in the library (`node_update`'s four dense products in PyTorch).
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import uvu


def _c(t):
    return t.contiguous()


class _ConvVJP(torch.autograd.Function):
    """(x, Y, w, g) -> (dx, dY, dw); backward = the double backward."""

    @staticmethod
    def forward(ctx, x, Y, w, g, plan, graph, dx_mode):
        n, e, i = graph.n_nodes, graph.n_edges, plan.info
        dx = torch.empty_like(x)
        dY = torch.empty(max(e, 1), i.dim_sh, dtype=x.dtype, device=x.device)[:e]
        dw = torch.empty(max(e, 1), i.n_paths, i.mul, dtype=x.dtype, device=x.device)[:e]
        plan.bwd(n, x, Y, w, graph.recv_offsets, graph.src, graph.send_offsets, graph.send_eids,
                 graph.send_recv, g, dx=dx, dY=dY, dw=dw, dx_mode=dx_mode)
        ctx.save_for_backward(x, Y, w, g)
        ctx.plan, ctx.graph = plan, graph
        return dx, dY, dw

    @staticmethod
    @once_differentiable
    def backward(ctx, ax, aY, aw):
        x, Y, w, g = ctx.saved_tensors
        plan, graph = ctx.plan, ctx.graph
        n, e = graph.n_nodes, graph.n_edges
        need = ctx.needs_input_grad
        gx = torch.empty_like(x) if need[0] else None
        gY = torch.empty_like(Y) if need[1] and e > 0 else (torch.zeros_like(Y) if need[1] else None)
        gw = torch.empty_like(w) if need[2] and e > 0 else (torch.zeros_like(w) if need[2] else None)
        gg = torch.empty_like(g) if need[3] else None
        plan.hvp(n, x, Y, w, graph.recv_offsets, graph.src, graph.send_offsets, graph.send_eids, g,
                 ax=None if ax is None else _c(ax), aY=None if aY is None else _c(aY),
                 aw=None if aw is None else _c(aw), grad_d_out=gg, grad_x=gx,
                 grad_Y=gY if e > 0 else None, grad_w=gw if e > 0 else None)
        return gx, gY, gw, gg, None, None, None


class _Conv(torch.autograd.Function):
    """(x, Y, w) -> out; backward = the VJP (itself differentiable once more)."""

    @staticmethod
    def forward(ctx, x, Y, w, plan, graph, dx_mode):
        i = plan.info
        out = torch.empty(graph.n_nodes, i.mul, i.dim_out, dtype=x.dtype, device=x.device)
        plan.fwd(graph.n_nodes, x, Y, w, graph.recv_offsets, graph.src, out)
        ctx.save_for_backward(x, Y, w)
        ctx.plan, ctx.graph, ctx.dx_mode = plan, graph, dx_mode
        return out

    @staticmethod
    def backward(ctx, g):
        x, Y, w = ctx.saved_tensors
        dx, dY, dw = _ConvVJP.apply(x, Y, w, _c(g), ctx.plan, ctx.graph, ctx.dx_mode)
        return dx, dY, dw, None, None, None


def uvu_conv(x, Y, w, plan: "uvu.Plan", graph: "uvu.Graph", dx_mode: int = uvu.UVU_DX_STAGED):
    """out = the UVU convolution of x [N][U][D_x], Y [E][D_Y], w [E][P][U] over `graph`, with
    autograd support up to second order (VJP and double backward run in the library)."""
    return _Conv.apply(_c(x), _c(Y), _c(w), plan, graph, dx_mode)


class _RadialHidden(torch.autograd.Function):
    """r [E] -> h [E][widths[-1]] (uvu_radial_hidden); backward = uvu_radial_hidden_bwd (dr and
    the layers' gradients)."""

    @staticmethod
    def forward(ctx, r, weights, plan, r_cut, p_env, widths):
        h = torch.empty(r.numel(), widths[-1], dtype=r.dtype, device=r.device)
        plan.radial_hidden(r, r_cut, p_env, widths, weights, h)
        ctx.save_for_backward(r, weights)
        ctx.plan, ctx.r_cut, ctx.p_env, ctx.widths = plan, r_cut, p_env, widths
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        r, weights = ctx.saved_tensors
        dr = torch.empty_like(r)
        dW = torch.empty_like(weights)
        ctx.plan.radial_hidden_bwd(r, ctx.r_cut, ctx.p_env, ctx.widths, weights, _c(dh), dr, dW)
        return dr, dW, None, None, None, None


class _RadialWeights(torch.autograd.Function):
    """(h, W_last) -> w = h W_last (uvu_radial_weights); backward = uvu_radial_weights_bwd."""

    @staticmethod
    def forward(ctx, h, w_last, plan):
        i = plan.info
        w = torch.empty(h.shape[0], i.n_paths, i.mul, dtype=h.dtype, device=h.device)
        plan.radial_weights(h, w_last, w)
        ctx.save_for_backward(h, w_last)
        ctx.plan = plan
        return w

    @staticmethod
    @once_differentiable
    def backward(ctx, dw):
        h, w_last = ctx.saved_tensors
        need = ctx.needs_input_grad
        dh = torch.empty_like(h) if need[0] else None
        dwl = torch.empty_like(w_last) if need[1] else None
        ctx.plan.radial_weights_bwd(h, w_last, _c(dw), dh=dh, dw_last=dwl)
        return dh, dwl, None


def radial_conv(r, x, Y, weights, w_last, plan: "uvu.Plan", graph: "uvu.Graph", r_cut: float, p_env: int,
                widths, dx_mode: int = uvu.UVU_DX_STAGED):
    """The convolution with radial weights from edge lengths r [E]: h = uvu_radial_hidden(r) (the
    SiLU network, layers back to back in `weights`), w = h W_last (materialised on the tensor
    cores), out = uvu_conv(x, Y, w).  First derivatives with respect to r (forces), x, Y, the
    layers and W_last run in the library; second derivatives through the radial network are not
    provided."""
    h = _RadialHidden.apply(_c(r), _c(weights), plan, float(r_cut), int(p_env), [int(v) for v in widths])
    w = _RadialWeights.apply(h, _c(w_last), plan)
    return uvu_conv(x, Y, w, plan, graph, dx_mode)


class _GroupNorm(torch.autograd.Function):
    """(x, gamma, beta) -> y (uvu_group_norm_fwd); backward = uvu_group_norm_bwd."""

    @staticmethod
    def forward(ctx, x, gamma, beta, offsets, groups, act, eps, max_rows):
        y = torch.empty_like(x)
        mean = torch.empty(offsets.numel() - 1, groups, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        uvu.group_norm_fwd(x, gamma, beta, offsets, groups, y, mean, rstd, act=act, eps=eps, max_rows=max_rows)
        ctx.save_for_backward(x, gamma, beta, offsets, mean, rstd)
        ctx.groups, ctx.act, ctx.max_rows = groups, act, max_rows
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gamma, beta, offsets, mean, rstd = ctx.saved_tensors
        dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
        uvu.group_norm_bwd(_c(dy), x, gamma, beta, offsets, ctx.groups, mean, rstd, dx, dgamma, dbeta, act=ctx.act,
                           max_rows=ctx.max_rows)
        return dx, dgamma, dbeta, None, None, None, None, None


def group_norm(x, gamma, beta, offsets, groups: int, act: int = uvu.UVU_ACT_SILU, eps: float = 1e-5, max_rows=None):
    """y = act(group norm of x [N][C]) over the rows of each graph (`offsets` [B+1] int32), in fp32, bf16 or
    f16; gamma and beta [C] fp32.  `max_rows`: a length that no graph exceeds (a hint)."""
    return _GroupNorm.apply(_c(x), _c(gamma), _c(beta), offsets, int(groups), act, float(eps), max_rows)


def _heads(t):
    return t if t.stride(-1) == 1 else t.contiguous()


class _CrossAttention(torch.autograd.Function):
    """(q, k, v) -> out (uvu_attn_fwd); backward = uvu_attn_bwd, with only the gradients that are asked for."""

    @staticmethod
    def forward(ctx, q, k, v, attention, keep):
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
        attention.fwd(q, k, v, out, lse, keep=keep)
        ctx.save_for_backward(q, k, v, out, lse, *([] if keep is None else [keep]))
        ctx.attention = attention
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        q, k, v, out, lse, *keep = ctx.saved_tensors
        new = lambda t: torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
        dq = new(q) if ctx.needs_input_grad[0] else None
        dk, dv = (new(k), new(v)) if any(ctx.needs_input_grad[1:3]) else (None, None)
        ctx.attention.bwd(q, k, v, out, lse, _c(d_out), dq=dq, dk=dk, dv=dv, keep=keep[0] if keep else None)
        return dq, dk, dv, None, None


def cross_attention(q, k, v, attention: "uvu.Attention", keep=None):
    """The attention of q [Tq][q_heads][D] to the states k, v [Tk][kv_heads][D] of the same graph; `keep` [Tk]
    (uint8 or bool): states with 0 take no part.  Rows without a kept state give zeros and take no gradient."""
    return _CrossAttention.apply(_heads(q), _heads(k), _heads(v), attention, keep)


class _Dropout(torch.autograd.Function):
    """(x, residual) -> residual + dropout(x) (uvu_dropout_fwd); backward = uvu_dropout_bwd."""

    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, inner):
        y = torch.empty_like(x)
        uvu.dropout_fwd(x, p, seed, y, offset=offset, inner=inner, residual=residual)
        ctx.p, ctx.seed, ctx.offset, ctx.inner = p, seed, offset, inner
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dx = None
        if ctx.needs_input_grad[0]:
            dy = _c(dy)
            dx = torch.empty_like(dy)
            uvu.dropout_bwd(dy, ctx.p, ctx.seed, dx, offset=ctx.offset, inner=ctx.inner)
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None, None


def dropout(x, p: float, seed: int, offset: int = 0, inner: int = 1, residual=None):
    """residual + dropout(x), the mask a function of (seed, offset) that the backward forms again; `inner`
    consecutive values share a draw.  A call uses ceil(x.numel() / inner / 8) offsets."""
    return _Dropout.apply(_c(x), None if residual is None else _c(residual), float(p), int(seed), int(offset), int(inner))


def node_update(m, offsets, context, attention: "uvu.Attention", weights, groups: int, p: float = 0.0, seed: int = 0,
                offset: int = 0, keep=None, scalar: int = 0, max_rows=None):
    """The update of the nodes after a convolution: m [N][U][D] is uvu_conv's output for a packed batch of
    graphs (node `offsets` [B+1] int32), context [Tk][F] the states of an encoder that the graphs attend to.

        s = silu(group norm of m's invariant column)      [N][U]
        s = s + dropout(attention(s w_q, context w_k, context w_v) w_o)
        h = dropout of whole channels (m sigmoid(s))      [N][U][D]

    weights: gamma, beta [U], w_q [U][q_heads D_h], w_k, w_v [F][kv_heads D_h], w_o [q_heads D_h][U].  `scalar` is a
    column of D that belongs to a 0e path (column 0 of the first path where x and sh begin with 0e).  A dropped channel
    loses all of its components, so h stays equivariant.  Returns (s, h); uses two calls' offsets."""
    gamma, beta, w_q, w_k, w_v, w_o = weights
    n, u, d = m.shape
    s = group_norm(m[:, :, scalar], gamma, beta, offsets, groups, max_rows=max_rows)
    q = (s @ w_q).view(n, attention.q_heads, attention.head_dim)
    k = (context @ w_k).view(-1, attention.kv_heads, attention.head_dim)
    v = (context @ w_v).view(-1, attention.kv_heads, attention.head_dim)
    a = cross_attention(q, k, v, attention, keep).reshape(n, attention.q_heads * attention.head_dim) @ w_o
    s = dropout(a, p, seed, offset, residual=s)
    h = dropout(m * torch.sigmoid(s)[:, :, None], p, seed, offset + (n * u + 7) // 8, inner=d)
    return s, h


class _Embedding(torch.autograd.Function):
    """table -> rows of it (uvu_embed_fwd); backward = uvu_embed_bwd."""

    @staticmethod
    def forward(ctx, table, index, scale, inner, column):
        shape = (index.shape[0], table.shape[1]) if inner is None else (index.shape[0], table.shape[1], inner)
        out = torch.empty(shape, dtype=table.dtype, device=table.device)
        uvu.embed_fwd(index, table, out, scale=scale, column=column)
        ctx.save_for_backward(index)
        ctx.scale, ctx.column, ctx.rows = scale, column, table.shape[0]
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        (index,) = ctx.saved_tensors
        dtable = torch.empty(ctx.rows, dout.shape[1], dtype=dout.dtype, device=dout.device)
        uvu.embed_bwd(index, _c(dout), dtable, scale=ctx.scale, column=ctx.column)
        return dtable, None, None, None, None


def embedding(index, table, scale: float = 1.0, inner=None, column: int = 0):
    """scale * table[index] for index [T] int32 and table [rows][C] (fp32, bf16 or f16): [T][C], or with `inner` the features
    [T][C][inner] whose `column` (that of a 0e irrep) holds the values and whose others are zero.  An index outside the table
    gives zeros and takes no gradient."""
    return _Embedding.apply(_c(table), _c(index), float(scale), None if inner is None else int(inner), int(column))


class _RmsNorm(torch.autograd.Function):
    """(x, gamma) -> y (uvu_rms_norm_fwd); backward = uvu_rms_norm_bwd."""

    @staticmethod
    def forward(ctx, x, gamma, eps):
        y = torch.empty_like(x)
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        uvu.rms_norm_fwd(x, gamma, y, rstd, eps=eps)
        ctx.save_for_backward(x, gamma, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, gamma, rstd = ctx.saved_tensors
        dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
        uvu.rms_norm_bwd(_c(dy), x, gamma, rstd, dx, dgamma)
        return dx, dgamma, None


class _AddRmsNorm(torch.autograd.Function):
    """(x, residual, gamma) -> (y, h) (uvu_rms_norm_fwd); backward = uvu_rms_norm_bwd, whose dx is both operands' gradient."""

    @staticmethod
    def forward(ctx, x, residual, gamma, eps):
        ctx.set_materialize_grads(False)
        y, h = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        uvu.rms_norm_fwd(x, gamma, y, rstd, residual=residual, h=h, eps=eps)
        ctx.save_for_backward(h, gamma, rstd)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, gamma, rstd = ctx.saved_tensors
        if dy is None:  # only the stream is used
            return dh, dh, None if dh is None else torch.zeros_like(gamma), None
        dx, dgamma = torch.empty_like(h), torch.empty_like(gamma)
        uvu.rms_norm_bwd(_c(dy), h, gamma, rstd, dx, dgamma, dh=None if dh is None else _c(dh))
        return dx, dx, dgamma, None


def rms_norm(x, gamma, residual=None, eps: float = 1e-5):
    """y = RMS norm of x [N][C] or [N][C][inner] with gamma [C] fp32, over all values of a row (the components of an irrep share
    their channel's gamma, so equivariant features stay equivariant).  With a residual, (y, h): h = x + residual is the
    stream that goes on, and y the norm of it."""
    if residual is None:
        return _RmsNorm.apply(_c(x), _c(gamma), float(eps))
    return _AddRmsNorm.apply(_c(x), _c(residual), _c(gamma), float(eps))

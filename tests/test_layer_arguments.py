"""Arguments of the embedding, RMS norm and orthogonalisation entries, checked before any launch: these tests need no GPU."""
import ctypes

import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import autograd, optim, uvu

A = 4096  # a pointer that nothing may follow
F32, F64 = uvu.UVU_F32, uvu.UVU_F64


def refused(f, *args):
    with pytest.raises(uvu.UVUError) as e:
        f(*args)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("change, status", [
    (dict(dtype=F64), 2), (dict(dtype=9), 1), (dict(tokens=-1), 1), (dict(tokens=2 ** 31 - 1), 1), (dict(rows=0), 1),
    (dict(rows=2 ** 31 - 1), 1), (dict(channels=0), 1), (dict(inner=0), 1), (dict(column=4), 1), (dict(column=-1), 1),
    (dict(channels=65536, inner=512), 1), (dict(scale=float("nan")), 1), (dict(scale=1e39), 1), (dict(index=None), 1),
    (dict(index=A + 2), 1), (dict(table=None), 1), (dict(table=A + 2), 1), (dict(out=None), 1), (dict(ws=None), 1), (dict(ws=A + 8), 1),
    (dict(size=15), 1)], ids=str)
def test_embedding(change, status):
    c = dict(dtype=F32, tokens=3, rows=7, channels=8, inner=4, column=1, scale=1.0, index=A, table=A, out=A, ws=A, size=2 ** 40) | change
    head = [c[k] for k in ("dtype", "tokens", "rows", "channels", "inner", "column", "scale", "index")]
    assert refused(uvu.uvu_embed_bwd, *head, c["out"], c["table"], c["ws"], c["size"], None)[0] == status
    if not {"ws", "size"} & set(change):
        assert refused(uvu.uvu_embed_fwd, *head, c["table"], c["out"], None)[0] == status


def test_embedding_of_no_tokens():
    uvu.uvu_embed_fwd(F32, 0, 7, 8, 1, 0, 1.0, None, None, None, None)
    b = ctypes.c_size_t(5)
    uvu.uvu_embed_workspace(F32, 0, 7, 8, 1, ctypes.byref(b))
    assert b.value == 0


@pytest.mark.parametrize("change, status", [
    (dict(dtype=F64), 2), (dict(rows=-1), 1), (dict(rows=2 ** 31 - 1), 1), (dict(channels=0), 1), (dict(channels=8193), 1),
    (dict(channels=4097, inner=2), 1), (dict(channels=65536, inner=65536), 1), (dict(eps=-1.0), 1), (dict(eps=float("inf")), 1),
    (dict(x=None), 1), (dict(x=A + 2), 1), (dict(gamma=None), 1), (dict(h=None), 1), (dict(residual=None), 1), (dict(y=None), 1)], ids=str)
def test_rms_norm(change, status):
    c = dict(dtype=F32, rows=3, channels=8, inner=4, eps=1e-5, x=A, residual=A, gamma=A, h=2 * A, y=A, rstd=A) | change
    head = [c[k] for k in ("dtype", "rows", "channels", "inner")]
    tail = [c[k] for k in ("x", "residual", "gamma", "h", "y")]
    assert refused(uvu.uvu_rms_norm_fwd, *head, c["eps"], *tail, c["rstd"], None)[0] == status
    assert refused(uvu.uvu_rms_norm_quant, *head, c["eps"], 32, *tail, A, None)[0] == status
    if not {"eps", "residual", "y"} & set(change):
        assert refused(uvu.uvu_rms_norm_bwd, *head, c["x"], c["h"], c["gamma"], A, None, A, A, A, 2 ** 40, None)[0] == status


def test_rms_norm_more():
    assert refused(uvu.uvu_rms_norm_fwd, F32, 3, 8, 1, 1e-5, A, A, A, 2 * A, 2 * A, A, None)[0] == 1  # h and y are one tensor
    assert refused(uvu.uvu_rms_norm_quant, F32, 3, 8, 1, 1e-5, -1, A, None, A, None, A, A, None)[0] == 1
    assert refused(uvu.uvu_rms_norm_quant, F32, 3, 8, 1, 1e-5, 8, A, None, A, None, A, None, None)[0] == 1  # no scales
    uvu.uvu_rms_norm_fwd(F32, 0, 8, 1, 1e-5, None, None, None, None, None, None, None)
    uvu.uvu_rms_norm_quant(F32, 0, 8, 1, 1e-5, 8, None, None, None, None, None, None, None)


def shape(**change):
    c = dict(dtype=F32, n_matrices=2, rows=8, cols=16, steps=5, reserved=0, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, scale=1.0,
             g_matrix=128, g_row=16, o_matrix=128, o_row=16) | change
    return ctypes.byref(uvu.OrthoShape(*[c[f] for f, _ in uvu.OrthoShape._fields_]))


@pytest.mark.parametrize("change, status", [
    (dict(dtype=F64), 2), (dict(n_matrices=-1), 1), (dict(n_matrices=65536), 1), (dict(rows=0), 1), (dict(cols=16385), 1), (dict(steps=-1), 1),
    (dict(steps=65), 1), (dict(reserved=1), 1), (dict(a=float("nan")), 1), (dict(c=1e39), 1), (dict(scale=float("inf")), 1), (dict(eps=-1e-9), 1),
    (dict(g_row=-1), 1), (dict(o_row=15), 1), (dict(o_matrix=0), 1), (dict(o_matrix=127), 1), (dict(o_matrix=16, o_row=31), 1)], ids=str)
def test_orthogonalize(change, status):
    assert refused(uvu.uvu_orthogonalize, shape(**change), A, A, A, 2 ** 40, None)[0] == status
    b = ctypes.c_size_t()
    assert refused(uvu.uvu_orthogonalize_workspace, shape(**change), ctypes.byref(b))[0] == status


def test_orthogonalize_more():
    assert refused(uvu.uvu_orthogonalize, None, A, A, A, 0, None)[0] == 1
    uvu.uvu_orthogonalize(shape(n_matrices=0), None, None, None, 0, None)
    b = ctypes.c_size_t()
    uvu.uvu_orthogonalize_workspace(shape(o_matrix=16, o_row=32), ctypes.byref(b))  # rows of one matrix between those of the other
    assert refused(uvu.uvu_orthogonalize, shape(), None, A, A, 2 ** 40, None)[0] == 1
    assert refused(uvu.uvu_orthogonalize, shape(), A, A + 2, A, 2 ** 40, None)[0] == 1
    assert refused(uvu.uvu_orthogonalize, shape(g_row=32, g_matrix=256), A, A, A, 2 ** 40, None)[0] == 1  # in place at other strides


def test_tensors_of_the_host():
    x, w, i, m = torch.zeros(4, 8), torch.ones(8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    q = torch.zeros(4, 8, dtype=torch.uint8)
    for f in (lambda: uvu.embed_fwd(i, x, x.clone()), lambda: uvu.embed_bwd(i, x, x.clone()), lambda: uvu.rms_norm_fwd(x, w, x.clone()),
              lambda: uvu.rms_norm_quant(x, w, q, torch.zeros(4, 1), group=0), lambda: uvu.rms_norm_bwd(x, x, w, m, x.clone(), w.clone()),
              lambda: uvu.orthogonalize(x, x.clone()), lambda: autograd.embedding(i, x), lambda: autograd.rms_norm(x, w),
              lambda: autograd.rms_norm(x, w, residual=x)):
        with pytest.raises(TypeError, match="CUDA tensors"):
            f()


def test_shapes_of_tensors(monkeypatch):
    """What the C entries cannot see: types, shapes and strides, on tensors whose device is taken as given."""
    monkeypatch.setattr(uvu, "_device", lambda t: -1)
    x, w, i = torch.zeros(4, 8), torch.ones(8), torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 8, dtype=torch.uint8)
    bad = [lambda: uvu.embed_fwd(i.long(), x, x), lambda: uvu.embed_fwd(i[:3], x, x), lambda: uvu.embed_fwd(i, x, x[:, :4]),
           lambda: uvu.embed_fwd(i, x.half(), x), lambda: uvu.embed_fwd(i, x[:, :7], torch.zeros(4, 8)),
           lambda: uvu.embed_fwd(torch.zeros(8, dtype=torch.int32)[::2], x, x), lambda: uvu.embed_fwd(i, x, torch.zeros(4, 8, 2, 1)),
           lambda: uvu.rms_norm_fwd(x.t(), torch.ones(4), x), lambda: uvu.rms_norm_fwd(x, w.half(), x),
           lambda: uvu.rms_norm_fwd(x, w, x, residual=x), lambda: uvu.rms_norm_fwd(x, w, x, h=x),
           lambda: uvu.rms_norm_fwd(x, w, x, torch.zeros(3)), lambda: uvu.rms_norm_fwd(x, w, x.half()),
           lambda: uvu.rms_norm_quant(x, w, x, torch.zeros(4, 1)), lambda: uvu.rms_norm_quant(x, w, q, torch.zeros(4, 2), group=8),
           lambda: uvu.rms_norm_quant(x, w, q, torch.zeros(4, 1), group=-1), lambda: uvu.rms_norm_quant(x, w, q[:, :7], torch.zeros(4, 1)),
           lambda: uvu.rms_norm_bwd(x, x, w, torch.zeros(4), x, w, dh=x[:2]), lambda: uvu.orthogonalize(x.t(), x.t()),
           lambda: uvu.orthogonalize(x, x.half()), lambda: uvu.orthogonalize(x, x[:2]), lambda: uvu.orthogonalize(x[0], x[0])]
    for f in bad:
        with pytest.raises((TypeError, ValueError)):
            f()


def test_strides_of_matrices():
    t = torch.zeros(3, 5, 40)
    assert uvu._matrices("g", t) == (3, 5, 40, 200, 40)
    assert uvu._matrices("g", t[:, :, 8:20]) == (3, 5, 12, 200, 40)
    assert uvu._matrices("g", t[::2, ::2]) == (2, 3, 40, 400, 80)
    assert uvu._matrices("g", t[0]) == (1, 5, 40, 0, 40)
    assert uvu._matrices("g", t[:1, :1]) == (1, 1, 40, 0, 40)


def test_muon_takes_matrices():
    with pytest.raises(ValueError, match="matrices"):
        optim.Muon([torch.zeros(3, requires_grad=True)])
    for bad in (dict(lr=-1.0), dict(momentum=1.0), dict(weight_decay=-1.0)):
        with pytest.raises(ValueError):
            optim.Muon([torch.zeros(3, 3, requires_grad=True)], **bad)

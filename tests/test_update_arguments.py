"""Arguments of the node-update operators, checked before any launch: these tests need no GPU."""
import ctypes
import types

import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import autograd, uvu

A = 4096  # a pointer that nothing may follow


def refused(f, *args):
    with pytest.raises(uvu.UVUError) as e:
        f(*args)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("missing", ["gamma", "beta"])
@pytest.mark.parametrize("rows", [0, 3])
def test_group_norm_without_parameters(missing, rows):
    """The kernel reads gamma and beta for an empty batch too."""
    gamma, beta = (None if missing == n else A for n in ("gamma", "beta"))
    status, text = refused(uvu.uvu_group_norm_fwd, uvu.UVU_F32, rows, 1, rows, 8, 2, 0, 1e-5, A, A, gamma, beta, A, A, A, None, 0, None)
    assert status == 1 and f"{missing} is NULL" in text


def test_tensors_of_the_host():
    """Tensors that agree with one another but lie in host memory."""
    x, w, off = torch.zeros(4, 8), torch.ones(8), torch.tensor([0, 4], dtype=torch.int32)
    m, q, lse = torch.zeros(1, 2), torch.zeros(4, 2, 8), torch.zeros(4, 2)
    for f in (lambda: uvu.group_norm_fwd(x, w, w, off, 2, x.clone(), m, m.clone()),
              lambda: uvu.group_norm_bwd(x, x, w, w, off, 2, m, m, x.clone(), w.clone(), w.clone()),
              lambda: uvu.dropout_fwd(x, 0.1, 1, x.clone()),
              lambda: uvu.dropout_bwd(x, 0.1, 1, x.clone()),
              lambda: uvu.Attention(2, 2, 8, off, off).fwd(q, q, q, q.clone(), lse),
              lambda: autograd.group_norm(x, w, w, off, 2),
              lambda: autograd.dropout(x, 0.1, 1)):
        with pytest.raises(TypeError, match="CUDA tensors"):
            f()


def test_tensors_of_another_device(monkeypatch):
    """The kernels are launched on the current device."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    there = types.SimpleNamespace(get_device=lambda: 1)
    with pytest.raises(ValueError, match="device 1"):
        uvu._device(there)
    here = types.SimpleNamespace(get_device=lambda: 0)
    assert uvu._device(here) == 0


def test_workspace_of_the_caller():
    """A workspace in host memory, and one whose bytes are not all its own."""
    host = torch.empty(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace"):
        uvu._scratch(64, host, 0)
    with pytest.raises(ValueError, match="workspace"):
        uvu._scratch(64, host[:1].expand(64), -1)
    assert uvu._scratch(64, host, -1)[:2] == (host.data_ptr(), 64)


@pytest.mark.parametrize("nq, nk, dq, dkv", [(0, 5, A, None), (5, 0, None, A), (0, 0, A, A), (0, 5, None, None)])
def test_gradients_without_values(nq, nk, dq, dkv):
    """Only gradients of no rows or no states are asked for, with pointers that are not NULL: nothing is launched."""
    s = uvu.AttnShape(uvu.UVU_F32, 1, nq, nk, nq, nk, 1, 1, 8, 0, 1.0, 8, 8, 8, 8, 8, 8, 8, 8)
    uvu.uvu_attn_bwd(ctypes.byref(s), *[A] * 9, dq, dkv, dkv, None, 0, None)


@pytest.mark.parametrize("rows, heads", [(5, 1), (1, 5), (1, 1), (5, 3), (0, 3)])
def test_strides_of_axes_of_one(rows, heads):
    """A tensor and its transpose of transpose are the same operand; torch calls both contiguous."""
    at = object.__new__(uvu.Attention)
    at.device, at.head_dim = -1, 8
    plain, turned = torch.zeros(rows, heads, 8), torch.zeros(heads, rows, 8).transpose(0, 1)
    if min(rows, heads) < 2:
        assert turned.is_contiguous() and at._operand("d_out", turned, heads, rows, plain.dtype) == \
            at._operand("out", plain, heads, rows, plain.dtype)
    else:
        assert at._operand("out", plain, heads, rows, plain.dtype) == (24, 8)
        assert at._operand("out", turned, heads, rows, plain.dtype) == (8, 40)


def test_inner_beyond_an_int():
    """2^32 + 1 would arrive in the library as 1."""
    for inner in (2 ** 31, 2 ** 32 + 1):
        with pytest.raises(ValueError, match="inner"):
            uvu._draws(torch.empty(2 * inner, device="meta"), inner)
    assert uvu._draws(torch.empty(2 ** 32 - 2, device="meta"), 2 ** 31 - 1) == 2

"""Calls of the node-update operators at the edges of their contracts: unusual strides, empty batches, rows whose mask leaves
nothing, small cotangents, and the kernels that only large batches choose."""
import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import autograd, uvu

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


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

"""Workspaces that the wrappers allocate themselves come from the pool of the stream that the kernels run on: a block of
another stream's pool could be handed out again, on the wrapper's return, while the kernels still use it."""
import contextlib
import types

import numpy as np
import pytest
import torch

from clebsch_gordan_tensor_receiver_gb300 import uvu

SIDE = types.SimpleNamespace(cuda_stream=0x10)


@pytest.fixture
def pools(monkeypatch):
    """The streams under which uint8 tensors were allocated; launches are left out."""
    seen, inside = [], []

    @contextlib.contextmanager
    def stream(s):
        inside.append(s)
        yield
        inside.pop()

    real = torch.empty

    def empty(*shape, **kw):
        if kw.get("dtype") == torch.uint8:
            seen.append(inside[-1] if inside else None)
        return real(*shape, **kw)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", empty)
    for name in ("uvu_radial_weights", "uvu_radial_weights_bwd", "uvu_radial_hidden_bwd", "uvu_tp_bwd", "uvu_mix_fwd", "uvu_mix_bwd",
                 "uvu_conv_uvw_fwd", "uvu_conv_bwd", "uvu_conv_hvp", "uvu_csr_from_sorted_recv", "uvu_csr_transpose",
                 "uvu_csr_transpose_workspace"):
        monkeypatch.setattr(uvu, name, lambda *a: None)
    # the size queries that would ask a device
    for name in ("radial_weights_workspace", "radial_weights_bwd_workspace", "radial_hidden_bwd_workspace", "tp_workspace_bytes",
                 "workspace_bytes"):
        monkeypatch.setattr(uvu.Plan, name, lambda self, *a: 64)
    monkeypatch.setattr(uvu.Plan, "mix_workspace_bytes", lambda self, *a: (64, 64))

    def hvp_bytes(plan, n, e, b):
        b._obj.value = 64

    monkeypatch.setattr(uvu, "uvu_conv_hvp_workspace", hvp_bytes)
    return seen


def calls():
    plan = uvu.Plan("16x0e+16x1o", "1x0e+1x1o", 1)
    f, i = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int32)
    return {
        "radial_weights": lambda s: plan.radial_weights(f, f, f, stream=s),
        "radial_weights_bwd": lambda s: plan.radial_weights_bwd(f, f, f, stream=s),
        "radial_hidden_bwd": lambda s: plan.radial_hidden_bwd(f, 5.0, 5, [4, 16], f, f, f, f, stream=s),
        "tp_bwd": lambda s: plan.tp_bwd(4, f, f, f, f, dw=f, w_shared=True, stream=s),
        "mix_fwd": lambda s: plan.mix_fwd(4, 16, f, f, f, stream=s),
        "mix_bwd": lambda s: plan.mix_bwd(4, 16, f, f, f, stream=s),
        "uvw_fwd": lambda s: plan.uvw_fwd(4, f, f, f, i, i, f, 16, f, f, stream=s),
        "bwd": lambda s: plan.bwd(4, f, f, f, i, i, i, i, i, f, dx=f, dx_mode=uvu.UVU_DX_STAGED, stream=s),
        "hvp": lambda s: plan.hvp(4, f, f, f, i, i, i, i, f, grad_x=f, stream=s),
        "Graph": lambda s: uvu.Graph(4, i, i, stream=s),
        "scratch": lambda s: uvu._scratch(64, None, "cpu", s),
    }


@pytest.mark.parametrize("name", ["radial_weights", "radial_weights_bwd", "radial_hidden_bwd", "tp_bwd", "mix_fwd", "mix_bwd", "uvw_fwd",
                                  "bwd", "hvp", "Graph", "scratch"])
def test_workspace_of_the_stream(pools, name):
    calls()[name](SIDE)
    assert pools == [SIDE], name


@pytest.mark.gpu
def test_memory_is_not_reused_under_the_kernels():
    """Group norm and attention on `stream=`, which is busy, while the current stream takes and overwrites blocks of the same
    sizes: the results are those of the current stream."""
    rng = np.random.default_rng(4)
    dev = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    off, k_off = (torch.tensor(o, dtype=torch.int32, device="cuda") for o in ([0, 90, 400], [0, 700, 1000]))
    x, dy, gamma, beta = dev(400, 128), dev(400, 128), dev(128), dev(128)
    q, k, v, do = dev(400, 4, 32), dev(1000, 2, 32), dev(1000, 2, 32), dev(400, 4, 32)
    at = uvu.Attention(4, 2, 32, off, k_off, 310, 700)

    def outputs():
        e = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        return [e(400, 128), e(2, 8), e(2, 8), e(400, 128), e(128), e(128), e(400, 4, 32), e(400, 4), e(400, 4, 32), e(1000, 2, 32),
                e(1000, 2, 32)]

    def step(o, **kw):
        uvu.group_norm_fwd(x, gamma, beta, off, 8, *o[:3], **kw)
        uvu.group_norm_bwd(dy, x, gamma, beta, off, 8, o[1], o[2], *o[3:6], **kw)
        at.fwd(q, k, v, o[6], o[7], **kw)
        at.bwd(q, k, v, o[6], o[7], do, *o[8:], **kw)

    want, got = outputs(), outputs()
    step(want)
    sizes = [*uvu.group_norm_workspace_bytes(x, 2, 8), *at.workspace_bytes(q, k)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    step(got, stream=side)
    held = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4) if n]
    torch.cuda.synchronize()
    assert held and all(torch.equal(a, b) for a, b in zip(got, want))

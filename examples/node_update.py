"""A convolution and a node update trained together: molecules whose atoms attend to an encoder's states.

Every molecule has its own atoms (a packed batch, offsets) and its own context states (a pocket's residues, a prompt's
tokens).  One layer convolves the atoms' features over the edges within the molecule, normalises the invariant channels,
lets them attend to the molecule's states, and drops channels out; a readout of the sum over atoms is fitted to random
targets.  All operators and their gradients are the library's; the dense products and the optimiser are PyTorch's.

    python examples/node_update.py [--molecules 64] [--steps 200]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from clebsch_gordan_tensor_receiver_gb300 import autograd, uvu, workloads  # noqa: E402

CHANNELS, STATE = 64, 48
HEADS, KV_HEADS, HEAD_DIM, GROUPS = 4, 2, 16, 8


def molecules(n, rng):
    """Node offsets, context offsets, and edges (receiver-sorted): 5 to 40 atoms, 0 to 60 states, 4 neighbours an atom."""
    atoms, states = rng.integers(5, 41, size=n), rng.integers(0, 61, size=n)
    node_off, state_off = (np.concatenate([[0], np.cumsum(c)]).astype(np.int32) for c in (atoms, states))
    recv = np.repeat(np.arange(node_off[-1]), 4)
    graph = np.repeat(np.repeat(np.arange(n), atoms), 4)
    src = node_off[graph] + rng.integers(0, atoms[graph])
    return node_off, state_off, recv.astype(np.int32), src.astype(np.int32)


def train(n_molecules=64, steps=200, p=0.1, seed=0, device="cuda"):
    """The losses of the first and the last step."""
    rng = np.random.default_rng(seed)
    node_off, state_off, recv, src = molecules(n_molecules, rng)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    f32 = lambda *shape: dev(rng.standard_normal(shape).astype(np.float32))  # noqa: E731
    nodes, states, edges = int(node_off[-1]), int(state_off[-1]), src.size

    plan = uvu.Plan(f"{CHANNELS}x0e+{CHANNELS}x1o", "1x0e+1x1o+1x2e", 2)
    graph = uvu.Graph(nodes, dev(recv), dev(src))
    Y = dev(workloads.sh_inputs(workloads.unit_vectors(edges, rng), 2).astype(np.float32))
    x, context = f32(nodes, CHANNELS, plan.info.dim_x), f32(states, STATE)
    off, s_off = dev(node_off), dev(state_off)
    longest = lambda o: int(np.diff(o).max())  # noqa: E731
    attention = uvu.Attention(HEADS, KV_HEADS, HEAD_DIM, off, s_off, max_q=longest(node_off), max_k=longest(state_off))
    keep = dev(rng.random(states) < 0.9)  # padding that an encoder left in its states
    target = f32(n_molecules)

    scaled = lambda a, b: (f32(a, b) * a ** -0.5)  # noqa: E731
    weights = [torch.ones(CHANNELS, device=device), torch.zeros(CHANNELS, device=device), scaled(CHANNELS, HEADS * HEAD_DIM),
               scaled(STATE, KV_HEADS * HEAD_DIM), scaled(STATE, KV_HEADS * HEAD_DIM), scaled(HEADS * HEAD_DIM, CHANNELS)]
    w_edge = f32(edges, plan.info.n_paths, CHANNELS) * 0.5
    read = scaled(CHANNELS, 1)
    params = [*weights, w_edge, read]
    for t in params:
        t.requires_grad_(True)
    opt = torch.optim.Adam(params, lr=1e-2)
    which = dev(np.repeat(np.arange(n_molecules), np.diff(node_off)))
    draws = 2 * ((nodes * CHANNELS + 7) // 8)  # offsets that a step uses

    losses = []
    for step in range(steps):
        m = autograd.uvu_conv(x, Y, w_edge, plan, graph)
        s, h = autograd.node_update(m, off, context, attention, weights, GROUPS, p=p, seed=seed, offset=step * draws,
                                    keep=keep, max_rows=longest(node_off))
        # invariants: the scalars and the norms of the gated channels
        atom = (s + h.square().sum(2).add(1e-6).sqrt()) @ read
        energy = torch.zeros(n_molecules, device=device).index_add(0, which, atom[:, 0])
        loss = (energy - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    first, last = float(losses[0]), float(losses[-1])
    if uvu.Attention.device_status() or plan.device_status():
        raise RuntimeError("a kernel gave up a wait")
    return first, last


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--molecules", type=int, default=64)
    a.add_argument("--steps", type=int, default=200)
    a = a.parse_args()
    first, last = train(a.molecules, a.steps)
    print(f"loss {first:.4f} -> {last:.4f} in {a.steps} steps")

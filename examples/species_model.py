"""A layer trained from species on: an embedding, a convolution, an RMS norm of the residual stream, and Muon.

The atoms' first features 64x0e+64x1o are a table's rows by species (the scalars; the vectors begin at zero).  One layer
convolves them over the molecules' edges, mixes the result back to the features' size, adds it to the stream and normalises; a
readout of the invariants, summed over a molecule's atoms, is fitted to random targets.  The dense products are PyTorch's,
everything else the library's.  Matrices are updated by Muon, the table, the norm and the radial weights by Adam.

    python examples/species_model.py [--molecules 64] [--steps 100]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from clebsch_gordan_tensor_receiver_gb300 import autograd, optim, uvu, workloads  # noqa: E402

CHANNELS, SPECIES = 64, 10


def train(n_molecules=64, steps=100, seed=0, device="cuda"):
    """The losses of the steps, and the parameters."""
    rng = np.random.default_rng(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    f32 = lambda *shape: dev(rng.standard_normal(shape).astype(np.float32))  # noqa: E731
    atoms = rng.integers(5, 41, size=n_molecules)
    first, nodes = np.concatenate([[0], np.cumsum(atoms)]), int(atoms.sum())
    molecule = np.repeat(np.arange(n_molecules), atoms)
    recv = np.repeat(np.arange(nodes), 4)
    src = first[molecule[recv]] + rng.integers(0, atoms[molecule[recv]])
    edges = src.size

    plan = uvu.Plan(f"{CHANNELS}x0e+{CHANNELS}x1o", "1x0e+1x1o", 1)
    graph = uvu.Graph(nodes, dev(recv.astype(np.int32)), dev(src.astype(np.int32)))
    Y = dev(workloads.sh_inputs(workloads.unit_vectors(edges, rng), 1).astype(np.float32))
    species = dev(rng.integers(0, SPECIES, size=nodes).astype(np.int32))
    # the paths that give 0e and 1o again, and where their components lie in a row of the convolution's output
    outs, at = {0: [], 1: []}, 0
    for l1, l2, l3 in plan.info.paths:
        if l3 <= 1 and (l1 + l2 + l3) % 2 == 0:
            outs[l3].append(at)
        at += 2 * l3 + 1

    table = f32(SPECIES, CHANNELS)
    gamma = torch.ones(CHANNELS, device=device)
    w_edge = f32(edges, plan.info.n_paths, CHANNELS) * 0.5
    mixers = {k: f32(len(v), CHANNELS, CHANNELS) * CHANNELS ** -0.5 for k, v in outs.items()}
    read = f32(CHANNELS, CHANNELS) * CHANNELS ** -0.5
    adam, muon = [table, gamma, w_edge], [*mixers.values(), read]
    for t in adam + muon:
        t.requires_grad_(True)
    optimisers = [torch.optim.Adam(adam, lr=1e-2), optim.Muon(muon, lr=1e-2)]
    which, target = dev(molecule), f32(n_molecules)

    losses = []
    for _ in range(steps):
        x = autograd.embedding(species, table, scale=CHANNELS ** -0.5, inner=plan.info.dim_x)
        m = autograd.uvu_conv(x, Y, w_edge, plan, graph)
        new = []
        for l, cols in outs.items():  # [N][U][paths][2l+1] by [paths][U][W]
            part = torch.stack([m[:, :, i:i + 2 * l + 1] for i in cols], 2)
            new.append(torch.einsum("nupd,puw->nwd", part, mixers[l]))
        y, stream = autograd.rms_norm(torch.cat(new, 2), gamma, residual=x)
        inv = y[:, :, 0] + y[:, :, 1:].square().sum(2)
        atom = (torch.tanh(inv @ read) + stream[:, :, 0]).mean(1)
        energy = torch.zeros(n_molecules, device=device).index_add(0, which, atom)
        loss = (energy - target).square().mean()
        for o in optimisers:
            o.zero_grad()
        loss.backward()
        for o in optimisers:
            o.step()
        losses.append(loss.detach())
    if plan.device_status():
        raise RuntimeError("a kernel gave up a wait")
    return torch.stack(losses).tolist(), adam + muon


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--molecules", type=int, default=64)
    a.add_argument("--steps", type=int, default=100)
    a = a.parse_args()
    losses, _ = train(a.molecules, a.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

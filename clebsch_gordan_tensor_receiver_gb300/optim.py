"""The Muon optimiser (Jordan, "Muon: an optimizer for hidden layers in neural networks", 2024) for the weight matrices of a
model: mixing matrices [P][U][W], last radial layers, dense layers.  Its orthogonalised updates run in the library
(uvu_orthogonalize); the momentum and the weights' own update are elementwise in PyTorch.
"""

from __future__ import annotations

import torch

from . import uvu


MOST = 65535  # matrices of one call


class Muon(torch.optim.Optimizer):
    """Momentum, then W <- (1 - lr weight_decay) W - lr max(1, rows / cols)^(1/2) O, with O the momentum (looked ahead where
    `nesterov`) made nearly orthogonal, matrix by matrix.  Parameters are [rows][cols] or batches [matrices][rows][cols]; those of
    one type and size are made orthogonal in one call.  Other parameters (tables, norms' gamma, biases) belong to another
    optimiser.

    The momentum and the update are fp32 for 16-bit parameters too: a 16-bit average takes no step of less than half its
    own (with momentum 0.95 and bf16, a gradient within 8% of it changes nothing).  The parameter itself rounds once for the decay and once for the update."""

    def __init__(self, params, lr: float = 0.02, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
                 steps: int = 5, coefficients=uvu.MUON, eps: float = 1e-7):
        if lr < 0 or not 0 <= momentum < 1 or weight_decay < 0:
            raise ValueError("lr and weight_decay must be >= 0 and momentum in [0, 1)")
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov, weight_decay=weight_decay, steps=steps,
                                      coefficients=tuple(coefficients), eps=eps))

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        for p in self.param_groups[-1]["params"]:
            if p.dim() not in (2, 3):
                self.param_groups.pop()
                raise ValueError(f"Muon takes matrices or batches of matrices, not a parameter of shape {tuple(p.shape)}")

    def load_state_dict(self, state_dict):
        """As PyTorch's, which casts what it loads to the parameter's type; the momentum stays in fp32."""
        super().load_state_dict(state_dict)
        numbers = (i for group in state_dict["param_groups"] for i in group["params"])
        for i, p in zip(numbers, (p for group in self.param_groups for p in group["params"])):
            buf = state_dict["state"].get(i, {}).get("momentum")
            if buf is not None:
                self.state[p]["momentum"] = buf.to(p.device, torch.float32, copy=True)

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            alike = {}  # parameters whose updates go through one call
            for p in group["params"]:
                if p.grad is None or p.numel() == 0:
                    continue
                alike.setdefault((p.shape[-2:], p.dtype, p.device), []).append(p)
            for (size, _, _), params in alike.items():
                self._update(group, size, params)
        return loss

    def _update(self, group, size, params):
        m = group["momentum"]
        updates = []
        for p in params:
            state = self.state[p]
            if "momentum" not in state:
                state["momentum"] = torch.zeros_like(p, dtype=torch.float32, memory_format=torch.contiguous_format)
            buf = state["momentum"]
            grad = p.grad.float()
            buf.lerp_(grad, 1 - m)
            updates.append((grad.lerp(buf, m) if group["nesterov"] else buf).reshape(-1, *size))
        u = torch.cat(updates)
        with torch.cuda.device(u.device):
            for part in u.split(MOST):
                uvu.orthogonalize(part, part, steps=group["steps"], coefficients=group["coefficients"], eps=group["eps"])
        rate = -group["lr"] * max(1.0, size[0] / size[1]) ** 0.5
        at = 0
        for p, part in zip(params, updates):
            n = part.shape[0]
            p.mul_(1 - group["lr"] * group["weight_decay"])
            p.add_(u[at:at + n].view(p.shape), alpha=rate)
            at += n

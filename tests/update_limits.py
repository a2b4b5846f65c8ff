"""Limits of the relative Frobenius error of the attention's 16-bit results, shared by the GPU tests and by the CPU test that
shows what they let through."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def values(t):
    return t.double().cpu().numpy()


def relative(got, ref):
    got = values(got) if isinstance(got, torch.Tensor) else got
    return float(np.linalg.norm(got - ref) / np.linalg.norm(ref))


def own_rounding(ref, dtype):
    t = torch.from_numpy(np.ascontiguousarray(ref))
    return float((t.to(dtype).double() - t).norm() / t.norm())


def unit(dtype):
    return 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8


def output_limit(ref, dtype):
    """Of out.  The result's own rounding, e0, is taken from the exact values (below a type's smallest normal number it is more than
    u).  P is rounded to the type for the product: u = 2^-p at most for each term, some 0.4 u in the norm of a sum.  Together at
    most 1.25 e0 + u, with room for fp32's 2^-20."""
    return 1.25 * own_rounding(ref, dtype) + unit(dtype)


def gradient_limit(ref, dtype):
    """Of dq, dk and dv: as out, and delta from the rounded output shifts a row's dS by at most another u |do| |out| P."""
    return 1.25 * own_rounding(ref, dtype) + 2 * unit(dtype)

"""What the limits of tests/update_limits.py let through, on the CPU: the roundings that 16-bit attention makes pass, a lost term
or a wrong factor does not."""
import numpy as np
import pytest
import torch

from oracle import update
from update_limits import TYPES, gradient_limit, output_limit, relative


def rounded(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).double().numpy()


def problem(dtype, nq, nk, d):
    rng = np.random.default_rng(nq + nk + d)
    q, k, v, do = (rounded(rng.standard_normal((n, 1, d)), dtype) for n in (nq, nk, nk, nq))
    return q, k, rounded(v + 0.25, dtype), do, [0, nq], [0, nk], d ** -0.5


def steps(q, k, v, do, scale, dtype=None, delta=True):
    """out, dq, dk, dv, with P, dS, delta and the results rounded as the kernels do where a type is given."""
    r = (lambda a: a) if dtype is None else (lambda a: rounded(a, dtype))
    q, k, v, do = (t[:, 0] for t in (q, k, v, do))
    s = scale * q @ k.T
    p = np.exp(s - s.max(1, keepdims=True))
    total = p.sum(1, keepdims=True)
    out = r(r(p) @ v / total)
    p /= total
    ds = p * (do @ v.T - (do * out).sum(1, keepdims=True) * delta)
    shift = 2.0 ** 16  # f16 holds both at a scale
    return [t[:, None] for t in (out, r(r(ds * shift) @ k * scale / shift), r(r(ds * shift).T @ q * scale / shift),
                                 r(r(p * 256).T @ do / 256))]


SIZES = [(200, 900, 64), (40, 2900, 128), (600, 600, 16)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("nq, nk, d", SIZES)
def test_limits(nq, nk, d, kind):
    dtype = TYPES[kind]
    q, k, v, do, qo, ko, scale = problem(dtype, nq, nk, d)
    out = update.attention(q, k, v, qo, ko, scale)[0]
    ref = [out, *update.attention_vjp(q, k, v, qo, ko, scale, do)[0]]
    limits = [output_limit(out, dtype)] + [gradient_limit(r, dtype) for r in ref[1:]]
    for a, r in zip(steps(q, k, v, do, scale), ref):
        assert relative(a, r) < 1e-12
    # the kernels' roundings have room, a factor that is a twentieth off has not
    for a, r, most in zip(steps(q, k, v, do, scale, dtype), ref, limits):
        assert relative(a, r) <= 0.8 * most
        for wrong in (a * 1.05, a * 0.95, 0 * a):
            assert relative(wrong, r) > most
    # without delta, dq and dk are wrong
    _, dq, dk, _ = steps(q, k, v, do, scale, dtype, delta=False)
    assert relative(dq, ref[1]) > 3 * limits[1] and relative(dk, ref[2]) > 3 * limits[2]
    # a twentieth of the states lost
    few = slice(0, nk - nk // 20)
    lost = steps(q, k[few], v[few], do, scale, dtype)
    assert relative(lost[0], ref[0]) > limits[0] and relative(lost[1], ref[1]) > limits[1]

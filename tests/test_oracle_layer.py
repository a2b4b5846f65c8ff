"""Pins of oracle.layer: gradients against differences, closed forms, invariances.  No GPU."""
import numpy as np
import pytest

from oracle import layer

MUON = (3.4445, -4.7750, 2.0315)


def test_embed_is_a_product_with_zeros_and_ones():
    rng = np.random.default_rng(1)
    index, table = np.array([2, 0, 2, -1, 5, 1]), rng.standard_normal((5, 3))
    pick = (index[:, None] == np.arange(5)).astype(float)
    out = layer.embed(index, table, 0.5, 4, 2)
    np.testing.assert_allclose(out[:, :, 2], 0.5 * pick @ table)
    assert not out[:, :, [0, 1, 3]].any()
    dout = rng.standard_normal(out.shape)
    d, size, count = layer.embed_vjp(index, dout, 5, 0.5, 2)
    np.testing.assert_allclose(d, 0.5 * pick.T @ dout[:, :, 2])
    np.testing.assert_allclose((d * table).sum(), (out * dout).sum())  # the adjoint
    assert list(count) == [1, 1, 2, 0, 0] and (size >= np.abs(d)).all()


def test_rms_norm_gradient_by_differences():
    rng = np.random.default_rng(2)
    h, gamma, dy, dh = (rng.standard_normal(s) for s in ((4, 3, 2), 3, (4, 3, 2), (4, 3, 2)))
    dx, dg = layer.rms_norm_vjp(h, gamma, 1e-3, dy, dh)
    f = lambda h, g: (layer.rms_norm(h, g, 1e-3)[0] * dy).sum() + (h * dh).sum()  # noqa: E731
    step = 1e-6
    for at in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[at] = step
        assert abs((f(h + e, gamma) - f(h - e, gamma)) / (2 * step) - dx[at]) < 1e-7
    for c in range(3):
        e = np.zeros(3)
        e[c] = step
        assert abs((f(h, gamma + e) - f(h, gamma - e)) / (2 * step) - dg[c]) < 1e-7


def test_rms_norm_of_a_row():
    y, rstd = layer.rms_norm(np.array([[[3.0], [4.0]]]), np.array([1.0, 2.0]), 0.0)
    np.testing.assert_allclose(rstd, 1 / np.sqrt(12.5))
    np.testing.assert_allclose(y[0, :, 0], np.array([3.0, 8.0]) / np.sqrt(12.5))


def test_e4m3_steps():
    for v, step in ((448.0, 32), (256.0, 32), (255.0, 16), (1.0, 0.125), (0.99, 0.0625), (2.0 ** -6, 2.0 ** -9), (0.0, 2.0 ** -9)):
        assert layer.e4m3_step(np.array(v)) == step


@pytest.mark.parametrize("shape", [(6, 6), (4, 9), (9, 4), (1, 5), (5, 1)])
def test_newton_schulz_acts_on_the_singular_values(shape):
    """Odd polynomials of X: the singular vectors stay, each singular value goes through a s + b s^3 + c s^5."""
    rng = np.random.default_rng(3)
    g = rng.standard_normal(shape)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    for x in layer.newton_schulz(g, 5, MUON, 1e-7):
        np.testing.assert_allclose(x, u * s @ v, atol=1e-12)
        s = MUON[0] * s + MUON[1] * s ** 3 + MUON[2] * s ** 5
    assert ((s > 0.3) & (s < 1.7)).all()  # wide: 0.05 and more of the largest value ends there

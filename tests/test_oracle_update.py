"""Pins of the node-update oracle: gradients against central differences, softmax and normalisation
identities, and the generator against its published answers."""
import numpy as np
import pytest

from oracle import update


def differences(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += step
        b[i] -= step
        g[i] = (f(a) - f(b)) / (2 * step)
    return g


@pytest.mark.parametrize("silu", [True, False])
def test_group_norm_gradients_against_differences(silu):
    rng = np.random.default_rng(3)
    off, groups, eps = np.array([0, 3, 3, 7]), 2, 1e-5
    x, dy = rng.standard_normal((7, 6)), rng.standard_normal((7, 6))
    gamma, beta = 1 + 0.3 * rng.standard_normal(6), 0.3 * rng.standard_normal(6)
    got = update.group_norm_vjp(x, gamma, beta, off, groups, silu, eps, dy)
    f = lambda a, b, c: (dy * update.group_norm(a, b, c, off, groups, silu, eps)[0]).sum()  # noqa: E731
    want = (differences(lambda t: f(t, gamma, beta), x), differences(lambda t: f(x, t, beta), gamma),
            differences(lambda t: f(x, gamma, t), beta))
    for a, b in zip(got, want):
        np.testing.assert_allclose(a, b, rtol=0, atol=2e-8 * (1 + np.abs(b).max()))


def test_group_norm_normalises():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((11, 8)) * 3 + 5
    y, _, _ = update.group_norm(x, np.ones(8), np.zeros(8), [0, 5, 11], 2, False, 0.0)
    for a, b in ((0, 5), (5, 11)):
        for g in range(2):
            part = y[a:b, 4 * g:4 * g + 4]
            assert abs(part.mean()) < 1e-14 and abs((part ** 2).mean() - 1) < 1e-13


def test_attention_gradients_against_differences():
    rng = np.random.default_rng(5)
    qo, ko = np.array([0, 2, 2, 5]), np.array([0, 3, 4, 8])
    q, k, v = rng.standard_normal((5, 4, 3)), rng.standard_normal((8, 2, 3)), rng.standard_normal((8, 2, 3))
    do = rng.standard_normal((5, 4, 3))
    keep = np.array([1, 0, 1, 1, 1, 1, 0, 1])
    (dq, dk, dv), _ = update.attention_vjp(q, k, v, qo, ko, 0.7, do, keep)
    f = lambda a, b, c: (do * update.attention(a, b, c, qo, ko, 0.7, keep)[0]).sum()  # noqa: E731
    for got, want in ((dq, differences(lambda t: f(t, k, v), q)), (dk, differences(lambda t: f(q, t, v), k)),
                      (dv, differences(lambda t: f(q, k, t), v))):
        np.testing.assert_allclose(got, want, rtol=0, atol=2e-8)


def test_attention_of_empty_rows():
    rng = np.random.default_rng(6)
    q, k = rng.standard_normal((4, 1, 2)), rng.standard_normal((3, 1, 2))
    out, lse, _ = update.attention(q, k, k, [0, 2, 4], [0, 0, 3], 1.0, np.zeros(3))
    assert not out.any() and np.isneginf(lse).all()
    grads, _ = update.attention_vjp(q, k, k, [0, 2, 4], [0, 0, 3], 1.0, np.ones_like(q), np.zeros(3))
    assert not any(g.any() for g in grads)


def test_philox_published_answers():
    # the known-answer vectors that the generator's authors publish with it (philox4x32, 10 rounds)
    full = 0xFFFFFFFF
    assert update.philox_words([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert update.philox_words([full] * 4, [full] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    pi = [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]
    assert update.philox_words(pi, [0xA4093822, 0x299F31D0]) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_keep_mask_rate():
    keep, scale = update.keep_mask(20000, 0.25, 9, 0)
    assert scale == 65536 / 49152
    assert abs(keep.mean() - 0.75) < 5 * (0.25 * 0.75 / 20000) ** 0.5

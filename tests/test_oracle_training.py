"""Pins of the float64 oracle for the gated delta rule with one decay per head and for the
backward passes of the prologue and of the output epilogue: gradients against central
differences of the forward oracle, and the rule itself against a recurrence written out here."""
import numpy as np
import pytest

from oracle import (gdr_recurrent, gdr_recurrent_backward, output_epilogue,
                    output_epilogue_backward, prologue, prologue_backward)


def central(f, x, h=1e-5):
    """d f / d x by central differences, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * h)
    return g


# The truncation error is h^2 f''' / 6 and the rounding one about 1e-16 |f| / h: with h = 1e-5
# and values of order 1 to 100 both stay under 1e-8.
ATOL = 2e-7


def test_gdr_recurrent_is_the_recurrence():
    r = np.random.default_rng(0)
    T, HK, HV, D = 9, 2, 4, 3
    q, k = r.normal(size=(T, HK, D)), r.normal(size=(T, HK, D))
    v, g, beta = r.normal(size=(T, HV, D)), -r.random((T, HV)), r.random((T, HV))
    s0 = r.normal(size=(2, HV, D, D))
    cu = [0, 4, 9]
    o, last = gdr_recurrent(q, k, v, g, beta, 0.7, s0, cu)
    for n in range(2):
        for h in range(HV):
            S = s0[n, h].copy()
            for t in range(cu[n], cu[n + 1]):
                kt, qt = k[t, h // 2], q[t, h // 2]
                S *= np.exp(g[t, h])
                S += beta[t, h] * np.outer(kt, v[t, h] - S.T @ kt)
                np.testing.assert_allclose(o[t, h], 0.7 * S.T @ qt, atol=1e-13)
            np.testing.assert_allclose(last[n, h], S, atol=1e-13)


def test_gdr_recurrent_backward_is_the_gradient():
    r = np.random.default_rng(1)
    T, HK, HV, D = 6, 1, 2, 3
    q, k = r.normal(size=(T, HK, D)), 0.5 * r.normal(size=(T, HK, D))
    v, g, beta = r.normal(size=(T, HV, D)), -r.random((T, HV)), r.random((T, HV))
    s0 = r.normal(size=(2, HV, D, D))
    cu = [0, 1, 6]
    do, dsN = r.normal(size=(T, HV, D)), r.normal(size=s0.shape)

    def loss():
        o, last = gdr_recurrent(q, k, v, g, beta, 0.7, s0, cu)
        return np.sum(do * o) + np.sum(dsN * last)

    got = gdr_recurrent_backward(q, k, v, g, beta, do, dsN, 0.7, s0, cu)
    for x, grad in zip((q, k, v, g, beta, s0), got):
        np.testing.assert_allclose(grad, central(loss, x), atol=ATOL)


@pytest.mark.parametrize("cache", [False, True])
def test_prologue_backward_is_the_gradient(cache):
    r = np.random.default_rng(2)
    H, D, cu = 1, 2, [0, 1, 1, 6]
    T, C = cu[-1], 3 * H * D
    x, w = r.normal(size=(T, C)), r.normal(size=(C, 4))
    past = r.normal(size=(3, 3, C)) if cache else None
    dq, dk, dv = (r.normal(size=(T, H, D)) for _ in range(3))

    def loss():
        q, k, v, _ = prologue(x, w, H, D, cu, past)
        return np.sum(dq * q) + np.sum(dk * k) + np.sum(dv * v)

    dx, dw, dcache = prologue_backward(x, w, dq, dk, dv, H, D, cu, past)
    np.testing.assert_allclose(dx, central(loss, x), atol=ATOL)
    np.testing.assert_allclose(dw, central(loss, w), atol=ATOL)
    if cache:
        np.testing.assert_allclose(dcache, central(loss, past), atol=ATOL)
        assert np.all(dcache[1] == 0)  # the empty sequence


def test_output_epilogue_backward_is_the_gradient():
    r = np.random.default_rng(3)
    o, z, d = (r.normal(size=(3, 2, 4)) for _ in range(3))
    w = r.normal(size=4)
    z[0, 0, 0], z[0, 0, 1] = 30.0, -30.0

    def loss():
        return np.sum(d * output_epilogue(o, z, w, 1e-3))

    for x, grad in zip((o, z, w), output_epilogue_backward(o, z, w, d, 1e-3)):
        np.testing.assert_allclose(grad, central(loss, x), atol=ATOL)

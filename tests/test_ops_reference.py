"""The plain float64 forms of the sequence-block operators against central
differences and hand-evaluated values (CPU)."""

import numpy as np
import pytest

from tests import ops_reference as ref

EPS = 1e-6


def differences(f, a):
    """Central differences of the scalar f at the array a (changed in place and
    put back)."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + EPS
        hi = f()
        a[i] = keep - EPS
        lo = f()
        a[i] = keep
        g[i] = (hi - lo) / (2 * EPS)
    return g


@pytest.mark.parametrize("D,gate,lengths", [(1, False, None), (1, True, [4, 0, 3]),
                                            (2, False, [2, 4, 1]), (2, True, None)])
def test_scan_gradient_is_the_difference_quotient(D, gate, lengths):
    rng = np.random.default_rng(3)
    T, N, H, G = 4, 3, 2, 3 if gate else 2
    gx, h0 = rng.standard_normal((T, N, D * G * H)), rng.standard_normal((D, N, H))
    dy, dhy = rng.standard_normal((T, N, D * H)), rng.standard_normal((D, N, H))

    def loss():
        y, hy, _ = ref.scan(gx, h0, D, gate, lengths)
        return (y * dy).sum() + (hy * dhy).sum()

    dgx, dh0 = ref.scan_backward(gx, ref.scan(gx, h0, D, gate, lengths)[2], dy, dhy, D, gate)
    # second-order differences of O(1) quantities: rounding 1e-16 / EPS plus EPS^2
    assert np.abs(differences(loss, gx) - dgx).max() < 1e-8
    assert np.abs(differences(loss, h0) - dh0).max() < 1e-8


def test_scan_by_hand():
    # p = 0: f = 1/2.  h: 2 -> (2 + 4) / 2 = 3 -> (3 + 1) / 2 = 2
    gx = np.array([[[0.0, 4.0]], [[0.0, 1.0]]])
    y, hy, _ = ref.scan(gx, np.full((1, 1, 1), 2.0), 1, False)
    assert y.ravel().tolist() == [3.0, 2.0] and hy.item() == 2.0


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
def test_glu_gradient_is_the_difference_quotient(act):
    rng = np.random.default_rng(4)
    x, W = rng.standard_normal((3, 4)), rng.standard_normal((10, 4))
    dy = rng.standard_normal((3, 5))
    loss = lambda: (ref.glu(x, W, act) * dy).sum()  # noqa: E731
    dx, dW = ref.glu_backward(x, W, dy, act)
    assert np.abs(differences(loss, x) - dx).max() < 1e-7
    assert np.abs(differences(loss, W) - dW).max() < 1e-7


def test_w4_nibbles_in_order():
    q = np.array([[0x21, 0x43]], dtype=np.uint8)  # 1, 2, 3, 4
    s = np.array([[1.0, 10.0]])
    assert ref.w4_weights(q, s, None, 4, 2).tolist() == [[-7.0, -6.0, -50.0, -40.0]]
    z = np.array([[1, 0]], dtype=np.uint8)
    assert ref.w4_weights(q, s, z, 3, 2).tolist() == [[0.0, 1.0, 30.0]]

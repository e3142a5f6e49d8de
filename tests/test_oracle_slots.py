"""Pins of the many-adapter oracle: hand-worked maps, and the layer against
one call of the single-adapter oracle per token."""

import numpy as np

from oracle import linear, slots


def test_token_slots_by_hand():
    assert slots.token_slots([2, 0, 3], [7, 1, 4], 7).tolist() == [7, 7, 4, 4, 4, -1, -1]
    assert slots.token_slots([2, -5, 3], [7, 1, 4], 4).tolist() == [7, 7, 4, 4]
    assert slots.token_slots([], [], 2).tolist() == [-1, -1]


def test_each_token_is_the_single_adapter_layer():
    rng = np.random.default_rng(0)
    x, W = rng.standard_normal((6, 64)), rng.standard_normal((64, 64))
    A, B = rng.standard_normal((3, 4, 64)), rng.standard_normal((3, 64, 4))
    scale, ids = np.array([0.5, 2.0, 1.0]), np.array([2, -1, 0, 3, 1, 1])
    h, size = slots.linear_fwd_slots(x, W, A, B, scale, ids)
    for m, a in enumerate(ids):
        if 0 <= a < 3:
            ref, _ = linear.linear_fwd(x[m:m + 1], W, A[a], B[a], 4 * scale[a])
        else:
            ref = x[m:m + 1] @ W.T
        np.testing.assert_allclose(h[m], ref[0], rtol=1e-12, atol=1e-12)
        assert np.all(size[m] >= np.abs(h[m] - W @ x[m]) - 1e-9)

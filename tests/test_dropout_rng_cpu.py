"""Host-side checks of the counter-based dropout calls, and the oracle's
gradient with that mask against differences."""

import ctypes

import numpy as np
import pytest

import bit_nf4_quantized_11_b200 as q
from oracle import linear, philox

EINVAL, ESHAPE, EWS = -1, -2, -3
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_11_b200 import build
    build.build()
    q._LIB = None          # bind anew: a test that reloads the module leaves the old module's types in the library
    return q.load()


def test_refusals(lib):
    w = q._Weight(FAKE, FAKE, FAKE, FAKE, 64, 128)

    def fwd(x=FAKE, M=4, A=FAKE, B=FAKE, r=8, rng=FAKE, p=0.1, h=FAKE, us=FAKE, ws=FAKE, size=1 << 30):
        return lib.qlora_linear_fwd_dropout_rng(x, M, ctypes.byref(w), A, B, r, 8.0, rng, p, h, us, ws, size, None)

    def bwd(dh=FAKE, x=FAKE, us=FAKE, M=4, r=8, rng=FAKE, p=0.1, dx=FAKE, dA=FAKE, dB=FAKE, ws=FAKE, size=1 << 30):
        return lib.qlora_linear_bwd_dropout_rng(dh, x, us, M, ctypes.byref(w), FAKE, FAKE, r, 8.0, rng, p, dx, dA, dB,
                                                ws, size, None)
    for name in ("x", "A", "B", "rng", "h", "us"):
        assert fwd(**{name: None}) == EINVAL and fwd(**{name: FAKE + 4}) == EINVAL, name
    for name in ("dh", "x", "us", "rng", "dx", "dA", "dB"):
        assert bwd(**{name: None}) == EINVAL and bwd(**{name: FAKE + 4}) == EINVAL, name
    for f in (fwd, bwd):
        for p in (-1e-9, 1.0, float("nan"), float("inf")):
            assert f(p=p) == EINVAL
        assert f(M=0) == ESHAPE and f(r=257) == ESHAPE and f(r=0) == ESHAPE
        assert f(ws=None) == EWS and f(size=0) == EWS and f(ws=FAKE + 16) == EWS
    k = lib.qlora_dropout_keep_bits
    assert k(None, 0.1, 4, 64, FAKE, None) == EINVAL
    assert k(FAKE + 4, 0.1, 4, 64, FAKE, None) == EINVAL
    assert k(FAKE, 1.0, 4, 64, FAKE, None) == EINVAL
    assert k(FAKE, 0.1, -1, 64, FAKE, None) == EINVAL
    assert k(FAKE, 0.1, 4, 64, None, None) == EINVAL
    assert k(FAKE, 0.1, 4, 96, FAKE, None) == ESHAPE
    assert k(FAKE, 0.1, 4, 0, FAKE, None) == ESHAPE
    assert k(FAKE, 0.1, 1 << 31, 64, FAKE, None) == ESHAPE
    assert k(FAKE, 0.1, 0, 64, None, None) == 0


def test_workspace_sizes(lib):
    # du in parts of 3 x 80 ranks per column group
    for r, cols in ((8, 24), (16, 48), (12, 48), (80, 240), (88, 480), (256, 960)):
        assert q.workspace_size(q.OP_LINEAR_BWD_DROPOUT_RNG, 1000, 512, 256, r) >= 1000 * cols * 2
    assert q.workspace_size(q.OP_LINEAR_FWD_DROPOUT_RNG, 4096, 512, 256, 16) == 0
    assert q.workspace_size(q.OP_LINEAR_FWD_DROPOUT_RNG, 8, 512, 256, 16) > 0


def test_oracle_gradient_against_differences():
    rng = np.random.default_rng(0)
    M, n, o, r, p = 5, 64, 64, 3, 0.25
    x, W, A, B, dh = (rng.standard_normal(s) for s in ((M, n), (o, n), (r, n), (o, r), (M, o)))
    keep = philox.keep_mask(7, 1, p, M, n)
    loss = lambda x, A, B: (dh * linear.linear_fwd_dropout(x, W, A, B, 2.0, keep, p)[0]).sum()   # noqa: E731
    dx, dA, dB = linear.linear_bwd_dropout(dh, x, W, A, B, 2.0, keep, p)
    for i, g in enumerate((dx, dA, dB)):
        v = rng.standard_normal(g.shape)
        args = [x, A, B]
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-4 * v, args[i] - 1e-4 * v
        assert abs((loss(*up) - loss(*down)) / 2e-4 - (g * v).sum()) <= 1e-6 * np.abs(g * v).sum()

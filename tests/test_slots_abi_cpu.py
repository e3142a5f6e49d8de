"""Argument checks of the many-adapter calls that need no GPU: every refusal
comes back before any CUDA work (the pointers are aligned dummies)."""

import ctypes

import pytest

import bit_nf4_quantized_11_b200 as q

EINVAL, ESHAPE, EWS = -1, -2, -3
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from bit_nf4_quantized_11_b200 import build
    build.build()
    q._LIB = None          # bind anew: a test that reloads the module leaves the old module's types in the library
    return q.load()


def _fwd(lib, x=FAKE, M=4, w=None, A=FAKE, B=FAKE, n=2, r=8, scale=FAKE, ids=FAKE, h=FAKE, ws=FAKE, size=1 << 30,
         cols=128, rows=64):
    w = q._Weight(FAKE, FAKE, FAKE, FAKE, rows, cols) if w is None else w
    return lib.qlora_linear_fwd_slots(x, M, ctypes.byref(w), A, B, n, r, scale, ids, h, ws, size, None)


def test_linear_fwd_slots_refusals(lib):
    for name in ("x", "A", "B", "scale", "ids", "h"):
        assert _fwd(lib, **{name: None}) == EINVAL, name
        assert _fwd(lib, **{name: FAKE + 2}) == EINVAL, name
    for name in ("x", "A", "B", "h"):
        assert _fwd(lib, **{name: FAKE + 8}) == EINVAL, name
    assert _fwd(lib, w=q._Weight(None, FAKE, FAKE, FAKE, 64, 128)) == EINVAL
    assert _fwd(lib, M=0) == ESHAPE
    assert _fwd(lib, M=1 << 31) == ESHAPE
    assert _fwd(lib, n=0) == ESHAPE
    assert _fwd(lib, n=1 << 28) == ESHAPE
    assert _fwd(lib, r=0) == ESHAPE
    assert _fwd(lib, r=257) == ESHAPE
    assert _fwd(lib, cols=100) == ESHAPE
    assert _fwd(lib, rows=32) == ESHAPE
    assert _fwd(lib, ws=None) == EWS
    assert _fwd(lib, ws=FAKE + 16) == EWS
    assert _fwd(lib, size=0) == EWS
    need = q.workspace_size(q.OP_LINEAR_FWD_SLOTS, 4, 128, 64, 8)
    assert need > 0 and _fwd(lib, size=need - 1) == EWS


def test_workspace_does_not_depend_on_the_table(lib):
    assert q.workspace_size(q.OP_LINEAR_FWD_SLOTS, 0, 128, 64, 8) == 0
    assert q.workspace_size(q.OP_LINEAR_FWD_SLOTS, 100, 4096, 4096, 12) >= 100 * 16 * 2
    with pytest.raises(ValueError):
        q.workspace_size(q.OP_LINEAR_FWD_SLOTS, -1, 128, 64, 8)


def test_token_slots_refusals(lib):
    f = lib.qlora_token_slots
    assert f(FAKE, FAKE, -1, 4, FAKE, None) == EINVAL
    assert f(FAKE, FAKE, 1, -4, FAKE, None) == EINVAL
    assert f(None, FAKE, 1, 4, FAKE, None) == EINVAL
    assert f(FAKE, None, 1, 4, FAKE, None) == EINVAL
    assert f(FAKE, FAKE, 1, 4, None, None) == EINVAL
    assert f(FAKE + 1, FAKE, 1, 4, FAKE, None) == EINVAL
    assert f(FAKE, FAKE, 1, 1 << 31, FAKE, None) == ESHAPE
    assert f(None, None, 0, 0, None, None) == 0           # nothing to write

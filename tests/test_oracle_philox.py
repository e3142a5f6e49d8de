"""Pins of the counter-based mask: the generator against the published
known-answer vectors of Philox4x32-10 (the same round, three times more), and
the mask's shares and independence."""

import numpy as np

from oracle import philox


def test_ten_rounds_give_the_published_vectors():
    assert philox.philox4x32((0, 0, 0, 0), (0, 0), 10) == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    f = 0xFFFFFFFF
    assert philox.philox4x32((f, f, f, f), (f, f), 10) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert philox.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), 10) == (
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)


def test_thresholds():
    assert philox.threshold(0.0) == 0 and philox.threshold(0.5) == 32768 and philox.threshold(0.05) == 3277
    assert philox.threshold(0.9999999) == 65535


def test_shares_and_different_masks():
    # 64 x 1024 draws: the share kept is within 5 standard deviations of 1 - T / 65536
    for p in (0.05, 0.5):
        k = philox.keep_mask(1, 2, p, 64, 1024)
        q = 1 - philox.threshold(p) / 65536
        assert abs(k.mean() - q) < 5 * np.sqrt(q * (1 - q) / k.size)
    a, b, c = (philox.keep_mask(s, o, 0.5, 16, 512) for s, o in ((1, 2), (3, 2), (1, 5)))
    for u, v in ((a, b), (a, c), (a[1:], a[:-1]), (a[:, 8:], a[:, :-8])):
        n = u.size
        assert abs((u == v).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
    assert philox.keep_mask(-5, -7, 0.0, 3, 64).all()

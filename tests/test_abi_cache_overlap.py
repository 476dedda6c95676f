"""Paged-cache calls whose outputs lie over their inputs are refused on the host (no GPU).

Every call here is refused: the pointers lead nowhere.
"""
from __future__ import annotations

import ctypes

from tests.test_abi import L  # noqa: F401

P = ctypes.c_void_p
FAR = P(1 << 40)
UNSUPPORTED = 5


def at(byte):
    return P(0x100000 + byte)


def test_append_with_lengths_over_lengths(L):
    B = 8

    def ap(sl, ns, cn=None, kp=at(1 << 20), vp=at(2 << 20), ke=at(3 << 20), ve=at(4 << 20), c=2):
        return L.parallax_kv_append(at(5 << 20), at(6 << 20), None, None, kp, vp, ke if c == 2 else None,
                                    ve if c == 2 else None, at(7 << 20), sl, cn, ns, None, B, 2, 5, 64, 4, 8, 128, 1, c,
                                    None)
    for byte in (4, 28, -4, -28):
        assert ap(at(64), at(64 + byte)) == UNSUPPORTED
        assert ap(FAR, at(64 + byte), cn=at(64)) == UNSUPPORTED
    # K and V in the same pages, or exponents of one array
    size = 8 * 2 * 64 * 128
    for byte in (0, size - 16, 16 - size):
        assert ap(at(64), None, vp=at((1 << 20) + byte)) == UNSUPPORTED
    assert ap(at(64), None, ve=at((3 << 20) + 63)) == UNSUPPORTED


def test_evict_with_outputs_over_inputs(L):
    B, Hkv, ps, mp, nmp = 2, 2, 64, 4, 2

    def ev(sl=at(0), ns=at(64), w=at(1 << 20), nw=None):
        return L.parallax_kv_evict(at(2 << 20), at(3 << 20), at(4 << 20), at(5 << 20), at(6 << 20), sl, w, at(7 << 20), ns,
                                   at(8 << 20), nw, B, Hkv, ps, mp, nmp, 8, 128, 100, 10, 2, None)
    assert ev(ns=at(4)) == UNSUPPORTED and ev(ns=at(-4)) == UNSUPPORTED
    old, new = B * Hkv * ps * mp * 4, B * Hkv * ps * nmp * 4
    for byte in (16, old - 16, 16 - new):
        assert ev(nw=at((1 << 20) + byte)) == UNSUPPORTED

"""Pins of the paged-cache oracle to facts that do not come from it (CPU)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc


def test_codes_are_torch_float8():
    c = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(c).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(np.isnan(t), np.isnan(oc.CODES))
    assert np.array_equal(t[~np.isnan(t)], oc.CODES[~np.isnan(t)])


def test_encode_rounds_as_torch_does():
    rng = np.random.default_rng(0)
    mids = (oc.CODES[:126] + oc.CODES[1:127]) / 2              # every tie
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000), mids, -mids, oc.CODES[:127],
                        np.nextafter(mids, 0), np.nextafter(mids, 1e9), [0.0, -0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oc.encode(x.astype(np.float64)), want)
    assert np.all(oc.encode([np.inf, -np.inf, np.nan]) == 0x7F)


@pytest.mark.parametrize("a,e", [(448.0, 0), (449.0, 1), (224.0, -1), (0.0, -120), (1e-45, -120), (3.3e38, 120)])
def test_exponent(a, e):
    assert oc.exponent(a) == e


def _cache(rng, num_pages, Hkv, ps, d):
    codes = rng.integers(0, 126, (num_pages, Hkv, ps, d)).astype(np.uint8)
    return codes, rng.integers(-8, -4, (num_pages, Hkv, ps // 16)).astype(np.int8)


def test_append_keeps_what_fits_and_grows_its_block():
    rng = np.random.default_rng(1)
    kp, ke = _cache(rng, 4, 2, 32, 64)
    vp, ve = _cache(rng, 4, 2, 32, 64)
    table = np.array([[2, 0], [1, 3]], np.int32)
    x = rng.standard_normal((2, 2, 20, 64))
    x[1, 1, 0, 0] = 1e4                                        # a new row far above its block's
    out = oc.append(x, x, kp, vp, ke, ve, table, [5, 31], [20, 3])
    vals, was = oc.values(out[0], out[2]), oc.values(kp, ke)
    for b, s, n in ((0, 5, 20), (1, 31, 3)):
        got = oc.rows(vals, table[b], s + n)
        old = oc.rows(was, table[b], s)
        # half a step of the rounding; a moved code is at most half a subnormal step off
        step = 2.0 ** -10 * 2.0 ** np.repeat(oc.rows(out[2][..., None], table[b], 4)[..., 0], 16, 1)[:, :s + n, None]
        assert np.all(np.abs(got[:, s:] - x[b, :, :n]) <= np.maximum(np.abs(x[b, :, :n]) * 2.0 ** -4, step[:, s:]))
        assert np.all(np.abs(got[:, :s] - old) <= np.maximum(np.abs(old) * 2.0 ** -4, step[:, :s]))
    # the smallest exponent that holds the new row
    assert out[2][3, 1, 0] == oc.exponent(np.abs(x[1, 1, 1:3]).max()) and out[2][1, 1, 1] == oc.exponent(1e4)
    assert list(out[4]) == [25, 34]


def test_decode_is_the_contiguous_oracle_and_weights_sum_to_one_per_head():
    rng = np.random.default_rng(2)
    kp, vp = rng.standard_normal((7, 2, 16, 64)), rng.standard_normal((7, 2, 16, 64))
    table = rng.permutation(7)[:6].reshape(2, 3).astype(np.int32)
    q, rho = rng.standard_normal((2, 6, 64)), rng.standard_normal((2, 6, 64))
    sl = np.array([33, 48], np.int32)
    y, lse, w = oc.decode(q, rho, kp, vp, table, sl, np.zeros((2, 2, 48)))
    y2, lse2 = oracle.default().decode_paged(q, rho, kp, vp, table, sl)
    assert np.allclose(y, y2, rtol=0, atol=1e-12) and np.allclose(lse, lse2, rtol=0, atol=1e-12)
    assert np.allclose(w.sum(2), 3.0, atol=1e-12) and np.all(w[0, :, 33:] == 0)
    # one key takes everything; equal keys share alike
    k1 = np.zeros_like(kp)
    _, _, w1 = oc.decode(q, None, k1, vp, table, [1, 48], np.zeros((2, 2, 48)))
    assert np.allclose(w1[0, :, 0], 3.0) and np.allclose(w1[1], 3.0 / 48)


def test_evict_small_case_by_hand():
    ps, d = 16, 64
    kp = np.arange(3 * ps, dtype=np.float64).reshape(3, 1, ps, 1) * np.ones(d)
    w = np.zeros((1, 1, 32))
    w[0, 0, :20] = [5, 1, 9, 1, 7] + [0] * 12 + [3, 0, 0]
    out = oc.evict(kp, kp, None, None, np.array([[0, 1]]), [20], w, np.array([[2]]), 6, 2,
                   np.full((1, 1, 6), -1), np.full((1, 1, 16), -1.0))
    assert list(out[5][0, 0]) == [0, 2, 4, 17, 18, 19] and list(out[4]) == [6]
    assert list(out[0][2, 0, :7, 0]) == [0, 2, 4, 17, 18, 19, 38]
    assert list(out[6][0, 0, :7]) == [5, 9, 7, 3, 0, 0, -1]
    tie = oc.evict(kp, kp, None, None, np.array([[0, 1]]), [20], w, np.array([[2]]), 6, 0,
                   np.full((1, 1, 6), -1), np.full((1, 1, 16), -1.0))
    assert list(tie[5][0, 0]) == [0, 1, 2, 3, 4, 17]
    tie = oc.evict(kp, kp, None, None, np.array([[0, 1]]), [20], w, np.array([[2]]), 5, 0,
                   np.full((1, 1, 5), -1), np.full((1, 1, 16), -1.0))
    assert list(tie[5][0, 0]) == [0, 1, 2, 4, 17]              # of the two of weight 1 the lower


def test_evict_groups_blocks_of_different_exponents():
    rng = np.random.default_rng(3)
    kp, ke = _cache(rng, 4, 1, 32, 64)
    w = rng.random((1, 1, 64))
    table, new = np.array([[1, 0]]), np.array([[3]])
    out = oc.evict(kp, kp, ke, ke, table, [64], w, new, 32, 0, np.zeros((1, 1, 32), int), np.zeros((1, 1, 32)))
    keep = out[5][0, 0]
    assert np.array_equal(np.sort(np.argsort(-w[0, 0])[:32]), keep)
    got, was = oc.values(out[0], out[2])[3, 0], oc.rows(oc.values(kp, ke), table[0], 64)[0][keep]
    assert np.all(np.abs(got - was) <= np.maximum(2.0 ** -4 * np.abs(was), 2.0 ** (-10 - 5)))


PLANTED = {
    "append_scale_of_old_rows_ignored": ("e = max(e, was)", "e = max(e, EMIN)", test_append_keeps_what_fits_and_grows_its_block),
    "append_old_rows_not_moved": ("moved = encode(CODES[old] * 2.0 ** (was - e))", "moved = old", test_append_keeps_what_fits_and_grows_its_block),
    "decode_weights_not_summed_over_heads": ("wacc[b, h // G, :n] += s", "wacc[b, h // G, :n] = s",
                                             test_decode_is_the_contiguous_oracle_and_weights_sum_to_one_per_head),
    "evict_ties_to_the_newer": ("key=lambda t: (-w[t], t)", "key=lambda t: (-w[t], -t)", test_evict_small_case_by_hand),
    "evict_recent_forgotten": ("r = min(recent, n)\n        lens", "r = 0\n        lens", test_evict_small_case_by_hand),
    "evict_rows_not_moved_to_the_new_exponent": ("x = np.where((e == e.max())[:, None], x, encode(CODES[x] * 2.0 ** (e - e.max())[:, None]))",
                                                 "pass", test_evict_groups_blocks_of_different_exponents),
}


@pytest.mark.parametrize("name", sorted(PLANTED))
def test_planted_mistakes_are_caught(name, monkeypatch):
    old, new, pin = PLANTED[name]
    src = open(oc.__file__).read()
    assert src.count(old) == 1
    import types

    m = types.ModuleType("mutant")
    m.__dict__["__name__"] = "mutant"
    exec(compile(src.replace(old, new), "mutant", "exec"), m.__dict__)
    monkeypatch.setitem(globals(), "oc", m)
    with pytest.raises(AssertionError):
        pin()

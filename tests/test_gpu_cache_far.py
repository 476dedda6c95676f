"""The cache decodes where weights, values and probes lie far apart, against the fp64 oracle.

The bound of a result is made of what each token contributes to it: a token that the softmax leaves no
weight, however large its V or its probe product, must not cost the others a bit.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import softmax_learned_covariance_b200 as plx
from oracle import cache as oc
from tests.test_gpu_cache import DEV, Cache, bf16, f64, no_error

pytestmark = pytest.mark.gpu


def refill(c, kv, vv):
    """The pool with these values: fp64, rounded to the cache's type."""
    if not c.q8:
        c.pages = [f64(bf16(x)) for x in (kv, vv)]
    else:
        c.exp, c.codes = [], []
        for x in (kv, vv):
            amax = np.abs(x).reshape(c.n, c.Hkv, c.ps // 16, 16 * c.d).max(-1)
            e = np.array([oc.exponent(a) for a in amax.ravel()], np.int8).reshape(amax.shape)
            c.exp.append(e)
            c.codes.append(oc.encode(x * 2.0 ** -np.repeat(e.astype(float), 16, -1)[..., None]))
    c.upload()


def crowd(c, B):
    """The table with B sequences; the new ones name no page."""
    c.table = np.concatenate([c.table, np.full((B - c.B, c.table.shape[1]), -9, np.int32)])
    c.B = B
    c.tab = torch.from_numpy(c.table).to(DEV)


def bounds(q, rho, c, sl):
    """Per (b, h, element) bound of y.

    A score sums d exact products in fp32: 2 (d + 8) 2^-24 sum|q k| covers truncating adds; its scale and its
    distance from the reference add roundings of 2^-24 of their size, the exponential 2^-21.  A weight is carried
    as two 16-bit parts, 2^-21 (e4m3) or 2^-16 (bf16) of it.  A sum adds each of a warp's L / 64 tiles twice,
    16 products at a time, then the merges: (L / 32 + 64) 2^-23 of the sum of magnitudes.  All that is relative
    to a token's own contribution.  fp16 parts (e4m3) also have a smallest step: a weight and its product with a
    are off by 2^-25 where the largest contribution 2^ve weight so far is held at 2^10 or more, which is
    2^-35 |code| of that (the bound takes twice as much).
    """
    B, Hq, d = q.shape
    G = Hq // c.Hkv
    kv, vv = c.values()
    out = np.zeros((B, Hq, d))
    for b in range(B):
        L = int(sl[b])
        if L == 0:
            continue
        k, v = oc.rows(kv, c.table[b], L), oc.rows(vv, c.table[b], L)
        if c.q8:
            t = np.arange(L)
            two = 2.0 ** c.exp[1][c.table[b][t // c.ps], :, t % c.ps // 16].T.astype(float)
        for h in range(Hq):
            kk, x = k[h // G], np.abs(v[h // G])
            z = kk @ q[b, h] / np.sqrt(d)
            mag = np.abs(kk) @ np.abs(q[b, h]) / np.sqrt(d)
            s = np.exp(z - z.max())
            s /= s.sum()
            e = (2 * (d + 8) * mag + 8 * np.abs(z) + 4 * (z.max() - z)) * 2.0 ** -24 + 2.0 ** -21
            e += (2.0 ** -21 if c.q8 else 2.0 ** -16) + (L / 32 + 64) * 2.0 ** -23
            el = s @ e                                           # of the sum of the weights
            o = s @ v[h // G]
            eo = (s * e) @ x + np.abs(o) * el
            if c.q8:
                codes = (x / two[h // G][:, None]).sum(0)
                eo += 2.0 ** -34 * codes * (s * two[h // G]).max()
            total = eo + 8 * 2.0 ** -24 * np.abs(o)
            if rho is not None:
                a = kk @ rho[b, h]
                da = 2 * (d + 8) * (np.abs(kk) @ np.abs(rho[b, h])) * 2.0 ** -24
                ta = s * (e * np.abs(a) + da)
                abar, m = s @ a, (s * a) @ v[h // G]
                ea = ta.sum() + abs(abar) * el
                em = ta @ x + np.abs(m) * el
                if c.q8:
                    em += 2.0 ** -34 * codes * (s * np.abs(a) * two[h // G]).max()
                total += em + abs(abar) * eo + np.abs(o) * ea + eo * ea
                total += 8 * 2.0 ** -24 * (np.abs(m) + np.abs(o * abar))
            out[b, h] = total
    return out


def decode(c, q, rho, sl):
    sld = torch.tensor(sl, dtype=torch.int32, device=DEV)
    r = None if rho is None else rho.to(DEV)
    if c.q8:
        y, _ = plx.parallax_decode_paged_q8(q.to(DEV), r, c.kp, c.vp, c.ke, c.ve, c.tab, sld)
    else:
        w = torch.zeros((c.B, c.Hkv, c.table.shape[1] * c.ps), device=DEV)
        y, _ = plx.parallax_decode_paged_acc(q.to(DEV), r, c.kp, c.vp, c.tab, sld, w)
    no_error()
    return f64(y)


def check(c, q, rho, sl):
    y = decode(c, q, rho, sl)
    q64, r64 = f64(q), None if rho is None else f64(rho)
    n = sum(1 for x in sl if x)                                  # the others are behind these and empty
    assert not any(sl[n:]) and np.all(y[n:] == 0)
    kv, vv = c.values()
    yr, _, _ = oc.decode(q64[:n], None if rho is None else r64[:n], kv, vv, c.table, sl[:n])
    tol = bounds(q64[:n], None if rho is None else r64[:n], c, sl[:n])
    assert np.all(np.abs(y[:n] - yr) <= tol + 2.0 ** -24 * np.abs(yr) + 1e-40)


# how the decode is cut: pages of 128, tokens of a table, sequences in it
PLANS = {"ctas": (4, 6), "ranges": (16, 6), "ctas of long items": (16, 1200), "warps": (4, 600)}


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("with_rho", [True, False])
@pytest.mark.parametrize("G", [3, 6])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("plan", list(PLANS))
def test_tokens_without_weight_cost_the_others_nothing(plan, d, G, with_rho, q8):
    """V far larger, or a probe product far larger, under weights of e^-60; and one token with nearly all the
    weight and no V: what the rest contributes is the result."""
    mp, crowded = PLANS[plan]
    rng = np.random.default_rng(mp + d + G)
    B, Hkv, ps = 6, 2, 128
    c = Cache(rng, B, Hkv, ps, mp, d, q8, spare=0)
    kv, vv = (rng.standard_normal((c.n, Hkv, ps, d)) for _ in range(2))
    kv[..., 0] = 0.0
    down, up = -60.0 * np.sqrt(d) / 6.0, 17.0 * np.sqrt(d) / 6.0   # of channel 0, where q is 6
    L = mp * ps
    rows = lambda b, t: (c.table[b, t // ps], slice(None), slice(t % ps, t % ps + 16))
    for b, t in ((0, 0), (1, L // 2), (1, L - 16), (2, L - 32)):   # large V without weight, first, inside, last
        kv[rows(b, t)][..., 0] = down
        vv[rows(b, t)] *= 2.0 ** (24 if b < 2 else 40)
    for b, t in ((3, 0), (4, L // 2 + 5)):                         # nearly all the weight without V
        at = (c.table[b, t // ps], slice(None), t % ps)
        kv[at][..., 0] = up
        vv[at] = 0.0
    kv[rows(5, 16)][..., 0] = down                                 # a large probe product without weight
    refill(c, kv, vv)
    sl = [L, L - 3, L, L, L - 100, L - 1]
    if crowded > B:
        crowd(c, crowded)
        sl += [0] * (crowded - B)
    q = rng.standard_normal((c.B, Hkv * G, d))
    q[..., 0] = 6.0
    rho = rng.standard_normal((c.B, Hkv * G, d)) * 0.3
    rho[..., 0] = 0.0
    rho[5, :, 0] = 300.0
    check(c, bf16(q), bf16(rho) if with_rho else None, sl)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_probe_products_past_fp16(d, q8):
    """|k.rho| far above 65504, among others that are not."""
    rng = np.random.default_rng(40)
    c = Cache(rng, 3, 2, 16, 20, d, q8)
    q, rho = rng.standard_normal((3, 6, d)), rng.standard_normal((3, 6, d))
    rho[1] *= 2.0 ** 20
    rho[2] *= 2.0 ** 110
    check(c, bf16(q), bf16(rho), [320, 317, 200])


@pytest.mark.parametrize("bits", [-130, -118, -100, 100, 118, 126])
@pytest.mark.parametrize("d", [64, 128])
def test_vectors_at_the_ends_of_their_type(d, bits):
    """q and rho near bf16's largest and smallest values, under keys that bring their products back to 1."""
    rng = np.random.default_rng(41)
    c = Cache(rng, 3, 2, 16, 20, d)
    k, v = (rng.standard_normal((c.n, 2, 16, d)) for _ in range(2))
    refill(c, k * 2.0 ** min(-bits, 125), v)
    q, rho = (rng.uniform(0.5, 1.9, (3, 6, d)) * rng.choice([-1.0, 1.0], (3, 6, d)) * s for s in (1.0, 0.1))
    check(c, bf16(q * 2.0 ** bits), bf16(rho * 2.0 ** bits), [320, 317, 5])

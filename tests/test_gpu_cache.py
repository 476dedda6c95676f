"""The paged cache's write, decode and eviction (through the binding) vs the fp64 oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import softmax_learned_covariance_b200 as plx
from oracle import cache as oc

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def codes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def no_error():
    assert plx.parallax_last_device_error() == 0


class Cache:
    """A pool of pages with a table, on the device and as the oracle's arrays."""

    def __init__(self, rng, B, Hkv, ps, mp, d, q8=True, spare=2, more=0, scale=(1.0, 1.0)):
        n = B * mp + B * more + spare
        self.q8, self.d, self.ps, self.n, self.Hkv, self.B = q8, d, ps, n, Hkv, B
        ids = rng.permutation(n).astype(np.int32)
        self.table = ids[:B * mp].reshape(B, mp).copy()
        self.table2 = ids[B * mp:B * (mp + more)].reshape(B, more).copy() if more else None
        x = [rng.standard_normal((n, Hkv, ps, d)) * s for s in scale]
        if q8:
            nb = ps // 16
            self.exp, self.codes = [], []
            for v in x:
                amax = np.abs(v).reshape(n, Hkv, nb, 16 * d).max(-1)
                e = np.ceil(np.log2(amax / 448.0)).astype(np.int8)
                self.exp.append(e)
                self.codes.append(oc.encode(v * 2.0 ** -np.repeat(e.astype(float), 16, -1)[..., None]))
        else:
            self.pages = [f64(bf16(v)) for v in x]
        self.upload()

    def upload(self):
        if self.q8:
            self.kp, self.vp = (torch.from_numpy(c).to(DEV).view(E4M3) for c in self.codes)
            self.ke, self.ve = (torch.from_numpy(e).to(DEV) for e in self.exp)
        else:
            self.kp, self.vp = (bf16(p).to(DEV) for p in self.pages)
            self.ke = self.ve = None
        self.tab = torch.from_numpy(self.table).to(DEV)
        self.tab2 = None if self.table2 is None else torch.from_numpy(self.table2).to(DEV)

    def widen(self, tokens):
        """The table with room for `tokens`; the new entries name no page."""
        more = -(-tokens // self.ps) - self.table.shape[1]
        self.table = np.concatenate([self.table, np.full((self.B, more), -9, np.int32)], 1)
        self.tab = torch.from_numpy(self.table).to(DEV)

    def values(self):
        return [oc.values(c, e) for c, e in zip(self.codes, self.exp)] if self.q8 else self.pages

    def raw(self):
        """(kpages, vpages, kexp, vexp) as the oracle takes them."""
        return (*self.codes, *self.exp) if self.q8 else (*self.pages, None, None)

    def check(self, want):
        """The device's pool equals the oracle's, bit for bit (one NaN as good as another)."""
        for got, ref in zip((self.kp, self.vp), want[:2]):
            if self.q8:
                g, r = codes_of(got).copy(), ref.copy()
                for a in (g, r):
                    a[(a & 0x7F) == 0x7F] = 0x7F
                assert np.array_equal(g, r)
            else:
                assert np.array_equal(f64(got), ref, equal_nan=True)
        if self.q8:
            for got, ref in zip((self.ke, self.ve), want[2:4]):
                assert np.array_equal(got.cpu().numpy(), ref)


# ------------------------------------------------------------------ append
def run_append(c, k, v, seqlens, counts=None, wacc=None, **kw):
    sl = torch.tensor(seqlens, dtype=torch.int32, device=DEV)
    cn = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
    return plx.parallax_kv_append(k, v, c.kp, c.vp, c.tab, sl, kexp=c.ke, vexp=c.ve, counts=cn, wacc=wacc, **kw)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps,mp", [(16, 7), (64, 2), (128, 1)])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 61])
def test_append(T, ps, mp, d, q8):
    rng = np.random.default_rng(T * 1000 + ps + d)
    B, Hkv = 5, 3
    c = Cache(rng, B, Hkv, ps, mp, d, q8)
    k, v = (bf16(rng.standard_normal((B, Hkv, T, d)) * s) for s in (30.0, 0.02))
    seqlens, counts = [0, 5, 15, 32, 51], [T, T, 0, max(1, T // 2), T]
    w = rng.random((B, Hkv, mp * ps)).astype(np.float32)
    wd = torch.from_numpy(w).to(DEV)
    want = oc.append(f64(k), f64(v), *c.raw(), c.table, seqlens, counts, w)
    ns = run_append(c, k.to(DEV), v.to(DEV), seqlens, counts, wd)
    assert ns.tolist() == want[4].tolist()
    c.check(want)
    assert np.array_equal(wd.cpu().numpy(), want[5])
    no_error()


def test_append_strided_and_without_counts():
    """A [B, T, Hkv, d] projection's transpose, and slices of a wider one; counts default to T."""
    rng = np.random.default_rng(3)
    B, Hkv, T, d = 2, 4, 19, 128
    c = Cache(rng, B, Hkv, 32, 2, d)
    both = bf16(rng.standard_normal((B, T, 2, Hkv, d))).to(DEV)
    k, v = both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2)
    want = oc.append(f64(k), f64(v), *c.raw(), c.table, [0, 40], None)
    ns = run_append(c, k, v, [0, 40])
    assert ns.tolist() == [19, 59]
    c.check(want)
    no_error()


def test_append_extreme_values():
    """Zeros, the smallest and largest magnitudes, infinities, NaN, and blocks that grow under old rows."""
    rng = np.random.default_rng(4)
    B, Hkv, T, d = 6, 2, 20, 64
    c = Cache(rng, B, Hkv, 16, 4, d)
    x = rng.standard_normal((B, Hkv, T, d))
    x[0] = 0.0
    x[1] *= 1e-38
    x[2] *= 5e37
    x[3, :, 3, 5], x[3, :, 4, 6], x[3, 0, 7, 8] = np.inf, -np.inf, np.nan
    x[3, 1] = np.nan                                 # nothing finite
    x[4] *= 2.0 ** 60                                # old rows become subnormal, then zero
    x[5, :, ::2] *= 2.0 ** 9
    k = bf16(x)
    sl = [3, 3, 3, 0, 7, 9]
    want = oc.append(f64(k), f64(k), *c.raw(), c.table, sl)
    run_append(c, k.to(DEV), k.to(DEV), sl)
    c.check(want)
    no_error()


def test_append_token_by_token():
    """Forty single-token writes: each equals the oracle's write on the device's own state."""
    rng = np.random.default_rng(5)
    B, Hkv, d = 3, 2, 128
    c = Cache(rng, B, Hkv, 16, 4, d)
    sl, ref = [0, 1, 14], c.raw()
    for i in range(40):
        k, v = (bf16(rng.standard_normal((B, Hkv, 1, d)) * 2.0 ** rng.integers(-6, 6)) for _ in range(2))
        want = oc.append(f64(k), f64(v), *ref, c.table, sl)
        ns = run_append(c, k.to(DEV), v.to(DEV), sl)
        ref, sl = want[:4], ns.tolist()
        assert sl == want[4].tolist()
    c.check(ref)
    no_error()


def test_append_past_the_end_and_to_bad_pages():
    rng = np.random.default_rng(6)
    B, Hkv, T, d = 3, 2, 20, 64
    c = Cache(rng, B, Hkv, 16, 2, d)
    c.table[1, 1] = c.n                              # out of range
    c.table[2, 0] = -1
    c.upload()
    k = bf16(rng.standard_normal((B, Hkv, T, d)))
    ns = run_append(c, k.to(DEV), k.to(DEV), [20, 0, 0])
    assert ns.tolist() == [32, 20, 20]
    assert plx.parallax_last_device_error() == 8
    # what fits is written: 12 tokens of sequence 0, the first page of 1, the second of 2
    ref = c.raw()
    for b, s, t0, n in ((0, 20, 0, 12), (1, 0, 0, 16), (2, 16, 16, 4)):
        t = c.table.copy()
        t[:b], t[b + 1:] = -1, -1
        part = np.zeros((B, Hkv, n, d))
        part[b] = f64(k)[b, :, t0:t0 + n]
        cn = [0] * B
        cn[b] = n
        sls = [0] * B
        sls[b] = s
        ref = oc.append(part, part, *ref[:4], t, sls, cn)
    c.check(ref)


# ------------------------------------------------------------------ decode
def bounds(q, rho, kv, vv, table, sl, Hkv, q8):
    """Per (b, h) bounds (y, lse, s) of the kernel's rounding, from the arithmetic.

    A score sums d exact products in fp32: 2 (d + 8) 2^-24 sum|q k| covers truncating adds; the weights'
    exponential is good to 2^-21, a weight carried as two 16-bit parts to 2^-21 (e4m3: fp16) or 2^-16
    (bf16), with an absolute floor of 2^-24 against the largest weight and value (16 2^-24 for the
    probe's); a value sum adds each of a warp's L/64 tiles twice, 16 products at a time, and the merges:
    (L/32 + 64) 2^-23 of the sum of magnitudes.
    """
    B, Hq, d = q.shape
    by, bl, bs = np.zeros((B, Hq)), np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        L = int(sl[b])
        if L == 0:
            continue
        k, v = oc.rows(kv, table[b], L), oc.rows(vv, table[b], L)
        for h in range(Hq):
            kk, vmax = np.abs(k[h // (Hq // Hkv)]), np.abs(v[h // (Hq // Hkv)]).max()
            z = k[h // (Hq // Hkv)] @ q[b, h] / np.sqrt(d)
            mag = (kk @ np.abs(q[b, h])).max() / np.sqrt(d)
            eps = (2 * (d + 8) * mag + 8 * np.abs(z).max()) * 2.0 ** -24 + 2.0 ** -21
            l = np.exp(z - z.max()).sum()
            epw = 2 * eps + (2.0 ** -21 if q8 else 2.0 ** -16)
            acc = (L / 32 + 64) * 2.0 ** -23
            by[b, h] = vmax * (epw + acc + L * 2.0 ** -24 / l)
            if rho is not None:
                a = np.abs(k[h // (Hq // Hkv)] @ rho[b, h]).max()
                da = 2 * (d + 8) * (kk @ np.abs(rho[b, h])).max() * 2.0 ** -24
                by[b, h] += vmax * (4 * a * (epw + acc) + 4 * da + 2 * L * 2.0 ** -20 / l)
            bl[b, h] = eps + acc + 2.0 ** -22 * abs(np.log(l) + z.max())
            bs[b, h] = 2 * eps + 2 * acc
    return by, bl, bs


def check_decode(c, q, rho, sl, out_dtype=torch.float32, with_acc=True, seed=0):
    rng = np.random.default_rng(seed)
    Hkv, cap = c.Hkv, c.table.shape[1] * c.ps
    w = rng.random((c.B, Hkv, cap)).astype(np.float32) if with_acc else None
    wd = torch.from_numpy(w).to(DEV) if with_acc else None
    sld = torch.tensor(sl, dtype=torch.int32, device=DEV)
    r = None if rho is None else rho.to(DEV)
    if c.q8:
        y, lse = plx.parallax_decode_paged_q8(q.to(DEV), r, c.kp, c.vp, c.ke, c.ve, c.tab, sld, wacc=wd,
                                              out_dtype=out_dtype)
    else:
        y, lse = plx.parallax_decode_paged_acc(q.to(DEV), r, c.kp, c.vp, c.tab, sld, wd, out_dtype=out_dtype)
    no_error()
    kv, vv = c.values()
    q64, r64 = f64(q), None if rho is None else f64(rho)
    yr, lr, wr = oc.decode(q64, r64, kv, vv, c.table, sl, w)
    by, bl, bs = bounds(q64, r64, kv, vv, c.table, sl, Hkv, c.q8)
    yg, lg = f64(y), f64(lse)
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(yg - yr) <= by[..., None] * (1 + half) + half * np.abs(yr) + 1e-40)
    empty = np.isneginf(lr)
    assert np.array_equal(np.isneginf(lg), empty) and np.all(yg[empty] == 0)
    assert np.all(np.abs(lg[~empty] - lr[~empty]) <= bl[~empty])
    if with_acc:
        wg = f64(wd)
        G = q.shape[1] // Hkv
        add = wr - w
        tol = add * bs.reshape(c.B, Hkv, G).max(2)[..., None] + 2.0 ** -23 * (wr + G)
        assert np.all(np.abs(wg - wr) <= tol)
        for b in range(c.B):
            assert np.array_equal(wg[b, :, sl[b]:], w[b, :, sl[b]:])          # rows behind the last token
    return y, lse, wd


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("with_rho", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8, 9, 17])
def test_decode(G, ps, d, with_rho, q8):
    rng = np.random.default_rng(G * 100 + ps + d)
    B, Hkv, mp = 7, 2, max(2, 300 // ps)
    c = Cache(rng, B, Hkv, ps, mp, d, q8)
    q = bf16(rng.standard_normal((B, Hkv * G, d)))
    rho = bf16(rng.standard_normal((B, Hkv * G, d)) * 0.905) if with_rho else None
    check_decode(c, q, rho, [0, 1, 15, 16, 17, ps + 1, mp * ps])
    c.widen(2320)                    # a table for which the work is cut over the CTAs whatever the lengths
    check_decode(c, q, rho, [mp * ps, 33, 0, 1, 2 * ps, ps - 1, 0])


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("with_rho", [True, False])
def test_decode_split_over_a_long_cache(with_rho, q8):
    rng = np.random.default_rng(8)
    c = Cache(rng, 2, 2, 128, 40, 128, q8)
    q = bf16(rng.standard_normal((2, 6, 128)))
    rho = bf16(rng.standard_normal((2, 6, 128)) * 0.05) if with_rho else None
    y, lse, w = check_decode(c, q, rho, [5003, 129])
    y2, lse2, w2 = check_decode(c, q, rho, [5003, 129])
    assert torch.equal(y, y2) and torch.equal(lse, lse2) and torch.equal(w, w2)     # no schedule in the result


def test_decode_many_sequences_and_bf16_output():
    """More items than CTAs, in short tables (a CTA per item) and in long ones that the lengths do not fill."""
    rng = np.random.default_rng(9)
    c = Cache(rng, 300, 16, 16, 2, 64)
    q, rho = (bf16(rng.standard_normal((300, 16, 64))) for _ in range(2))
    check_decode(c, q, rho, list(rng.integers(0, 33, 300)), out_dtype=torch.bfloat16)
    check_decode(c, q, rho, list(rng.integers(0, 33, 300)), with_acc=False)
    c = Cache(rng, 150, 3, 16, 25, 64)
    q, rho = (bf16(rng.standard_normal((150, 3 * 9, 64))) for _ in range(2))
    sl = rng.integers(0, 400, 150)
    sl[:40] = sl[-7:] = 0
    check_decode(c, q, rho, list(sl), out_dtype=torch.bfloat16)
    check_decode(c, q, None, list(rng.integers(0, 3, 150)))
    check_decode(c, q, None, [0] * 150)
    c.widen(2500)                    # and cut over the CTAs
    check_decode(c, q, rho, list(sl), out_dtype=torch.bfloat16)
    check_decode(c, q, None, list(rng.integers(0, 3, 150)))
    check_decode(c, q, None, [0] * 150)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("with_rho", [True, False])
@pytest.mark.parametrize("G", [3, 6])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_many_short_sequences(d, G, with_rho, q8):
    """So many short items that each warp has its own."""
    rng = np.random.default_rng(17 + G)
    B, Hkv = 310, 4
    c = Cache(rng, B, Hkv, 16, 8, d, q8)
    q = bf16(rng.standard_normal((B, Hkv * G, d)))
    rho = bf16(rng.standard_normal((B, Hkv * G, d)) * 0.905) if with_rho else None
    sl = rng.integers(0, 129, B)
    sl[:3] = sl[-2:] = 0
    check_decode(c, q, rho, list(sl))
    c.tab[7, 2:] = c.n + 1                                     # bad pages in one item only
    sld = torch.from_numpy(np.full(B, 128, np.int32)).to(DEV)
    w = torch.zeros((B, Hkv, 128), device=DEV)
    args = (q.to(DEV), None if rho is None else rho.to(DEV), c.kp, c.vp)
    y, lse = plx.parallax_decode_paged_q8(*args, c.ke, c.ve, c.tab, sld, wacc=w) if q8 else \
        plx.parallax_decode_paged_acc(*args, c.tab, sld, w)
    assert plx.parallax_last_device_error() == 8
    assert torch.isfinite(y).all() and torch.isfinite(lse).all()
    assert np.allclose(w.sum(2).cpu().numpy(), G, rtol=1e-4)


def test_decode_with_heavy_and_light_blocks():
    """Scores that rise late in the cache, V blocks whose exponents differ by far, a zero V block under the peak."""
    rng = np.random.default_rng(10)
    B, Hkv, ps, mp, d = 2, 2, 16, 24, 128
    c = Cache(rng, B, Hkv, ps, mp, d)
    for b in range(B):
        for p in range(mp):
            c.exp[0][c.table[b, p]] += np.int8(p // 8)         # keys grow: the reference maximum moves
            c.exp[1][c.table[b, p]] += np.int8((-9, 0, 5, -3)[p % 4])
    c.codes[1][c.table[0, mp - 1]] = 0                         # V = 0 where the scores are largest
    c.exp[1][c.table[0, mp - 1]] = -120
    c.upload()
    q, rho = bf16(rng.standard_normal((B, 4, d))), bf16(rng.standard_normal((B, 4, d)))
    check_decode(c, q, rho, [mp * ps, mp * ps - 5])
    check_decode(c, q, None, [mp * ps, mp * ps - 5])
    c.widen(3000)
    check_decode(c, q, rho, [mp * ps, mp * ps - 5])
    check_decode(c, q, None, [mp * ps - 7, mp * ps])


@pytest.mark.parametrize("scale", [(1.0, 1e-12), (1e-10, 1e-30), (1.0, 1e12), (3.0, 1e-5)])
def test_decode_of_small_and_large_values(scale):
    """V far from 1: what a tile's missing part or a bad page stands for does not set the scale of the sums."""
    rng = np.random.default_rng(16)
    c = Cache(rng, 8, 2, 16, 9, 128, scale=scale)
    q, rho = bf16(rng.standard_normal((8, 8, 128)) / scale[0]), bf16(rng.standard_normal((8, 8, 128)) * 0.1 / scale[0])
    for r in (rho, None):
        check_decode(c, q, r, [1, 5, 16, 17, 33, 47, 130, 144])
    c.widen(2100)
    check_decode(c, q, rho, [1, 5, 16, 17, 33, 47, 130, 144])
    c = Cache(rng, 3, 1, 16, 40, 64, scale=scale)
    check_decode(c, bf16(rng.standard_normal((3, 3, 64)) / scale[0]), None, [640, 393, 7])


def test_decode_ignores_what_lies_behind_a_sequence():
    """NaN codes past the last token, table entries out of range behind the last page: neither is seen."""
    rng = np.random.default_rng(11)
    for q8 in (True, False):
        B, Hkv, ps, mp, d = 2, 2, 32, 6, 64
        c = Cache(rng, B, Hkv, ps, mp, d, q8)
        q, rho = bf16(rng.standard_normal((B, 4, d))), bf16(rng.standard_normal((B, 4, d)))
        sl = [77, 5]
        y, lse, w = check_decode(c, q, rho, sl)
        for b in range(B):
            last = sl[b] // ps
            for t in (c.kp, c.vp):
                x = t.view(torch.uint8) if q8 else t
                x[c.table[b, last], :, sl[b] % ps:] = 0x7F if q8 else float("nan")
            c.tab[b, last + 1:] = 10 ** 6
        sld = torch.tensor(sl, dtype=torch.int32, device=DEV)
        w2 = torch.from_numpy(np.random.default_rng(0).random(w.shape).astype(np.float32)).to(DEV)
        if q8:
            y2, lse2 = plx.parallax_decode_paged_q8(q.to(DEV), rho.to(DEV), c.kp, c.vp, c.ke, c.ve, c.tab, sld, wacc=w2)
        else:
            y2, lse2 = plx.parallax_decode_paged_acc(q.to(DEV), rho.to(DEV), c.kp, c.vp, c.tab, sld, w2)
        assert torch.equal(y, y2) and torch.equal(lse, lse2) and torch.equal(w, w2)
        no_error()


def test_decode_nan_inside_a_sequence_shows_in_its_head_only():
    rng = np.random.default_rng(12)
    c = Cache(rng, 2, 2, 16, 3, 64)
    c.codes[0][c.table[1, 1], 0, 3, 7] = 0x7F
    c.upload()
    q = bf16(rng.standard_normal((2, 4, 64)))
    sl = torch.tensor([40, 40], dtype=torch.int32, device=DEV)
    y, lse = plx.parallax_decode_paged_q8(q.to(DEV), q.to(DEV), c.kp, c.vp, c.ke, c.ve, c.tab, sl)
    bad = torch.isnan(y).all(2).cpu()
    assert bad.tolist() == [[False] * 4, [True, True, False, False]]
    assert torch.isfinite(y.cpu()[~bad]).all() and torch.isnan(lse.cpu()[bad]).all()


def test_decode_bad_page_reads_as_zero():
    rng = np.random.default_rng(13)
    for q8 in (True, False):
        c = Cache(rng, 2, 2, 16, 3, 64, q8)
        q = bf16(rng.standard_normal((2, 4, 64)))
        w = torch.zeros((2, 2, 48), device=DEV)
        sl = torch.tensor([40, 40], dtype=torch.int32, device=DEV)
        hole = int(c.table[1, 1])
        c.tab[1, 1] = c.n + 3
        if q8:
            y, _ = plx.parallax_decode_paged_q8(q.to(DEV), q.to(DEV), c.kp, c.vp, c.ke, c.ve, c.tab, sl, wacc=w)
        else:
            y, _ = plx.parallax_decode_paged_acc(q.to(DEV), q.to(DEV), c.kp, c.vp, c.tab, sl, w)
        assert plx.parallax_last_device_error() == 8
        kv, vv = (x.copy() for x in c.values())
        kv[hole] = vv[hole] = 0.0
        yr, _, _ = oc.decode(f64(q), f64(q), kv, vv, c.table, [40, 40])
        by, _, _ = bounds(f64(q), f64(q), kv, vv, c.table, [40, 40], 2, q8)
        assert np.all(np.abs(f64(y) - yr) <= by[..., None])


def test_decode_agrees_with_the_bf16_paged_decode():
    """Codes are exact in bf16: the same values in a bf16 cache give the same result within both kernels' gates."""
    rng = np.random.default_rng(14)
    c = Cache(rng, 3, 2, 64, 10, 128)
    kv, vv = (bf16(x).to(DEV) for x in c.values())
    q, rho = bf16(rng.standard_normal((3, 8, 128))).to(DEV), bf16(rng.standard_normal((3, 8, 128)) * 0.05).to(DEV)
    sl = torch.tensor([640, 333, 1], dtype=torch.int32, device=DEV)
    y, lse = plx.parallax_decode_paged_q8(q, rho, c.kp, c.vp, c.ke, c.ve, c.tab, sl)
    y2, lse2 = plx.parallax_decode_paged(q, rho, kv, vv, c.tab, sl)
    assert float((y - y2).abs().max()) <= 2e-2 and float((lse - lse2).abs().max()) <= 1e-3


# ------------------------------------------------------------------ evict
def run_evict(c, w, sl, budget, recent, mp2):
    B, Hkv = c.B, c.Hkv
    kept0 = np.full((B, Hkv, budget), -7, np.int32)
    nw0 = np.full((B, Hkv, mp2 * c.ps), -7.0, np.float32)
    kept, nw = torch.from_numpy(kept0).to(DEV), torch.from_numpy(nw0).to(DEV)
    ns, k2, w2 = plx.parallax_kv_evict(c.kp, c.vp, c.tab, torch.tensor(sl, dtype=torch.int32, device=DEV),
                                       torch.from_numpy(w).to(DEV), c.tab2, budget, recent, kexp=c.ke, vexp=c.ve,
                                       kept=kept, new_wacc=nw)
    assert k2 is kept and w2 is nw
    want = oc.evict(*c.raw(), c.table, sl, w, c.table2, budget, recent, kept0, nw0)
    assert ns.tolist() == want[4].tolist()
    assert np.array_equal(kept.cpu().numpy(), want[5])
    assert np.array_equal(nw.cpu().numpy(), want[6], equal_nan=True)
    c.check(want)
    return kept


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps,mp,budget,recent", [(16, 9, 50, 7), (16, 9, 1, 0), (64, 3, 64, 64), (64, 3, 130, 0),
                                                 (32, 70, 1000, 100), (32, 70, 2240, 5)])
def test_evict(ps, mp, budget, recent, d, q8):
    rng = np.random.default_rng(ps + budget + d)
    B, Hkv = 6, 2
    mp2 = -(-budget // ps)
    c = Cache(rng, B, Hkv, ps, mp, d, q8, more=mp2)
    cap = mp * ps
    w = np.exp(2 * rng.standard_normal((B, Hkv, cap))).astype(np.float32)
    run_evict(c, w, [0, 1, min(budget, cap), min(budget + 1, cap), cap - 3, cap], budget, recent, mp2)
    no_error()


def test_evict_equal_and_unordered_weights():
    """All equal, a few values often, zeros of both signs, infinities, NaN, negatives, subnormals."""
    rng = np.random.default_rng(20)
    B, Hkv, ps, mp = 6, 2, 64, 40
    c = Cache(rng, B, Hkv, ps, mp, 64, more=20)
    cap = ps * mp
    w = np.zeros((B, Hkv, cap), np.float32)
    w[0] = 3.25
    w[1] = rng.integers(0, 4, (Hkv, cap))
    w[2] = rng.choice(np.array([0.0, -0.0], np.float32), (Hkv, cap))
    w[3] = rng.choice(np.array([np.inf, -np.inf, np.nan, 1.0, -1.0, 0.0], np.float32), (Hkv, cap))
    w[4] = rng.standard_normal((Hkv, cap)) * 1e-39
    w[5] = np.float32(1.0) + rng.integers(0, 3, (Hkv, cap)) * np.float32(2.0 ** -23)   # differ in the last bits
    run_evict(c, w, [cap] * B, 1200, 33, 20)
    no_error()


def test_evict_blocks_of_far_exponents():
    rng = np.random.default_rng(21)
    c = Cache(rng, 2, 2, 16, 20, 128, more=8)
    for e in c.exp:
        e[:] = rng.integers(-120, 121, e.shape)
    c.upload()
    w = rng.random((2, 2, 320)).astype(np.float32)
    run_evict(c, w, [320, 300], 128, 16, 8)
    no_error()


def test_evict_long_sequences():
    rng = np.random.default_rng(22)
    c = Cache(rng, 1, 2, 256, 130, 64, more=20)
    w = np.exp(3 * rng.standard_normal((1, 2, 130 * 256))).astype(np.float32)
    run_evict(c, w, [130 * 256 - 9], 5000, 300, 20)
    no_error()


def test_evict_bad_pages():
    """A kept row of a bad source page is zero, a bad destination page is not written, and both are reported."""
    rng = np.random.default_rng(23)
    c = Cache(rng, 2, 1, 16, 4, 64, more=2)
    ref = c.raw()
    w = np.ones((2, 1, 64), np.float32)
    w[:, :, 40:] = 2.0
    hole, lost = int(c.table[0, 0]), int(c.table2[1, 1])
    want = list(oc.evict(*ref, c.table, [64, 64], w, c.table2, 32, 0, np.zeros((2, 1, 32), np.int32),
                         np.zeros((2, 1, 32), np.float32)))
    c.tab[0, 0], c.tab2[1, 1] = -5, c.n
    kept = plx.parallax_kv_evict(c.kp, c.vp, c.tab, torch.tensor([64, 64], dtype=torch.int32, device=DEV),
                                 torch.from_numpy(w).to(DEV), c.tab2, 32, 0, kexp=c.ke, vexp=c.ve)[1]
    assert plx.parallax_last_device_error() == 8
    assert np.array_equal(kept.cpu().numpy(), want[5])
    for got, exp, codes, e, src, se in ((c.kp, c.ke, want[0], want[2], ref[0], ref[2]),
                                        (c.vp, c.ve, want[1], want[3], ref[1], ref[3])):
        codes[lost], e[lost] = src[lost], se[lost]             # not written
        page, n = int(c.table2[0, 0]), int((want[5][0, 0, :16] < 16).sum())
        assert hole != page and n == 8
        rows = oc.values(src, se)[hole]
        del rows
        g = codes_of(got)
        assert np.all(g[page, 0, :n] == 0)                     # rows of the bad page
        vals, ref_vals = oc.values(g, exp.cpu().numpy()), oc.values(codes, e)
        assert np.allclose(vals[page, 0, n:16], ref_vals[page, 0, n:16], rtol=2.0 ** -4, atol=2.0 ** -12)
        mine = [p for p in range(c.n) if p != page]
        assert np.array_equal(g[mine], codes[mine])


# ------------------------------------------------------------------ together
def test_the_serving_loop():
    """Prompts in, tokens decoded with weights, caches halved, tokens decoded on: the oracle's loop."""
    rng = np.random.default_rng(30)
    for q8 in (True, False):
        B, Hkv, G, ps, mp, d, budget = 3, 2, 3, 16, 8, 64, 40
        c = Cache(rng, B, Hkv, ps, mp, d, q8, more=mp)
        w0 = np.zeros((B, Hkv, mp * ps), np.float32)
        w = torch.from_numpy(w0).to(DEV)
        k, v = (bf16(rng.standard_normal((B, Hkv, 70, d))) for _ in range(2))
        counts = [70, 41, 5]
        sl = run_append(c, k.to(DEV), v.to(DEV), [0, 0, 0], counts, w)
        ref = oc.append(f64(k), f64(v), *c.raw(), c.table, [0, 0, 0], counts, w0)
        table, tab, lens = c.table, c.tab, ref[4]
        raw, wr = ref[:4], ref[5].astype(np.float64)

        def step(raw, table, tab, lens, sl, w, wr):
            k, v, q, rho = (bf16(rng.standard_normal(s)) for s in ((B, Hkv, 1, d), (B, Hkv, 1, d), (B, Hkv * G, d),
                                                                   (B, Hkv * G, d)))
            sl = plx.parallax_kv_append(k.to(DEV), v.to(DEV), c.kp, c.vp, tab, sl, kexp=c.ke, vexp=c.ve, wacc=w)
            r = oc.append(f64(k), f64(v), *raw, table, lens, None, wr)
            raw, lens, wr = r[:4], r[4], r[5]
            if q8:
                y, lse = plx.parallax_decode_paged_q8(q.to(DEV), rho.to(DEV), c.kp, c.vp, c.ke, c.ve, tab, sl, wacc=w)
                vals = oc.values(raw[0], raw[2]), oc.values(raw[1], raw[3])
            else:
                y, lse = plx.parallax_decode_paged_acc(q.to(DEV), rho.to(DEV), c.kp, c.vp, tab, sl, w)
                vals = raw[:2]
            yr, lr, wr = oc.decode(f64(q), f64(rho), *vals, table, lens, wr)
            by, bl, _ = bounds(f64(q), f64(rho), *vals, table, lens, Hkv, q8)
            assert np.all(np.abs(f64(y) - yr) <= by[..., None]) and np.all(np.abs(f64(lse) - lr) <= bl)
            return raw, lens, sl, wr

        for _ in range(5):
            raw, lens, sl, wr = step(raw, table, tab, lens, sl, w, wr)
        got_w = w.cpu().numpy()
        assert np.allclose(got_w, wr, rtol=1e-4, atol=1e-6)
        # the eviction goes by the device's weights: equal to the oracle's on those
        kept0, nw0 = np.zeros((B, Hkv, budget), np.int32), np.zeros((B, Hkv, mp * ps), np.float32)
        r = oc.evict(*raw, table, lens, got_w, c.table2, budget, 8, kept0, nw0)
        sl, kept, w = plx.parallax_kv_evict(c.kp, c.vp, tab, sl, w, c.tab2, budget, 8, kexp=c.ke, vexp=c.ve)
        assert np.array_equal(kept.cpu().numpy(), r[5]) and np.array_equal(w.cpu().numpy(), r[6])
        c.check(r)
        raw, lens, wr, table, tab = r[:4], r[4], r[6].astype(np.float64), c.table2, c.tab2
        for _ in range(3):
            raw, lens, sl, wr = step(raw, table, tab, lens, sl, w, wr)
        c.check(raw)
        assert sl.tolist() == lens.tolist() == [43, 43, 13]
        no_error()


def test_pages_that_two_sequences_share():
    """A prefix in shared pages: read by both sequences' decodes and evictions, each with its own weights."""
    rng = np.random.default_rng(35)
    c = Cache(rng, 2, 2, 16, 12, 64, more=4)
    c.table[1, :6] = c.table[0, :6]
    c.upload()
    q, rho = bf16(rng.standard_normal((2, 4, 64))), bf16(rng.standard_normal((2, 4, 64)))
    _, _, w = check_decode(c, q, rho, [192, 150])
    run_evict(c, w.cpu().numpy(), [192, 150], 60, 5, 4)
    no_error()


def test_captured_and_replayed():
    """A step (append, decode with weights, eviction) captured once and replayed equals the eager calls, twice."""
    rng = np.random.default_rng(31)
    B, Hkv, G, ps, mp, d = 2, 2, 4, 16, 90, 64
    c = Cache(rng, B, Hkv, ps, mp, d, more=20)
    k, v = (bf16(rng.standard_normal((B, Hkv, 3, d))).to(DEV) for _ in range(2))
    q, rho = (bf16(rng.standard_normal((B, Hkv * G, d))).to(DEV) for _ in range(2))
    sl = torch.tensor([1400, 77], dtype=torch.int32, device=DEV)
    ns, ns2 = torch.zeros_like(sl), torch.zeros_like(sl)
    w = torch.zeros((B, Hkv, mp * ps), device=DEV)
    y, lse = torch.empty((B, Hkv * G, d), device=DEV), torch.empty((B, Hkv * G), device=DEV)
    kept = torch.zeros((B, Hkv, 300), dtype=torch.int32, device=DEV)
    w2 = torch.zeros((B, Hkv, 20 * ps), device=DEV)

    def step():
        plx.parallax_kv_append(k, v, c.kp, c.vp, c.tab, sl, kexp=c.ke, vexp=c.ve, new_seqlens=ns, wacc=w)
        plx.parallax_decode_paged_q8(q, rho, c.kp, c.vp, c.ke, c.ve, c.tab, ns, wacc=w, y=y, lse=lse)
        plx.parallax_kv_evict(c.kp, c.vp, c.tab, ns, w, c.tab2, 300, 20, kexp=c.ke, vexp=c.ve, new_seqlens=ns2,
                              kept=kept, new_wacc=w2)

    def state():
        return [t.clone() for t in (c.kp.view(torch.uint8), c.vp.view(torch.uint8), c.ke, c.ve, w, y, lse, ns, ns2, kept, w2)]

    start = [c.kp.view(torch.uint8).clone(), c.vp.view(torch.uint8).clone(), c.ke.clone(), c.ve.clone()]
    step()
    torch.cuda.synchronize()
    eager = []

    def reset(i):
        for t, s in zip((c.kp.view(torch.uint8), c.vp.view(torch.uint8), c.ke, c.ve), start):
            t.copy_(s)
        w.zero_()
        k.mul_(1 + i)
        q.neg_()

    for i in range(2):
        reset(i)
        step()
        eager.append(state())
    g = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]      # two graphs of the same step, replayed in turn
    for graph in g:
        with torch.cuda.graph(graph):
            step()
    k.div_(2)
    for i in range(2):
        reset(i)
        g[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(state(), eager[i]):
            assert torch.equal(a, b)
    no_error()


def test_streams():
    """Calls on two streams at once, each with its own tensors, given and current stream alike."""
    rng = np.random.default_rng(32)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    jobs = []
    for i in range(2):
        c = Cache(rng, 4, 2, 64, 16 + 8 * i, 128)
        q = bf16(rng.standard_normal((4, 8, 128))).to(DEV)
        sl = torch.tensor([c.table.shape[1] * 64, 700, 3, 0], dtype=torch.int32, device=DEV)
        jobs.append((c, q, sl))
    alone = [plx.parallax_decode_paged_q8(q, q, c.kp, c.vp, c.ke, c.ve, c.tab, sl) for c, q, sl in jobs]
    acc = [torch.zeros((4, 2, c.table.shape[1] * 64), device=DEV) for c, _, _ in jobs]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        c, q, sl = jobs[0]
        outs[0].append(plx.parallax_decode_paged_q8(q, q, c.kp, c.vp, c.ke, c.ve, c.tab, sl, wacc=acc[0], stream=s1))
        c, q, sl = jobs[1]
        with torch.cuda.stream(s2):
            outs[1].append(plx.parallax_decode_paged_q8(q, q, c.kp, c.vp, c.ke, c.ve, c.tab, sl, wacc=acc[1]))
    torch.cuda.synchronize()
    for i in range(2):
        for y, lse in outs[i]:
            assert torch.equal(y, alone[i][0]) and torch.equal(lse, alone[i][1])
        n = jobs[i][2].cpu().numpy()
        total = acc[i].sum(2).cpu().numpy()
        assert np.allclose(total[n > 0], 20 * 4, rtol=1e-4) and np.all(total[n == 0] == 0)


def test_offsets_past_32_bits():
    """Pages past the 4 GiB mark of the pool give what the same pages give at its start."""
    rng = np.random.default_rng(33)
    B, Hkv, ps, mp, d = 2, 8, 128, 6, 128
    c = Cache(rng, B, Hkv, ps, mp, d, more=3, spare=0)
    n = (1 << 32) // (Hkv * ps * d) + c.n + 5
    far = n - c.n
    pools = []
    for near in (c.kp, c.vp):
        p = torch.zeros((n, Hkv, ps, d), dtype=torch.uint8, device=DEV)
        p[far:] = near.view(torch.uint8)
        pools.append(p.view(E4M3))
    exps = []
    for near in (c.ke, c.ve):
        e = torch.zeros((n, Hkv, ps // 16), dtype=torch.int8, device=DEV)
        e[far:] = near
        exps.append(e)
    q = bf16(rng.standard_normal((B, 16, d))).to(DEV)
    k = bf16(rng.standard_normal((B, Hkv, 21, d))).to(DEV)
    sl = torch.tensor([700, 100], dtype=torch.int32, device=DEV)
    got = []
    for kp, vp, ke, ve, off in ((c.kp, c.vp, c.ke, c.ve, 0), (*pools, *exps, far)):
        t, t2 = c.tab + off, c.tab2 + off
        w = torch.zeros((B, Hkv, mp * ps), device=DEV)
        ns = plx.parallax_kv_append(k, k, kp, vp, t, sl, kexp=ke, vexp=ve)
        y, lse = plx.parallax_decode_paged_q8(q, q, kp, vp, ke, ve, t, ns, wacc=w)
        ns2, kept, nw = plx.parallax_kv_evict(kp, vp, t, ns, w, t2, 300, 40, kexp=ke, vexp=ve)
        got.append((ns, y, lse, w, ns2, kept, nw, kp.view(torch.uint8)[off:], vp.view(torch.uint8)[off:], ke[off:], ve[off:]))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    no_error()


@pytest.mark.parametrize("split", ["ranges", "ctas", "warps"])
def test_forced_wait_timeout_is_reported_and_recoverable(split, monkeypatch):
    """Test hook: no warp copies its first tile, so its bounded wait expires; the next call is right again."""
    rng = np.random.default_rng(34)
    B, mp = (300, 2) if split == "warps" else (2, 30)
    c = Cache(rng, B, 2, 16, mp, 128)
    if split == "ranges":
        c.widen(2400)
    q = bf16(rng.standard_normal((B, 4, 128))).to(DEV)
    sl = torch.tensor([mp * 16, 20] * (B // 2), dtype=torch.int32, device=DEV)

    def call():
        w = torch.zeros((B, 2, c.table.shape[1] * 16), device=DEV)
        return plx.parallax_decode_paged_q8(q, q, c.kp, c.vp, c.ke, c.ve, c.tab, sl, wacc=w)[0]

    ok = call()
    no_error()
    monkeypatch.setenv("PARALLAX_DEBUG_FLAGS", "2")
    monkeypatch.setenv("PARALLAX_WAIT_TIMEOUT_MS", "50")
    call()
    assert plx.parallax_last_device_error() == 7
    monkeypatch.delenv("PARALLAX_DEBUG_FLAGS")
    monkeypatch.delenv("PARALLAX_WAIT_TIMEOUT_MS")
    y = call()
    no_error()
    assert torch.equal(y, ok)

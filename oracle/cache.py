"""fp64 oracle of the paged cache: its e4m3 format, the write, the decode with accumulated weights, the eviction.

Plain numpy in the order of the definitions, one sequence and KV head at a time; shares no code
with the CUDA path.  Codes are uint8 arrays, values fp64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16
EMIN, EMAX = -120, 120


def _code_table():
    v = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-x if s else x)
    return v


CODES = _code_table()


def encode(x):
    """e4m3 codes of fp64 x with |x| <= 448: nearest, ties to the even code, sign kept on zero; else NaN's."""
    x = np.asarray(x, np.float64)
    out = np.full(x.shape, 0x7F, np.uint8)
    ok = np.isfinite(x) & (np.abs(x) <= 448.0)
    a, pos = np.abs(x[ok]), CODES[:127]
    hi = np.clip(np.searchsorted(pos, a), 1, 126)          # pos[hi - 1] < a <= pos[hi] (a = 0: code 0 below)
    lo = hi - 1
    down, up = a - pos[lo], pos[hi] - a
    c = np.where(down < up, lo, np.where(up < down, hi, np.where(lo % 2 == 0, lo, hi)))
    out[ok] = c.astype(np.uint8) | (np.signbit(x[ok]).astype(np.uint8) << 7)
    return out


def exponent(amax: float) -> int:
    """The smallest e in [EMIN, EMAX] with amax <= 448 2^e."""
    for e in range(EMIN, EMAX + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return EMAX


def values(codes, exps):
    """[.., page_size, d] codes and [.., page_size / 16] exponents -> fp64."""
    e = np.repeat(np.asarray(exps, np.float64), BLOCK, axis=-1)[..., None]
    return CODES[np.asarray(codes)] * 2.0 ** e


def append(k, v, kpages, vpages, kexp, vexp, table, seqlens, counts=None, wacc=None):
    """Writes k, v [B, Hkv, T, d] fp64 into copies; returns (kpages, vpages, kexp, vexp, new_seqlens, wacc).

    e4m3 pages are uint8 codes with exponents; kexp None: pages hold the values themselves.
    """
    B, Hkv, T, d = k.shape
    ps = kpages.shape[2]
    pages, exps = [kpages.copy(), vpages.copy()], [None if e is None else e.copy() for e in (kexp, vexp)]
    lens = np.array(seqlens, np.int32)
    wacc = None if wacc is None else wacc.copy()
    for b in range(B):
        n = T if counts is None else int(counts[b])
        start = int(seqlens[b])
        lens[b] = start + n
        for h in range(Hkv):
            if wacc is not None:
                wacc[b, h, start:start + n] = 0.0
            for x, pg, ex in zip((k, v), pages, exps):
                for blk in range(start // BLOCK, -(-(start + n) // BLOCK) if n else 0):
                    t = np.arange(max(start, blk * BLOCK), min(start + n, (blk + 1) * BLOCK))
                    page, row0 = int(table[b, blk * BLOCK // ps]), blk * BLOCK % ps
                    new = x[b, h, t - start]
                    if ex is None:
                        pg[page, h, t % ps] = new
                        continue
                    e = exponent(np.max(np.abs(new[np.isfinite(new)]), initial=0.0))
                    there = int(t[0]) - blk * BLOCK
                    if there:
                        was = int(ex[page, h, row0 // BLOCK])
                        e = max(e, was)
                        old = pg[page, h, row0:row0 + there]
                        moved = encode(CODES[old] * 2.0 ** (was - e))
                        pg[page, h, row0:row0 + there] = moved
                    ex[page, h, row0 // BLOCK] = e
                    pg[page, h, t % ps] = encode(new * 2.0 ** -e)
    return pages[0], pages[1], exps[0], exps[1], lens, wacc


def rows(pages, table_row, n):
    """The first n rows of a sequence, [Hkv, n, d]."""
    ps = pages.shape[2]
    t = np.arange(n)
    return pages[np.asarray(table_row)[t // ps], :, t % ps].transpose(1, 0, 2)


def decode(q, rho, kpages, vpages, table, seqlens, wacc=None):
    """y [B, Hq, d], lse [B, Hq], wacc (a copy with the weights added); pages hold values, rho may be None."""
    B, Hq, d = q.shape
    Hkv = kpages.shape[1]
    G = Hq // Hkv
    y, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    wacc = None if wacc is None else np.array(wacc, np.float64)
    for b in range(B):
        n = int(seqlens[b])
        if n == 0:
            continue
        k, v = rows(kpages, table[b], n), rows(vpages, table[b], n)
        for h in range(Hq):
            kk, vv = k[h // G], v[h // G]
            z = kk @ q[b, h] / np.sqrt(d)
            lse[b, h] = z.max() + np.log(np.exp(z - z.max()).sum())
            s = np.exp(z - lse[b, h])
            o = s @ vv
            y[b, h] = o
            if rho is not None:
                a = kk @ rho[b, h]
                y[b, h] = o - (s * (a - s @ a)) @ (vv - o)
            if wacc is not None:
                wacc[b, h // G, :n] += s
    return y, lse, wacc


def evict(kpages, vpages, kexp, vexp, table, seqlens, wacc, new_table, budget, recent, kept, new_wacc):
    """Copies of (kpages, vpages, kexp, vexp) with the kept rows moved, new_seqlens, and kept, new_wacc filled."""
    B, Hkv, cap = wacc.shape
    ps = kpages.shape[2]
    src, dst = [kpages, vpages], [kpages.copy(), vpages.copy()]
    sexp, dexp = [kexp, vexp], [None if e is None else e.copy() for e in (kexp, vexp)]
    kept, new_wacc, lens = kept.copy(), new_wacc.copy(), np.array(seqlens, np.int32)
    for b in range(B):
        L = int(seqlens[b])
        n = min(L, budget)
        r = min(recent, n)
        lens[b] = n
        for h in range(Hkv):
            w = np.where(np.isnan(wacc[b, h, :L - r]), -np.inf, wacc[b, h, :L - r])
            heavy = sorted(range(L - r), key=lambda t: (-w[t], t))[:n - r]
            keep = sorted(heavy) + list(range(L - r, L))
            kept[b, h, :n] = keep
            new_wacc[b, h, :n] = wacc[b, h, keep]
            for i0 in range(0, n, BLOCK):
                t = np.array(keep[i0:i0 + BLOCK], np.int64)
                pg, page = table[b][t // ps], int(new_table[b, i0 // ps])
                r0 = i0 % ps
                for s, d_, se, de in zip(src, dst, sexp, dexp):
                    x = s[pg, h, t % ps]
                    if se is not None:
                        e = se[pg, h, t % ps // BLOCK].astype(np.int64)
                        de[page, h, r0 // BLOCK] = e.max()
                        x = np.where((e == e.max())[:, None], x, encode(CODES[x] * 2.0 ** (e - e.max())[:, None]))
                    d_[page, h, r0:r0 + t.size] = x
    return dst[0], dst[1], dexp[0], dexp[1], lens, kept, new_wacc

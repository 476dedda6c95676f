"""Every way the eviction finds its tokens: one CTA per head or a cluster of 2, 4 or 8, with the keys in
registers or read again for each digit; with ties, NaN and short sequences in each."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_cache import DEV, Cache, no_error, run_evict

pytestmark = pytest.mark.gpu

# tokens of a table and heads: a cluster grows while the table is longer than 4096 tokens per CTA and the heads
# are fewer than two per SM; a CTA whose share is at most 4096 tokens holds its keys
PLANS = {"one CTA": (2048, 6), "one CTA, keys read again": (4352, 320), "cluster of 2": (5120, 6),
         "cluster of 4": (10240, 6), "cluster of 8": (17408, 6), "cluster of 8, keys read again": (33280, 6)}


def weights(rng, kind, B, cap):
    if kind == "distinct":
        return np.exp(2 * rng.standard_normal((B, 1, cap))).astype(np.float32)
    if kind == "equal":
        return np.full((B, 1, cap), 0.75, np.float32)
    if kind == "few values":
        return rng.choice(np.array([np.nan, -np.inf, 0.0, -0.0, 1.0, 2.0], np.float32), (B, 1, cap))
    # ties at the border only, spread over the whole table: a third larger, a third equal, a third smaller
    return rng.permuted(np.tile(np.arange(cap, dtype=np.float32) % 3, (B, 1, 1)), axis=2)


@pytest.mark.parametrize("kind", ["distinct", "equal", "few values", "ties at the border"])
@pytest.mark.parametrize("plan", list(PLANS))
def test_selection(plan, kind):
    cap, heads = PLANS[plan]
    rng = np.random.default_rng(cap + len(kind))
    B, ps, d = 6, 256, 64
    mp, budget = cap // ps, cap // 2 - 77
    mp2 = -(-budget // ps)
    c = Cache(rng, B, 1, ps, mp, d, q8=False, more=mp2, spare=0)
    sl = [cap, cap - 5, 0, 9, budget, budget + 1]              # the longest, empty, short, and at the budget
    if heads > B:                                              # the others name no page and are empty
        c.table = np.concatenate([c.table, np.full((heads - B, mp), -9, np.int32)])
        c.table2 = np.concatenate([c.table2, np.full((heads - B, mp2), -9, np.int32)])
        c.B = heads
        c.tab, c.tab2 = torch.from_numpy(c.table).to(DEV), torch.from_numpy(c.table2).to(DEV)
        sl += [0] * (heads - B)
    w = np.zeros((c.B, 1, cap), np.float32)
    w[:B] = weights(rng, kind, B, cap)
    for recent in (0, 100, budget):
        run_evict(c, w, sl, budget, recent, mp2)
        c.upload()
    no_error()

"""Refusals of the paged-cache calls: the C entry points' host checks and the binding's (no GPU)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import softmax_learned_covariance_b200 as plx
from tests.test_abi import A16, L, MIS  # noqa: F401

P = ctypes.c_void_p
B16 = P(0x20000)
C16 = P(0x30000)


def test_decode_cache_host_validation(L):
    def q8(q=A16, rho=A16, kp=A16, vp=A16, ke=A16, ve=A16, bt=A16, sl=A16, y=A16, lse=None, w=None, B=2, Hq=4, Hkv=2,
           ps=64, mp=4, npg=8, d=128, i=1, o=0):
        return L.parallax_decode_paged_q8(q, rho, kp, vp, ke, ve, bt, sl, y, lse, w, B, Hq, Hkv, ps, mp, npg, d, i, o,
                                          None)
    for missing in ("q", "kp", "vp", "ke", "ve", "bt", "sl", "y"):
        assert q8(**{missing: None}) == 1, missing
    for bad in (dict(Hq=3), dict(Hq=1), dict(ps=48), dict(ps=8), dict(ps=8192), dict(mp=0), dict(npg=0), dict(d=96),
                dict(B=0), dict(Hkv=0), dict(mp=1 << 30), dict(npg=1 << 30, Hkv=2), dict(B=1 << 30, mp=1 << 24)):
        assert q8(**bad) == 2, bad
    for mis in ("q", "rho", "kp", "vp", "y", "w"):
        assert q8(**{mis: MIS}) == 3, mis
    assert q8(lse=P(0x10002)) == 3
    assert q8(i=0) == 4 and q8(i=2) == 4 and q8(o=2) == 4

    def acc(w=A16, rho=None, d=128, o=1):
        return L.parallax_decode_paged_acc(A16, rho, A16, A16, A16, A16, A16, None, w, 2, 4, 2, 64, 4, 8, d, 1, o, None)
    assert acc(w=None) == 1
    assert acc(d=32) == 2
    assert acc(w=MIS) == 3
    assert acc(o=3) == 4


def test_kv_append_host_validation(L):
    def ap(k=A16, v=A16, ks=None, vs=None, kp=A16, vp=A16, ke=A16, ve=A16, bt=A16, sl=A16, cn=None, ns=None, w=None, B=2,
           Hkv=2, T=5, ps=64, mp=4, npg=8, d=128, i=1, c=2):
        return L.parallax_kv_append(k, v, ks, vs, kp, vp, ke, ve, bt, sl, cn, ns, w, B, Hkv, T, ps, mp, npg, d, i, c, None)
    for missing in ("k", "v", "kp", "vp", "bt", "sl", "ke", "ve"):
        assert ap(**{missing: None}) == 1, missing
    for bad in (dict(T=0), dict(T=-1), dict(ps=20), dict(d=256), dict(B=0), dict(mp=0), dict(npg=0),
                dict(B=1 << 20, T=1 << 20)):
        assert ap(**bad) == 2, bad
    for mis in ("k", "v", "kp", "vp", "w"):
        assert ap(**{mis: MIS}) == 3, mis
    odd = (ctypes.c_longlong * 3)(1024, 128, 4)
    assert ap(ks=ctypes.addressof(odd)) == 3
    assert ap(i=0) == 4 and ap(c=0) == 4
    assert ap(c=1) == 4                                # a bf16 cache has no exponents
    assert ap(ns=A16) == 5                             # new_seqlens is another array than seqlens
    assert ap(sl=B16, cn=A16, ns=A16) == 5


def test_kv_evict_host_validation(L):
    def ev(kp=A16, vp=A16, ke=A16, ve=A16, bt=A16, sl=A16, w=A16, nt=B16, ns=B16, kept=A16, nw=None, B=2, Hkv=2, ps=64,
           mp=4, nmp=2, npg=8, d=128, budget=100, recent=10, c=2):
        return L.parallax_kv_evict(kp, vp, ke, ve, bt, sl, w, nt, ns, kept, nw, B, Hkv, ps, mp, nmp, npg, d, budget,
                                   recent, c, None)
    for missing in ("kp", "vp", "ke", "bt", "sl", "w", "nt", "ns", "kept"):
        assert ev(**{missing: None}) == 1, missing
    for bad in (dict(budget=0), dict(budget=129), dict(recent=-1), dict(recent=101), dict(nmp=0), dict(ps=24), dict(d=1)):
        assert ev(**bad) == 2, bad
    assert ev(w=MIS) == 3 and ev(vp=MIS) == 3
    assert ev(c=1) == 4 and ev(c=0) == 4
    # nothing in place
    assert ev(nt=A16) == 5 and ev(ns=A16) == 5 and ev(nw=A16) == 5


def test_binding_refuses_before_the_library():
    """Wrong dtypes, shapes and devices are Python errors; nothing reaches the device."""
    codes = torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    table, sl = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32)
    q, e = torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.zeros((4, 2, 1), dtype=torch.int8)
    with pytest.raises(ValueError):                    # CPU tensors
        plx.parallax_decode_paged_q8(q, None, codes, codes, e, e, table, sl)
    with pytest.raises(TypeError):
        plx.parallax_decode_paged_q8(q, None, codes.float(), codes, e, e, table, sl)
    with pytest.raises(TypeError):
        plx.parallax_decode_paged_acc(q, None, codes, codes, table, sl, torch.zeros((1, 2, 32)))
    with pytest.raises(ValueError):
        plx.parallax_decode_paged_acc(q, None, codes.to(torch.bfloat16), codes, table, sl, None)
    with pytest.raises(ValueError):
        plx.parallax_kv_append(q[:, :, None], q[:, :, None], codes, codes, table, sl, kexp=e, vexp=e)
    with pytest.raises(ValueError):
        plx.parallax_kv_evict(codes, codes, table, sl, torch.zeros((1, 2, 32)), table, 16, 0, kexp=e, vexp=e)


def test_cache_decode_schedule(tmp_path):
    """Every quad of every item belongs to one CTA's range, ranges are even, and the parts of a cut item are
    found where their CTAs left them."""
    import os
    import shutil
    import subprocess

    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    csrc = os.path.join(os.path.dirname(plx.__file__), "csrc")
    src = tmp_path / "sched.cpp"
    src.write_text(r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "decode_sched.h"
using namespace plx;
int main() {
    srand(1);
    for (int rep = 0; rep < 400; ++rep) {
        const int ctas = 1 + rand() % 700, items = 1 + rand() % 300;
        std::vector<long long> first(1, 0);
        for (int i = 0; i < items; ++i) first.push_back(first.back() + (rand() % 3 ? rand() % (rep % 50 + 1) : 0));
        const long long total = first.back();
        if (total == 0) continue;
        const int n = sched_ctas(total, ctas);
        if (n < 1 || n > ctas) return 1;
        std::vector<int> who(total, -1);
        for (int c = 0; c < n; ++c) {
            const long long a = sched_start(c, total, n), b = sched_start(c + 1, total, n);
            if (b <= a || b - a > total / n + 1) return 2;
            for (long long x = a; x < b; ++x) {
                if (who[x] != -1 || sched_owner(x, total, n) != c) return 3;
                who[x] = c;
            }
        }
        std::vector<int> slot_item(2 * n, -1);
        for (int i = 0; i < items; ++i) {
            if (first[i] == first[i + 1]) continue;
            const int c0 = who[first[i]], c1 = who[first[i + 1] - 1];
            const int parts = sched_owner(first[i + 1] - 1, total, n) - c0 + 1;
            if (parts != c1 - c0 + 1) return 4;
            if (parts == 1) continue;
            for (int c = c0; c <= c1; ++c) {
                const int slot = sched_slot(c, c == c0);      // as the CTA writes it
                if (slot != sched_part(c0, c - c0)) return 5;  // as the merge reads it
                if (slot < 0 || slot >= 2 * n || slot_item[slot] != -1) return 6;
                slot_item[slot] = i;
            }
        }
    }
    // the largest batches stay within 64 bits
    const long long total = (1ll << 36) / 64;
    return sched_owner(total - 1, total, 592) == 591 && sched_start(592, total, 592) == total ? 0 : 7;
}
""")
    exe = tmp_path / "sched"
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)])
    assert subprocess.call([str(exe)]) == 0

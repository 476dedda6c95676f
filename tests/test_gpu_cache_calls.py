"""The paged-cache calls beside their results: what they clear, what a failed one leaves, other threads."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess
import sys
import threading
import time

import numpy as np
import pytest
import torch

import softmax_learned_covariance_b200 as plx
from tests.test_gpu_cache import DEV, Cache, bf16, no_error, run_append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q8", [True, False])
def test_append_clears_the_weights_of_tokens_on_bad_pages(q8):
    """The accumulator belongs to the sequence: new tokens start at 0 there although their page is not written."""
    rng = np.random.default_rng(50)
    B, Hkv, T, d = 3, 2, 20, 64
    c = Cache(rng, B, Hkv, 16, 3, d, q8)
    c.table[1, 1] = c.n
    c.table[2, 0] = -1
    c.upload()
    w = torch.ones((B, Hkv, 48), device=DEV)
    k = bf16(rng.standard_normal((B, Hkv, T, d))).to(DEV)
    ns = run_append(c, k, k, [5, 7, 0], [20, 20, 3], w)
    assert ns.tolist() == [25, 27, 3]
    assert plx.parallax_last_device_error() == 8
    want = np.ones((B, Hkv, 48), np.float32)
    for b, (s, n) in enumerate(((5, 20), (7, 20), (0, 3))):
        want[b, :, s:s + n] = 0.0
    assert np.array_equal(w.cpu().numpy(), want)


def test_a_call_that_fails_leaves_nothing_to_the_next():
    """Scores for 2^35 table slots (a terabyte) cannot be had: that call reports it, the next one is a success."""
    rng = np.random.default_rng(51)
    c = Cache(rng, 2, 2, 16, 4, 64)
    q = bf16(rng.standard_normal((2, 16, 64))).to(DEV)
    sl = torch.tensor([64, 10] + [0] * 14, dtype=torch.int32, device=DEV)
    w = torch.zeros((2, 2, 64), device=DEV)
    y = torch.empty((2, 16, 64), device=DEV)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    L = plx.lib()

    def call(mp, B, Hkv, Hq):
        return L.parallax_decode_paged_q8(p(q), None, p(c.kp), p(c.vp), p(c.ke), p(c.ve), p(c.tab), p(sl), p(y), None,
                                          p(w), B, Hq, Hkv, 16, mp, c.n, 64, plx.BF16, plx.F32,
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert call(4, 2, 2, 16) == 0
    ok = y.clone()
    assert call(1 << 26, 16, 2, 16) == 6             # no launch: the scratch comes first
    y.zero_()
    assert call(4, 2, 2, 16) == 0
    assert torch.equal(y, ok)
    no_error()


def test_other_python_threads_run_during_a_call(tmp_path):
    """A call that waits inside the library (here a stand-in that sleeps) does not hold the interpreter."""
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "slow.cpp"
    src.write_text('#include <unistd.h>\nextern "C" int slow() { usleep(400000); return 0; }\n')
    so = str(tmp_path / "slow.so")
    subprocess.check_call([gxx, "-shared", "-fPIC", "-o", so, str(src)])
    slow = ctypes.cast(ctypes.CDLL(so).slow, ctypes.c_void_p).value
    rng = np.random.default_rng(52)
    c = Cache(rng, 1, 2, 16, 2, 64, more=1)
    q = bf16(rng.standard_normal((1, 2, 64))).to(DEV)
    k = bf16(rng.standard_normal((1, 2, 1, 64))).to(DEV)
    sl = torch.tensor([16], dtype=torch.int32, device=DEV)
    w = torch.zeros((1, 2, 32), device=DEV)
    calls = [lambda: plx.parallax_decode_paged_q8(q, None, c.kp, c.vp, c.ke, c.ve, c.tab, sl),
             lambda: plx.parallax_kv_append(k, k, c.kp, c.vp, c.tab, sl, kexp=c.ke, vexp=c.ve),
             lambda: plx.parallax_kv_evict(c.kp, c.vp, c.tab, sl, w, c.tab2, 8, 0, kexp=c.ke, vexp=c.ve)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    L = plx.lib()
    real = [ctypes.cast(f, ctypes.c_void_p).value for f in
            (L.parallax_decode_paged_q8, L.parallax_decode_paged_acc, L.parallax_kv_append, L.parallax_kv_evict)]
    stop, beats = threading.Event(), []

    def beat():
        while not stop.is_set():
            beats.append(time.monotonic())
            time.sleep(0.005)

    thread = threading.Thread(target=beat)
    native = plx._native()
    native.bind(slow, slow, slow, slow)
    try:
        thread.start()
        seen = []
        for f in calls:
            start = time.monotonic()
            f()
            end = time.monotonic()
            assert end - start >= 0.39
            seen.append(sum(start + 0.05 < t < end - 0.05 for t in list(beats)))
    finally:
        stop.set()
        thread.join()
        native.bind(*real)
    assert min(seen) >= 5                            # 60 beats of 5 ms fit, none while the interpreter is held


def test_arrays_beside_one_another_are_not_over_one_another():
    """Lengths, exponents and accumulators that are parts of one buffer each, next to each other."""
    rng = np.random.default_rng(53)
    B, Hkv, ps, mp, d = 4, 2, 16, 3, 64
    c = Cache(rng, B, Hkv, ps, mp, d, more=1)
    k = bf16(rng.standard_normal((B, Hkv, 5, d))).to(DEV)
    sl = torch.tensor([0, 7, 16, 40], dtype=torch.int32, device=DEV)
    w = torch.rand((B, Hkv, mp * ps), device=DEV)

    def serve(kp, vp, ke, ve, lens, sl, ns, w, nw):
        plx.parallax_kv_append(k, k, kp, vp, c.tab, sl, kexp=ke, vexp=ve, new_seqlens=ns, wacc=w)
        plx.parallax_kv_evict(kp, vp, c.tab, ns, w, c.tab2, 16, 2, kexp=ke, vexp=ve, new_seqlens=lens, new_wacc=nw)
        return [t.clone() for t in (kp.view(torch.uint8), vp.view(torch.uint8), ke, ve, lens, ns, w, nw)]

    apart = serve(c.kp.clone(), c.vp.clone(), c.ke.clone(), c.ve.clone(), torch.zeros_like(sl), sl.clone(),
                  torch.zeros_like(sl), w.clone(), torch.zeros((B, Hkv, ps), device=DEV))
    pages, exps = torch.stack([c.kp.view(torch.uint8), c.vp.view(torch.uint8)]).view(c.kp.dtype), torch.stack([c.ke, c.ve])
    lens = torch.stack([torch.zeros_like(sl), sl, torch.zeros_like(sl)])
    both = torch.cat([w.flatten(), torch.zeros(B * Hkv * ps, device=DEV)])
    beside = serve(pages[0], pages[1], exps[0], exps[1], lens[0], lens[1], lens[2], both[:w.numel()].view_as(w),
                   both[w.numel():].view(B, Hkv, ps))
    for a, b in zip(apart, beside):
        assert torch.equal(a, b)
    no_error()


FIRST_CALL = """
import sys
import torch
import softmax_learned_covariance_b200 as plx
gen = torch.Generator(device="cuda:0").manual_seed(1)
rand = lambda *shape: torch.randn(shape, device="cuda:0", generator=gen)
ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda:0")
pages = [rand(8, 2, 16, 64) for _ in range(2)]
k8, v8 = (x.to(torch.float8_e4m3fn) for x in pages)
kb, vb = (x.to(torch.bfloat16) for x in pages)
ke, ve = (torch.zeros((8, 2, 1), dtype=torch.int8, device="cuda:0") for _ in range(2))
table, new_table, sl = ints(*range(6)).view(2, 3), ints(6, 7).view(2, 1), ints(40, 17)
q, k, w = rand(2, 8, 64).to(torch.bfloat16), rand(2, 2, 3, 64).to(torch.bfloat16), rand(2, 2, 48).abs()
call = {
    "append": lambda: (plx.parallax_kv_append(k, k, k8, v8, table, sl, kexp=ke, vexp=ve), k8.view(torch.uint8)),
    "decode": lambda: (*plx.parallax_decode_paged_q8(q, q, k8, v8, ke, ve, table, sl, wacc=w), w),
    "evict": lambda: plx.parallax_kv_evict(k8, v8, table, sl, w, new_table, 16, 3, kexp=ke, vexp=ve),
    "paged": lambda: plx.parallax_decode_paged(q, q, kb, vb, table, sl),
}[sys.argv[1]]
state = [t.clone() for t in (k8.view(torch.uint8), v8.view(torch.uint8), ke, ve, w)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
got = [t.clone() for t in out]
for t, s in zip((k8.view(torch.uint8), v8.view(torch.uint8), ke, ve, w), state):
    t.copy_(s)
for a, b in zip(got, call()):
    assert torch.equal(a, b)
assert plx.parallax_last_device_error() == 0
print("fine")
"""


@pytest.mark.parametrize("op", ["append", "decode", "evict", "paged"])
def test_the_first_call_of_a_process_may_be_captured(op):
    """What the library sets up on a device is no part of the capture and does not end it."""
    here = os.path.dirname(os.path.dirname(os.path.abspath(plx.__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL, op], cwd=here, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr

"""Cases of the serving loop on a paged cache: writing tokens into it, attending to it, evicting from it.

The cache is a pool of pages [num_pages, Hkv, page_size, d] that a table maps per sequence.  Its rows are
bf16, or e4m3 codes with one power-of-two exponent per block of 16 tokens and KV head (value = code 2^exp).

  append  new keys and values of each sequence go behind its last token (prompt chunks, single tokens)
  decode  one query token per sequence: Parallax attention y = o - (m - o abar), or softmax attention
          without a probe; optionally adds each cached token's attention weight, summed over the query
          heads of its KV head, to an accumulator
  evict   keeps, per sequence and KV head, the newest tokens and the heaviest others up to a budget, in
          order, in pages of a second table

``run`` is the plain form (elementary torch operations, fp32) where ``own`` is false and the framework's
calls where it is true; ``exact`` is the definition in fp64, one sequence at a time.
"""
import math

import torch

own = False

BLOCK = 16          # tokens of a block that share an exponent
EMIN, EMAX = -120, 120
CODE_MAX = 448.0    # largest e4m3 value


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the write of one decode step of a serving batch: launch latency
        dict(name="append 1 token b64", op="append", cache="e4m3", B=64, Hkv=8, d=128, page=64, T=1, lo=2048, hi=4095,
             full=True),
        # a prompt of the 1.7B layer shape (16 heads, 4096 tokens, batch 8) entering an empty cache
        dict(name="append prompt b8 t4096", op="append", cache="e4m3", B=8, Hkv=16, d=128, page=64, T=4096, lo=0, hi=0,
             full=True),
        # ragged chunks that start inside a block, small pages, head dim 64
        dict(name="append ragged d64", op="append", cache="e4m3", B=5, Hkv=3, d=64, page=16, T=777, lo=5, hi=1000,
             full=False),
        # a single short chat: launch latency
        dict(name="decode b1 ctx128", op="decode", cache="e4m3", B=1, Hq=16, Hkv=16, d=128, page=16, lo=128, hi=128,
             rho=True, acc=False),
        # the serving shape of the paged benchmark, weights accumulated for a later eviction
        dict(name="decode b64 gqa acc", op="decode", cache="e4m3", B=64, Hq=32, Hkv=8, d=128, page=64, lo=2048,
             hi=4096, rho=True, acc=True),
        # one KV head per query head, full-length cache (the headline decode's shape)
        dict(name="decode b64 mha", op="decode", cache="e4m3", B=64, Hq=16, Hkv=16, d=128, page=64, lo=4096, hi=4096,
             rho=True, acc=False),
        # one long document, softmax attention: the split over the cache's length
        dict(name="softmax b1 ctx32768", op="decode", cache="e4m3", B=1, Hq=32, Hkv=8, d=128, page=128, lo=32768,
             hi=32768, rho=False, acc=False),
        # long documents in a batch: bandwidth
        dict(name="decode b16 ctx32768", op="decode", cache="e4m3", B=16, Hq=16, Hkv=16, d=128, page=64, lo=16384,
             hi=32768, rho=True, acc=False),
        # odd everything: seven query heads per KV head, an empty sequence, lengths that end inside a page
        dict(name="decode odd d64 acc", op="decode", cache="e4m3", B=3, Hq=21, Hkv=3, d=64, page=16, lo=0, hi=1501,
             rho=True, acc=True),
        # the bf16 cache with weights accumulated
        dict(name="decode bf16 gqa acc", op="decode", cache="bf16", B=64, Hq=32, Hkv=8, d=128, page=64, lo=2048,
             hi=4096, rho=True, acc=True),
        # halving the caches of a serving batch
        dict(name="evict b64 half", op="evict", cache="e4m3", B=64, Hkv=8, d=128, page=64, lo=3000, hi=4096,
             budget=2048, recent=256),
        # one long document cut to an eighth, bf16 cache
        dict(name="evict b1 long bf16", op="evict", cache="bf16", B=1, Hkv=8, d=128, page=64, lo=32768, hi=32768,
             budget=4096, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: at most the cache of the largest listed one."""
    op = rng.choice(["append", "decode", "decode", "evict"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["e4m3", "e4m3", "e4m3", "bf16"])
    Hkv = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
    B = _log(rng, 1, 96)
    room = {"append": 5e5, "decode": 3e6, "evict": 1.5e6}[op]   # rows (tokens times KV heads) of the batch
    most = max(64, min(32768, int(room / (B * Hkv))))       # tokens of a sequence
    hi = _log(rng, 17, most)
    lo = rng.choice([hi, hi // 2, hi // 3, 0]) if B > 1 else hi
    if op == "append":
        return dict(op=op, cache=cache, B=B, Hkv=Hkv, d=d, page=page,
                    T=rng.choice([1, _log(rng, 2, max(3, min(4096, most)))]), lo=lo // 4, hi=hi // 4,
                    full=rng.random() < 0.5)
    if op == "decode":
        G = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 12])
        rho = rng.random() < 0.7
        acc = rng.random() < 0.5 or cache == "bf16"         # the bf16 cache's new part is the accumulation
        return dict(op=op, cache=cache, B=B, Hq=G * Hkv, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, rho=rho, acc=acc)
    budget = rng.randint(max(1, hi // 10), hi)
    return dict(op=op, cache=cache, B=B, Hkv=Hkv, d=d, page=page, lo=lo, hi=hi, budget=budget,
                recent=rng.choice([0, budget // 8, budget // 2, budget]))


def _spread(B, lo, hi):
    """B whole numbers evenly over [lo, hi] (hi for one sequence)."""
    if B == 1:
        return [hi]
    return [lo + (hi - lo) * i // (B - 1) for i in range(B)]


def _counts(case):
    return _spread(case["B"], case["T"] if case["full"] else 0, case["T"])


def work(case):
    d, Hkv, B = case["d"], case["Hkv"], case["B"]
    elem = 1 if case["cache"] == "e4m3" else 2
    exps = 2 / BLOCK if case["cache"] == "e4m3" else 0       # exponent bytes of a token's K and V
    if case["op"] == "append":
        n = sum(_counts(case)) * Hkv
        return {"bytes": n * (2 * d * (2 + elem) + exps) + 8 * B, "flops": n * 2 * d * 2}
    if case["op"] == "decode":
        n, G = sum(_spread(B, case["lo"], case["hi"])), case["Hq"] // Hkv
        per = 2 * d * elem + exps + (8 if case["acc"] else 0)
        vec = d * (6 if case["rho"] else 4) + 4              # q, rho in, y, lse out
        return {"bytes": n * Hkv * per + B * case["Hq"] * vec, "flops": n * Hkv * G * d * (8 if case["rho"] else 4)}
    lens = _spread(B, case["lo"], case["hi"])
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": Hkv * (sum(lens) * 4 + kept * (2 * (2 * d * elem + exps) + 4 + 4)), "flops": Hkv * sum(lens) * 2.0}


# ---------------------------------------------------------------- inputs
def _two_to(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest e with amax <= 448 2^e, clamped (448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875).to(x.dtype), EMIN).clamp(EMIN, EMAX).to(torch.int32)


def _pool(gen, n, Hkv, page, d, cache, channels):
    """Pages of random tokens: bf16, or e4m3 codes and their exponents."""
    dev = "cuda"
    if cache == "bf16":
        x = torch.empty((n, Hkv, page, d), dtype=torch.bfloat16, device=dev).normal_(generator=gen)
        return (x * channels.to(torch.bfloat16) if channels is not None else x), None
    codes = torch.empty((n, Hkv, page, d), dtype=torch.float8_e4m3fn, device=dev)
    exps = torch.empty((n, Hkv, page // BLOCK), dtype=torch.int8, device=dev)
    step = max(1, (64 << 20) // (Hkv * page * d))
    for i in range(0, n, step):
        k = min(step, n - i)
        x = torch.empty((k, Hkv, page // BLOCK, BLOCK, d), device=dev).normal_(generator=gen)
        if channels is not None:
            x *= channels
        e = _exponent(x.abs().amax((3, 4)))
        exps[i:i + k] = e.to(torch.int8)
        codes[i:i + k] = (x * _two_to(-e)[..., None, None]).to(torch.float8_e4m3fn).view(k, Hkv, page, d)
    return codes, exps


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    perm = torch.randperm(B, generator=gen, device=dev)
    lens = torch.tensor(_spread(B, case["lo"], case["hi"]), device=dev)[perm].to(torch.int32)
    longest = case["hi"] + (case["T"] if case["op"] == "append" else 0)
    P = max(1, -(-longest // page))
    P2 = -(-case["budget"] // page) if case["op"] == "evict" else 0
    n = B * (P + P2)
    # keys have a few channels far larger than the others, values do not
    channels = torch.ones(d, device=dev)
    channels[torch.randperm(d, generator=gen, device=dev)[: d // 32]] = 4.0
    s = dict(case=dict(case), seqlens=lens)
    s["kpages"], s["kexp"] = _pool(gen, n, Hkv, page, d, case["cache"], channels)
    s["vpages"], s["vexp"] = _pool(gen, n, Hkv, page, d, case["cache"], None)
    ids = torch.randperm(n, generator=gen, device=dev).to(torch.int32)
    s["table"] = ids[: B * P].view(B, P).contiguous()
    if case["op"] == "append":
        T = case["T"]
        s["k"] = (torch.randn((B, Hkv, T, d), generator=gen, device=dev) * channels).to(torch.bfloat16)
        s["v"] = torch.randn((B, Hkv, T, d), generator=gen, device=dev).to(torch.bfloat16)
        s["counts"] = torch.tensor(_counts(case), device=dev)[perm].to(torch.int32)
    elif case["op"] == "decode":
        s["q"] = torch.randn((B, case["Hq"], d), generator=gen, device=dev).to(torch.bfloat16)
        s["rho"] = (torch.randn((B, case["Hq"], d), generator=gen, device=dev) * 0.05).to(torch.bfloat16) \
            if case["rho"] else None
        s["wacc"] = torch.rand((B, Hkv, P * page), generator=gen, device=dev) if case["acc"] else None
    else:
        # sums of attention weights: a few heavy tokens, many light ones
        s["wacc"] = torch.exp(2.0 * torch.randn((B, Hkv, P * page), generator=gen, device=dev))
        s["table2"] = ids[B * P:].view(B, P2).contiguous()
        s["kept"] = torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device=dev)
        s["wacc2"] = torch.zeros((B, Hkv, P2 * page), device=dev)
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    if own:
        return _own(s)
    return {"append": _append, "decode": _decode, "evict": _evict}[s["case"]["op"]](s)


def _own(s):
    import softmax_learned_covariance_b200 as px

    op = s["case"]["op"]
    if op == "append":
        lens = px.parallax_kv_append(s["k"], s["v"], s["kpages"], s["vpages"], s["table"], s["seqlens"],
                                     kexp=s["kexp"], vexp=s["vexp"], counts=s["counts"])
        return _cache(s, seqlens=lens)
    if op == "decode":
        if s["case"]["cache"] == "e4m3":
            y, lse = px.parallax_decode_paged_q8(s["q"], s["rho"], s["kpages"], s["vpages"], s["kexp"], s["vexp"],
                                                 s["table"], s["seqlens"], wacc=s["wacc"], out_dtype=torch.bfloat16)
        else:
            y, lse = px.parallax_decode_paged_acc(s["q"], s["rho"], s["kpages"], s["vpages"], s["table"],
                                                  s["seqlens"], s["wacc"], out_dtype=torch.bfloat16)
        return dict(y=y, lse=lse, wacc=s["wacc"])
    lens, kept, wacc = px.parallax_kv_evict(s["kpages"], s["vpages"], s["table"], s["seqlens"], s["wacc"], s["table2"],
                                            s["case"]["budget"], s["case"]["recent"], kexp=s["kexp"], vexp=s["vexp"],
                                            kept=s["kept"], new_wacc=s["wacc2"])
    return _cache(s, seqlens=lens, kept=kept, wacc=wacc)


def _cache(s, **more):
    return dict(kpages=s["kpages"], vpages=s["vpages"], kexp=s["kexp"], vexp=s["vexp"], **more)


def _bytes(pages):
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def _append(s):
    B, Hkv, T, d = s["k"].shape
    page, dev = s["kpages"].shape[2], s["k"].device
    start, n = s["seqlens"].long(), s["counts"].long()
    first = start // BLOCK * BLOCK                              # the block that the first new token falls into
    W = -(-(T + BLOCK - 1) // BLOCK) * BLOCK
    j = torch.arange(W, device=dev)
    pos = first[:, None] + j                                    # [B, W] token positions
    src = pos - start[:, None]
    new = (src >= 0) & (src < n[:, None])
    old = (src < 0) & (n[:, None] > 0)
    pg = s["table"].long().gather(1, (pos // page).clamp(max=s["table"].shape[1] - 1))
    row = pos % page
    bi, ji = torch.nonzero(new | old, as_tuple=True)
    where = (pg[bi, ji][:, None], torch.arange(Hkv, device=dev)[None], row[bi, ji][:, None])     # [rows, Hkv]
    take = src.clamp(0, T - 1)[:, None, :, None].expand(B, Hkv, W, d)
    for x, pages, exps in ((s["k"], s["kpages"], s["kexp"]), (s["v"], s["vpages"], s["vexp"])):
        xs = x.gather(2, take).float()
        held = _bytes(pages)[pg[:, :, None], torch.arange(Hkv, device=dev)[None, None], row[:, :, None]]   # [B,W,Hkv,d]
        if exps is None:
            out = torch.where(new[:, None, :, None], x.gather(2, take), held.transpose(1, 2))
            _bytes(pages)[where] = out.transpose(1, 2)[bi, ji]
            continue
        held = held.view(torch.float8_e4m3fn).float().transpose(1, 2)                             # [B,Hkv,W,d]
        fine = new[:, None, :, None] & torch.isfinite(xs)
        amax = torch.where(fine, xs.abs(), 0.0).view(B, Hkv, W // BLOCK, BLOCK * d).amax(3)
        blk = pos[:, ::BLOCK]
        bpg, brow = pg[:, ::BLOCK], blk % page // BLOCK
        e_old = exps[bpg[:, :, None], torch.arange(Hkv, device=dev)[None, None], brow[:, :, None]].int().transpose(1, 2)
        has_old = old[:, ::BLOCK][:, None]                      # a block with old rows starts with one
        e = torch.maximum(_exponent(amax), torch.where(has_old, e_old, EMIN))
        up = _two_to(-e).repeat_interleave(BLOCK, 2)[..., None]
        shift = _two_to(torch.where(has_old, e_old - e, 0).clamp(-126, 0)).repeat_interleave(BLOCK, 2)[..., None]
        code = torch.where(new[:, None, :, None], torch.where(torch.isfinite(xs), xs, math.nan) * up, held * shift)
        _bytes(pages)[where] = code.to(torch.float8_e4m3fn).view(torch.uint8).transpose(1, 2)[bi, ji]
        cb, cj = torch.nonzero((new | old).view(B, W // BLOCK, BLOCK).any(2), as_tuple=True)
        exps[bpg[cb, cj][:, None], torch.arange(Hkv, device=dev)[None], brow[cb, cj][:, None]] = \
            e.to(torch.int8).transpose(1, 2)[cb, cj]
    return _cache(s, seqlens=s["seqlens"] + s["counts"])


def _gathered(pages, exps, table):
    """The cache of every sequence in fp32: [B, Hkv, P * page, d]."""
    t = table.long()
    x = _bytes(pages)[t]                                        # [B, P, Hkv, page, d]
    B, P, Hkv, page, d = x.shape
    if exps is not None:
        x = x.view(torch.float8_e4m3fn).float().view(B, P, Hkv, page // BLOCK, BLOCK, d) * \
            _two_to(exps[t])[..., None, None]
    return x.float().view(B, P, Hkv, page, d).transpose(1, 2).reshape(B, Hkv, P * page, d)


def _decode(s):
    q, rho, L = s["q"].float(), s["rho"], s["seqlens"].long()
    B, Hq, d = q.shape
    k = _gathered(s["kpages"], s["kexp"], s["table"])
    Hkv, T = k.shape[1], k.shape[2]
    live = (torch.arange(T, device=q.device) < L[:, None])[:, None, None]                # [B, 1, 1, T]
    z = torch.matmul(q.view(B, Hkv, Hq // Hkv, d) / math.sqrt(d), k.transpose(2, 3))
    z = torch.where(live, z, -math.inf)
    top = z.amax(3, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = torch.exp(z - top)
    total = p.sum(3, keepdim=True)
    w = p / torch.where(total > 0, total, 1.0)
    a = torch.matmul(rho.float().view(B, Hkv, Hq // Hkv, d), k.transpose(2, 3)) if rho is not None else None
    del k
    v = torch.where(live[:, :, 0, :, None], _gathered(s["vpages"], s["vexp"], s["table"]), 0.0)
    y = torch.matmul(w, v)
    if a is not None:
        wa = torch.where(live, w * a, 0.0)
        y = y - (torch.matmul(wa, v) - y * wa.sum(3, keepdim=True))
    if s["wacc"] is not None:
        s["wacc"] += w.sum(2)
    lse = (torch.log(total) + top)[..., 0].view(B, Hq)
    return dict(y=y.view(B, Hq, d).to(torch.bfloat16), lse=lse, wacc=s["wacc"])


def _evict(s):
    c, L, wacc = s["case"], s["seqlens"].long(), s["wacc"]
    budget, recent, dev = c["budget"], c["recent"], wacc.device
    B, Hkv, cap = wacc.shape
    page = s["kpages"].shape[2]
    n = L.clamp(max=budget)
    pos = torch.arange(cap, device=dev)
    new = pos >= (L - torch.minimum(n, torch.full_like(n, recent)))[:, None]
    key = torch.where(torch.isnan(wacc), -math.inf, wacc).double()
    order = torch.where((pos >= L[:, None])[:, None], 1.0, torch.where(new[:, None], -1.0, 0.0)).expand(B, Hkv, cap)
    # newest first, then by weight, then by index: two stable sorts, the last key first
    by = torch.sort(key, dim=2, descending=True, stable=True).indices
    by = by.gather(2, torch.sort(order.gather(2, by), dim=2, stable=True).indices)
    budget_ = min(budget, cap)
    by = torch.where(torch.arange(budget_, device=dev) < n[:, None, None], by[..., :budget_], cap)
    kept = torch.sort(by, dim=2).values                         # [B, Hkv, budget], cap where nothing is kept
    i = torch.arange(budget_, device=dev)
    ok = (i < n[:, None])[:, None].expand(B, Hkv, budget_)
    src = kept.clamp(max=cap - 1)
    bi, hi, ii = torch.nonzero(ok, as_tuple=True)
    si = src[bi, hi, ii]
    s["kept"][bi, hi, ii] = si.to(torch.int32)
    s["wacc2"][bi, hi, ii] = wacc[bi, hi, si]
    sp, dp = s["table"][bi, si // page].long(), s["table2"][bi, ii // page].long()
    for pages, exps in ((s["kpages"], s["kexp"]), (s["vpages"], s["vexp"])):
        rows = _bytes(pages)[sp, hi, si % page]
        if exps is not None:
            es = exps[sp, hi, si % page // BLOCK].int()
            nb = -(-budget_ // BLOCK)
            full = torch.full((B, Hkv, nb * BLOCK), EMIN, dtype=torch.int32, device=dev)
            full[bi, hi, ii] = es
            e = full.view(B, Hkv, nb, BLOCK).amax(3)[bi, hi, ii // BLOCK]
            rows = (rows.view(torch.float8_e4m3fn).float() * _two_to((es - e).clamp(min=-126))[:, None])
            rows = rows.to(torch.float8_e4m3fn).view(torch.uint8)
            exps[dp, hi, ii % page // BLOCK] = e.to(torch.int8)
        _bytes(pages)[dp, hi, ii % page] = rows
    return _cache(s, seqlens=n.to(torch.int32), kept=s["kept"], wacc=s["wacc2"])


# ---------------------------------------------------------------- the definition in 64 bits
def _values(s, which, b, n):
    """Sequence b's first n rows of K or V in fp64, [Hkv, n, d]."""
    pages, exps = s[which + "pages"], s[which + "exp"]
    page = pages.shape[2]
    t = torch.arange(n, device=pages.device)
    ids = s["table"][b].long()[t // page]
    if exps is None:
        return pages[ids, :, t % page].double().transpose(0, 1)
    x = pages.view(torch.uint8)[ids, :, t % page].view(torch.float8_e4m3fn).float().double()
    return (x * torch.pow(2.0, exps[ids, :, t % page // BLOCK].double())[..., None]).transpose(0, 1)


def _code_values():
    """The finite e4m3 values, ascending and not negative."""
    m = torch.arange(8, dtype=torch.float64)
    sub = m / 8 * 2.0 ** -6
    rest = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16)]
    return torch.cat([sub] + rest)[:-1].cuda()                  # the last code is NaN


def _rounded(x):
    """x rounded to e4m3, ties to the even code, in fp64."""
    v = _code_values()
    mid = (v[:-1] + v[1:]) / 2
    a = x.abs().contiguous()
    lo, hi = torch.searchsorted(mid, a, right=False), torch.searchsorted(mid, a, right=True)
    i = torch.where((lo != hi) & (lo % 2 != 0), hi, lo)         # between two: the even one
    return torch.copysign(v[i], x)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "evict": _exact_evict}[case["op"]](s)


def _whole(s):
    """Pages as fp64 values of their codes, to be written into."""
    as64 = lambda p: (p.view(torch.uint8).view(torch.float8_e4m3fn).float() if p.dtype == torch.float8_e4m3fn
                      else p).double()
    exps = [None if s[n] is None else s[n].clone() for n in ("kexp", "vexp")]
    return as64(s["kpages"]), as64(s["vpages"]), exps


def _exact_append(s):
    if s["kpages"].numel() > 1 << 29:
        return None
    kd, vd, exps = _whole(s)
    page, Hkv = s["kpages"].shape[2], s["kpages"].shape[1]
    steps = CODE_MAX * torch.pow(2.0, torch.arange(EMIN, EMAX + 1, device="cuda").double())
    lens, counts = s["seqlens"].tolist(), s["counts"].tolist()
    for b, (start, n) in enumerate(zip(lens, counts)):
        if n == 0:
            continue
        t = torch.arange(start, start + n, device="cuda")
        ids = s["table"][b].long()[t // page]
        for x, out, ex in ((s["k"], kd, exps[0]), (s["v"], vd, exps[1])):
            rows = x[b, :, :n].double().transpose(0, 1)         # [n, Hkv, d]
            if ex is not None:
                first, last = start // BLOCK, (start + n - 1) // BLOCK
                big = torch.zeros((last - first + 1, Hkv), dtype=torch.float64, device="cuda")
                big.index_reduce_(0, t // BLOCK - first, rows.abs().amax(2), "amax")
                e = (torch.searchsorted(steps, big) + EMIN).clamp(max=EMAX)
                o = start - first * BLOCK
                bt = torch.arange(first, last + 1, device="cuda") * BLOCK
                bid, brow = s["table"][b].long()[bt // page], bt % page // BLOCK
                if o:
                    was = ex[bid[0], :, brow[0]].long()
                    e[0] = torch.maximum(e[0], was)
                    r = slice(int(brow[0]) * BLOCK, int(brow[0]) * BLOCK + o)
                    out[bid[0], :, r] = _rounded(out[bid[0], :, r] * torch.pow(2.0, (was - e[0]).double())[:, None, None])
                ex[bid, :, brow] = e.to(torch.int8)
                rows = _rounded(rows * torch.pow(2.0, -e[t // BLOCK - first].double())[..., None])
            out[ids, :, t % page] = rows
    return dict(kpages=kd, vpages=vd, kexp=exps[0], vexp=exps[1], seqlens=s["seqlens"] + s["counts"])


def _exact_decode(s):
    B, Hq, d = s["q"].shape
    Hkv = s["kpages"].shape[1]
    G = Hq // Hkv
    y = torch.zeros((B, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    wacc = None if s["wacc"] is None else s["wacc"].double()
    for b, n in enumerate(s["seqlens"].tolist()):
        if n == 0:
            continue
        k, v = _values(s, "k", b, n), _values(s, "v", b, n)
        z = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(Hkv, G, d), k) / math.sqrt(d)
        lse[b] = torch.logsumexp(z, 2).view(Hq)
        w = torch.softmax(z, 2)
        o = torch.einsum("hgt,htd->hgd", w, v)
        out = o
        if s["rho"] is not None:                                # y = o - sum_j s_j (v_j - o) ((k_j - kbar) . rho)
            r = s["rho"][b].double().view(Hkv, G, d)
            kbar = torch.einsum("hgt,htd->hgd", w, k)
            c = w * (torch.einsum("hgd,htd->hgt", r, k) - (kbar * r).sum(2, keepdim=True))
            out = o - (torch.einsum("hgt,htd->hgd", c, v) - c.sum(2, keepdim=True) * o)
        y[b] = out.reshape(Hq, d)
        if wacc is not None:
            wacc[b, :, :n] += w.sum(1)
    return dict(y=y, lse=lse, wacc=wacc)


def _exact_evict(s):
    if s["kpages"].numel() > 1 << 29:
        return None
    kd, vd, exps = _whole(s)
    page, c = s["kpages"].shape[2], s["case"]
    kept, wacc, lens = s["kept"].clone(), s["wacc2"].double(), []
    for b, L in enumerate(s["seqlens"].tolist()):
        n = min(L, c["budget"])
        lens.append(n)
        r = min(c["recent"], n)
        if n == 0:
            continue
        rank = torch.sort(s["wacc"][b, :, :L - r].double(), dim=1, descending=True, stable=True).indices[:, :n - r]
        tail = torch.arange(L - r, L, device="cuda").expand(rank.shape[0], r)
        keep = torch.sort(torch.cat([rank, tail], 1), dim=1).values          # [Hkv, n]
        h = torch.arange(keep.shape[0], device="cuda")[:, None]
        kept[b, :, :n] = keep.to(torch.int32)
        wacc[b, :, :n] = s["wacc"][b].double().gather(1, keep)
        i = torch.arange(n, device="cuda")[None]
        sp, dp = s["table"][b].long()[keep // page], s["table2"][b].long()[i // page]
        for out, ex in ((kd, exps[0]), (vd, exps[1])):
            rows = out[sp, h, keep % page]
            if ex is not None:
                es = ex[sp, h, keep % page // BLOCK].long()
                pad = torch.full((es.shape[0], -n % BLOCK), EMIN, device="cuda")
                e = torch.cat([es, pad], 1).view(es.shape[0], -1, BLOCK).amax(2).repeat_interleave(BLOCK, 1)[:, :n]
                rows = _rounded(rows * torch.pow(2.0, (es - e).double())[..., None])
                ex[dp, h, i % page // BLOCK] = e.to(torch.int8)
            out[dp, h, i % page] = rows
    return dict(kpages=kd, vpages=vd, kexp=exps[0], vexp=exps[1],
                seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"), kept=kept, wacc=wacc)

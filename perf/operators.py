"""Measured calls of the sink-window attention and of the paged cache.

Three operators: causal attention over a sliding window plus a few first
tokens (forward and backward, dense or packed batches), attention of one new
token over a paged key/value cache, and the cache's pages themselves (handing
out pages and writing new tokens, forking, freeing, compacting).  `run` makes
the library's calls where `own` is true and computes the same thing from
elementary torch operations in 32 bits where it is false.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the smallest layer call, where latency counts: one short prompt of the tiny sparse-attention configuration
        dict(name="fwd tiny", kind="fwd", B=1, Tq=512, L=512, Hq=4, Hkv=1, d=64, window=32, sinks=4, dtype="bf16",
             packed=False, fused_qkv=False, lens_seed=0),
        # a serving prefill step: ragged prompts packed back to back, q/k/v views of one projection, an fp16 model
        dict(name="fwd ragged fp16", kind="fwd", B=7, Tq=4999, L=4999, Hq=16, Hkv=4, d=128, window=512, sinks=4,
             dtype="fp16", packed=True, fused_qkv=True, lens_seed=3),
        # a whole 64K prompt in one call, 16 heads on one KV head, the largest amount of work
        dict(name="fwd 64k", kind="fwd", B=1, Tq=65536, L=65536, Hq=16, Hkv=1, d=128, window=2048, sinks=128,
             dtype="bf16", packed=False, fused_qkv=False, lens_seed=0),
        # training a small multi-head model on short texts
        dict(name="bwd small", kind="bwd", B=2, Tq=1000, L=1000, Hq=8, Hkv=8, d=64, window=65, sinks=4, dtype="bf16",
             packed=False, fused_qkv=False, lens_seed=0),
        # training on 16K contexts with 64 heads on 4 KV heads, window 512
        dict(name="bwd 16k", kind="bwd", B=1, Tq=16384, L=16384, Hq=64, Hkv=4, d=128, window=512, sinks=16,
             dtype="bf16", packed=False, fused_qkv=False, lens_seed=0),
        # one user's next token on a short context: latency
        dict(name="decode one", kind="decode", B=1, max_len=2048, Hq=16, Hkv=1, d=128, page=16, window=0, sinks=0,
             dtype="bf16", interleaved=False, lens_seed=0),
        # a busy server's step: ragged contexts with window and sinks, trimmed middles, K and V interleaved by page
        dict(name="decode window ragged", kind="decode", B=192, max_len=12345, Hq=64, Hkv=8, d=128, page=64,
             window=4096, sinks=64, dtype="fp16", interleaved=True, lens_seed=5),
        # 32 sequences at 128K, 16 heads on one KV head: the whole cache is read
        dict(name="decode 128k", kind="decode", B=32, max_len=131072, Hq=16, Hkv=1, d=128, page=64, window=0, sinks=0,
             dtype="bf16", interleaved=False, lens_seed=0),
        # one token of every running sequence gets its slot and is written (one layer's K and V)
        dict(name="append step", kind="append", B=256, tokens=1, max_len=8192, Hkv=8, d=128, page=16, dtype="bf16",
             lens_seed=1),
        # parallel sampling: 16 prompts, 8 samples each, every layer's cache (4 layers of K and V)
        dict(name="fork samples", kind="fork", B=16, children=8, max_len=6000, Hkv=4, d=128, page=64, layers=4,
             dtype="bf16", lens_seed=2),
        # the end of a batch: its sequences give their pages back, half of them shared
        dict(name="free batch", kind="free", B=256, children=1, max_len=16384, Hkv=1, d=64, page=16, layers=1,
             dtype="bf16", lens_seed=4),
        # a pool that is 40 % live after hours of traffic is packed to its front
        dict(name="compact pool", kind="compact", B=96, pages=6000, live=2400, Hkv=4, d=128, page=64, layers=4,
             dtype="bf16", lens_seed=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "decode", "decode", "append", "fork", "free", "compact"])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if kind in ("fwd", "bwd"):
        Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
        B = rng.choice([1, 1, 2, 3, 5, 8])
        Tq = _log(rng, 1, (32768 if kind == "fwd" else 8192) // B)
        packed = rng.random() < 0.4
        L = Tq + (0 if rng.random() < 0.6 else _log(rng, 1, 8192))
        window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, 16, 64, 130, 300])
        if kind == "bwd":                # one visible key has no gradient but rounding: at least two
            Tq, window = max(2, Tq), max(2, window)
        while B * Tq * Hq * (min(window, L) + sinks + 256) > (1.2e9 if kind == "bwd" else 2.2e9):
            window, Tq = max(2, window // 2), max(2, Tq * 3 // 4)
        return dict(kind=kind, B=B, Tq=Tq, L=max(L, Tq), Hq=Hq, Hkv=Hkv, d=d, window=window, sinks=sinks,
                    dtype=dtype if kind == "fwd" else "bf16", packed=packed, fused_qkv=L == Tq and rng.random() < 0.5,
                    lens_seed=rng.randrange(1 << 20))
    if kind == "decode":
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8, 16])
        B = _log(rng, 1, 256)
        max_len = _log(rng, 1, 131072)
        while B * max_len * Hkv > 4.2e6:
            B, max_len = max(1, B * 3 // 4), max(1, max_len * 3 // 4)
        windowed = rng.random() < 0.5
        return dict(kind=kind, B=B, max_len=max_len, Hq=Hq, Hkv=Hkv, d=d, page=rng.choice([1, 8, 16, 24, 64, 128, 256]),
                    window=_log(rng, 1, 8192) if windowed else 0, sinks=rng.choice([0, 4, 64, 100]) if windowed else 0,
                    dtype=dtype, interleaved=rng.random() < 0.5, lens_seed=rng.randrange(1 << 20))
    page, layers = rng.choice([8, 16, 24, 64, 128]), rng.choice([1, 2, 3, 4])
    common = dict(Hkv=Hkv, d=d, page=page, dtype=dtype, lens_seed=rng.randrange(1 << 20))
    if kind == "append":
        return dict(kind=kind, B=_log(rng, 1, 1024), tokens=rng.choice([1, 1, 3, 50]), max_len=_log(rng, 8, 4096),
                    **common)
    if kind == "compact":
        pages = _log(rng, 16, 12000 * 64 // (page * layers * Hkv) + 17)
        return dict(kind=kind, B=_log(rng, 1, 128), pages=pages, live=max(1, int(pages * rng.uniform(0.1, 0.95))),
                    layers=layers, **common)
    return dict(kind=kind, B=_log(rng, 1, 64), children=rng.choice([1, 2, 5, 8]), max_len=_log(rng, 1, 4096),
                layers=layers, **common)


def _lens(case):
    """Sequence lengths of a case: one of the largest length, the others spread down to one token over the logarithm."""
    B, top = case["B"], case.get("max_len") or case["L"]
    if case["kind"] == "decode" and not case["lens_seed"]:
        return [top] * B
    r = random.Random(case["lens_seed"])
    return [top] + [_log(r, max(1, top // 64), top) for _ in range(B - 1)]


def _query_lens(case):
    if not case["packed"]:
        return [case["Tq"]] * case["B"], [case["L"]] * case["B"]
    kl = _lens(case)
    if case["Tq"] == case["L"]:
        return list(kl), kl
    return [min(case["Tq"], n) for n in kl], kl


def _visible(p, window, sinks):
    return min(p + 1, window) + min(sinks, max(0, p + 1 - window))


def _pairs(n_q, n_k, window, sinks):
    p = torch.arange(n_k - n_q, n_k, dtype=torch.int64) + 1
    return int((p.clamp(max=window) + (p - window).clamp(min=0, max=sinks)).sum())


def work(case):
    kind, e = case["kind"], 2
    if kind in ("fwd", "bwd"):
        ql, kl = _query_lens(case)
        pairs = sum(_pairs(a, b, case["window"], case["sinks"]) for a, b in zip(ql, kl)) if case["packed"] else \
            case["B"] * _pairs(ql[0], kl[0], case["window"], case["sinks"])
        nq, nk = sum(ql) * case["Hq"] * case["d"] * e, sum(kl) * case["Hkv"] * case["d"] * e
        lse = sum(ql) * case["Hq"] * 4
        if kind == "fwd":
            return {"bytes": 2 * nq + 2 * nk + lse, "flops": 4 * case["d"] * case["Hq"] * pairs}
        return {"bytes": 4 * nq + 4 * nk + lse, "flops": 10 * case["d"] * case["Hq"] * pairs}
    lens = _lens(case) if kind != "compact" else []
    row = case["Hkv"] * case["d"] * e
    if kind == "decode":
        w = case["window"] or case["max_len"]
        seen = sum(_visible(n - 1, w, case["sinks"]) for n in lens)
        return {"bytes": 2 * seen * row + case["B"] * case["Hq"] * (2 * case["d"] * e + 4) + 4 * seen // case["page"],
                "flops": 4 * case["d"] * case["Hq"] * seen}
    if kind == "append":
        n = case["B"] * case["tokens"]
        return {"bytes": 4 * n * row + 4 * (5 * case["B"] + 2 * (n // case["page"] + 1)), "flops": 0}
    if kind == "fork":
        pages = sum(n // case["page"] for n in lens) * case["children"]
        tails = sum(1 for n in lens if n % case["page"]) * case["children"]
        return {"bytes": tails * 4 * case["layers"] * case["page"] * row + 4 * 4 * pages, "flops": 0}
    if kind == "free":
        return {"bytes": 4 * 4 * 2 * sum(-(-n // case["page"]) for n in lens), "flops": 0}
    moved = case["live"] * (1 - case["live"] / case["pages"])
    return {"bytes": moved * 4 * case["layers"] * case["page"] * row + 8 * case["pages"] + 4 * case["live"], "flops": 0}


# ------------------------------------------------------------------ inputs --
def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _attn_inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, Hq, Hkv, d = TYPES[case["dtype"]], case["Hq"], case["Hkv"], case["d"]
    ql, kl = _query_lens(case)
    qs = (sum(ql),) if case["packed"] else (case["B"], case["Tq"])
    ks = (sum(kl),) if case["packed"] else (case["B"], case["L"])
    if case["fused_qkv"] and qs == ks:
        qkv = _randn(gen, (*qs, Hq + 2 * Hkv, d), dt)
        q, k, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
    else:
        q, k, v = _randn(gen, (*qs, Hq, d), dt), _randn(gen, (*ks, Hkv, d), dt), _randn(gen, (*ks, Hkv, d), dt)
    # a trained model's queries lean towards the first keys: give both a common part
    lean = torch.randn(d, generator=gen, device="cuda").sign() * (2.0 / d ** 0.25)
    q += (0.5 * lean).to(dt)
    cu_q = cu_k = None
    if case["packed"]:
        cu_q = torch.tensor([0, *ql], device="cuda").cumsum(0).to(torch.int32)
        cu_k = torch.tensor([0, *kl], device="cuda").cumsum(0).to(torch.int32)
        k.index_add_(0, cu_k[:-1].long(), lean.to(dt).expand(len(kl), Hkv, d))
    else:
        k[:, 0] += lean.to(dt)
    return dict(q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, max_q=max(ql), max_k=max(kl), gen=gen)


def _pool(case, gen, lens, spare, share=1, extra=0):
    """Tables of sequences over a pool of pages in random order; `share` slots hold each sequence's pages."""
    page, B = case["page"], len(lens)
    held = torch.tensor([-(-n // page) for n in lens], device="cuda")
    n_held = int(sum(-(-n // page) for n in lens))
    n_pages = n_held + spare
    width = max(-(-(max(lens) + extra) // page), 1) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda")[None, :] < held[:, None]
    table[at] = order[:n_held].to(torch.int32)
    refcount = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refcount[order[:n_held]] = share
    return table, refcount, n_pages, order[n_held:]


def prepare(case, seed):
    kind, dt = case["kind"], TYPES[case["dtype"]]
    if kind in ("fwd", "bwd"):
        s = _attn_inputs(case, seed)
        gen = s.pop("gen")
        if kind == "bwd":
            out, lse = _plain_fwd(case, s)
            s |= dict(out=out, lse=lse, dout=_randn(gen, tuple(out.shape), dt))
        return {"case": case, **s}
    gen = torch.Generator(device="cuda").manual_seed(seed)
    Hkv, d, page = case["Hkv"], case["d"], case["page"]

    def caches(n_pages, layers):
        return [_randn(gen, (n_pages, page, Hkv, d), dt) for _ in range(2 * layers)]

    if kind == "compact":
        n_pages, live, B = case["pages"], case["live"], case["B"]
        ids = torch.randperm(n_pages, generator=gen, device="cuda")[:live].to(torch.int32)
        width = -(-live // B) + 1
        slot = torch.randint(0, B, (live,), generator=gen, device="cuda")
        slot = torch.where(torch.arange(live, device="cuda") < B * (live // B), torch.arange(live, device="cuda") % B, slot * 0)
        table = torch.full((B, width + live - B * (live // B)), -1, dtype=torch.int32, device="cuda")
        order = torch.argsort(slot, stable=True)
        nth = torch.arange(live, device="cuda") - torch.searchsorted(slot[order].contiguous(), slot[order].contiguous())
        table[slot[order], nth] = ids[order]
        refcount = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        refcount[ids.long()] = 1
        return _with_books(case, table, torch.zeros(B, dtype=torch.int32, device="cuda"), refcount,
                           caches=caches(n_pages, case["layers"]))
    lens = _lens(case)
    if kind == "decode":
        table, _, n_pages, unused = _pool(case, gen, lens, spare=3)
        kv = _randn(gen, (n_pages, 2, page, Hkv, d), dt) if case["interleaved"] else \
            _randn(gen, (2, n_pages, page, Hkv, d), dt).transpose(0, 1)
        kv[unused] = float("nan")                            # pages that nobody holds were never written
        lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        last = table[torch.arange(len(lens), device="cuda"), ((lens_t - 1) // page).long()].long()
        fresh = torch.arange(page, device="cuda")[None, :] > ((lens_t - 1) % page)[:, None]
        kv.transpose(1, 2)[last[:, None].expand(-1, page)[fresh],
                           torch.arange(page, device="cuda")[None, :].expand(len(lens), -1)[fresh]] = float("nan")
        if case["window"]:                                   # the pages that the window has passed went back to the pool
            lo = torch.arange(table.shape[1], device="cuda")[None, :] * page
            gone = (lo >= case["sinks"]) & (lo + page <= (lens_t - case["window"])[:, None])
            table.masked_fill_(gone, -1)
        return dict(case=case, q=_randn(gen, (case["B"], case["Hq"], d), dt), k=kv[:, 0], v=kv[:, 1], table=table,
                    lens=lens_t)
    B = len(lens)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if kind == "append":
        n = case["tokens"]
        new = sum(-(-(x + n) // page) - -(-x // page) for x in lens)
        table, refcount, n_pages, _ = _pool(case, gen, lens, spare=new + 5, extra=n)
        kc, vc = caches(n_pages, 1)
        return _with_books(case, table, lens_t, refcount, caches=[kc, vc],
                           seqs=torch.randperm(B, generator=gen, device="cuda").to(torch.int32),
                           n_new=torch.full((B,), n, dtype=torch.int32, device="cuda"),
                           cu=torch.arange(0, (B + 1) * n, n, dtype=torch.int32, device="cuda"),
                           k_new=_randn(gen, (B * n, Hkv, d), dt), v_new=_randn(gen, (B * n, Hkv, d), dt))
    C = case["children"]
    if kind == "fork":
        table, refcount, n_pages, _ = _pool(case, gen, lens, spare=B * C + 3)
        table = torch.cat([table, torch.full((B * C, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
        return _with_books(case, table, torch.cat([lens_t, lens_t.new_zeros(B * C)]), refcount,
                           caches=caches(n_pages, case["layers"]),
                           src=torch.arange(B, device="cuda").repeat_interleave(C).to(torch.int32),
                           dst=(B + torch.randperm(B * C, generator=gen, device="cuda")).to(torch.int32))
    # free: every sequence is held C + 1 times, the first C copies of every second one are freed
    table, refcount, _, _ = _pool(case, gen, lens, spare=7, share=C + 1)
    seqs = torch.randperm(B * C, generator=gen, device="cuda").to(torch.int32)
    return _with_books(case, table.repeat(C + 1, 1), lens_t.repeat(C + 1), refcount, seqs=seqs[: max(1, B * C * 3 // 4)])


def _with_books(case, table, lens, refcount, **more):
    """The cache's books (table, lengths, counts) in one buffer beside a copy of it, so that a pass can start from the same books."""
    flat = torch.cat([table.reshape(-1), lens, refcount])
    a, b = table.numel(), table.numel() + lens.numel()
    books = flat.clone()
    return dict(case=case, first=flat, books=books, table=books[:a].view(table.shape), lens=books[a:b], refcount=books[b:],
                **more)


# --------------------------------------------------------------------- run --
def run(s):
    case = s["case"]
    kind = case["kind"]
    if kind in ("append", "fork", "free", "compact"):
        s["books"].copy_(s["first"])
    if own:
        return _own(case, kind, s)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "append": _plain_append, "fork": _plain_fork,
            "free": _plain_free, "compact": _plain_compact}[kind](case, s)


def _own(case, kind, s):
    from fixed_pattern_sparse_sa_b200 import api
    if kind == "fwd":
        return api.sink_attn_fwd(s["q"], s["k"], s["v"], case["window"], case["sinks"], cu_q=s["cu_q"], cu_k=s["cu_k"],
                                 max_q=s["max_q"], max_k=s["max_k"])
    if kind == "bwd":
        return api.sink_attn_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], case["window"], case["sinks"],
                                 cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=s["max_q"], max_k=s["max_k"])
    if kind == "decode":
        return api.paged_attn_decode(s["q"], s["k"], s["v"], s["table"], s["lens"], window=case["window"] or None,
                                     sinks=case["sinks"])
    table, lens, refcount = s["table"], s["lens"], s["refcount"]
    if kind == "append":
        start = api.paged_extend(table, lens, refcount, s["seqs"], s["n_new"], case["page"])
        api.paged_write(s["k_new"], s["v_new"], *s["caches"], table, s["seqs"], start, cu_new=s["cu"])
        return [start, table, lens, refcount, *s["caches"]]
    if kind == "fork":
        done = api.paged_fork(table, lens, refcount, s["src"], s["dst"], case["page"], s["caches"])
        return [done, table, lens, refcount, *s["caches"]]
    if kind == "free":
        api.paged_free(table, lens, refcount, s["seqs"])
        return [table, lens, refcount]
    n_live = api.paged_compact(table, refcount, s["caches"])
    return [n_live, table, refcount, *s["caches"]]


# ------------------------------------------------------------- plain forms --
def _rows(cu, top, N):
    """Padded view of packed rows: [B, top] row numbers, lengths, and for each packed row its place in the padded view."""
    cu = cu.long()
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.arange(top, device=cu.device)).clamp(max=N - 1)
    r = torch.arange(N, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    return at, n, b * top + r - cu[b]


def _banded(q, k, v, n_q, n_k, window, sinks):
    """q [B, Tq, Hq, d], k, v [B, L, Hkv, d] in 32 bits, lengths [B]: blocks of queries against the band of keys that any of them sees, and the sinks."""
    B, Tq, Hq, d = q.shape
    L, Hkv = k.shape[1:3]
    G, dev = Hq // Hkv, q.device
    bs = min(256, Tq)
    nb = -(-Tq // bs)
    W = min(window, L + bs)
    M, S = W + bs - 1, min(sinks, L)
    qb = torch.nn.functional.pad(q, (0, 0, 0, 0, 0, nb * bs - Tq)).view(B, nb, bs, Hkv, G, d).permute(0, 1, 3, 4, 2, 5)
    p = (n_k - n_q)[:, None, None] + torch.arange(nb * bs, device=dev).view(1, nb, bs)          # positions of the queries
    j = p[:, :, :1] - (W - 1) + torch.arange(M, device=dev)                                     # [B, nb, M] keys of a block
    rows = torch.arange(B, device=dev)[:, None, None]
    jc = j.clamp(0, L - 1)
    kb, vb = k[rows, jc].permute(0, 1, 3, 4, 2), v[rows, jc].permute(0, 1, 3, 2, 4)             # [B, nb, Hkv, d, M], [B, nb, Hkv, M, d]
    gap = p[..., None] - j[:, :, None, :]
    see = (gap >= 0) & (gap < window) & ((j >= 0) & (j < n_k[:, None, None]))[:, :, None, :]
    js = torch.arange(S, device=dev)
    gap = p[..., None] - js
    see_s = (gap >= window) & (js < n_k[:, None, None, None])
    z = torch.cat([qb.reshape(B, nb, Hkv, G * bs, d) @ kb,
                   qb.reshape(B, nb, Hkv, G * bs, d) @ k[:, :S].permute(0, 2, 3, 1)[:, None]], -1)
    z = z.view(B, nb, Hkv, G, bs, M + S) * (1.0 / math.sqrt(d))
    z = z.masked_fill(~torch.cat([see, see_s], -1)[:, :, None, None], -math.inf)
    m = z.detach().amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = (z - m).exp()
    l = e.sum(-1, keepdim=True)
    ef = e.view(B, nb, Hkv, G * bs, M + S)
    o = ef[..., :M] @ vb + ef[..., M:] @ v[:, :S].permute(0, 2, 1, 3)[:, None]
    o = o.view(B, nb, Hkv, G, bs, d) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(B, nb * bs, Hq, d)[:, :Tq]
    lse = (m + l.log()).squeeze(-1).permute(0, 1, 4, 2, 3).reshape(B, nb * bs, Hq)[:, :Tq]
    return o, lse


def _padded(case, s, q, k, v):
    """The banded form's output for dense or packed inputs."""
    if s["cu_q"] is None:
        B = q.shape[0]
        n_q, n_k = (torch.full((B,), n, device=q.device) for n in (q.shape[1], k.shape[1]))
        return _banded(q, k, v, n_q, n_k, case["window"], case["sinks"])
    at_q, n_q, place = _rows(s["cu_q"], s["max_q"], q.shape[0])
    at_k, n_k, _ = _rows(s["cu_k"], s["max_k"], k.shape[0])
    o, lse = _banded(q[at_q], k[at_k], v[at_k], n_q, n_k, case["window"], case["sinks"])
    return o.flatten(0, 1)[place], lse.flatten(0, 1)[place]


def _plain_fwd(case, s):
    o, lse = _padded(case, s, s["q"].float(), s["k"].float(), s["v"].float())
    return o.to(s["q"].dtype), lse


def _plain_bwd(case, s):
    x = [s[n].float().detach().requires_grad_() for n in "qkv"]
    with torch.enable_grad():
        o, _ = _padded(case, s, *x)
        g = torch.autograd.grad(o, x, s["dout"].float())
    return tuple(t.to(s["q"].dtype) for t in g)


def _plain_decode(case, s):
    q, table, lens = s["q"], s["table"], s["lens"].long()
    B, Hq, d = q.shape
    page, Hkv, top = case["page"], case["Hkv"], case["max_len"]
    window = case["window"] or top
    pos = torch.arange(top, device=q.device)
    gap = lens[:, None] - 1 - pos
    see = (gap >= 0) & ((gap < window) | (pos < case["sinks"]))
    at = table[:, (pos // page).clamp(max=table.shape[1] - 1)].long().clamp(min=0)
    k = torch.where(see[..., None, None], s["k"][at, pos % page].float(), 0.0)
    v = torch.where(see[..., None, None], s["v"][at, pos % page].float(), 0.0)
    z = q.float().view(B, Hkv, Hq // Hkv, d) @ k.permute(0, 2, 3, 1) * (1.0 / math.sqrt(d))
    z = z.masked_fill(~see[:, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = (z - m).exp()
    l = e.sum(-1, keepdim=True)
    o = (e @ v.permute(0, 2, 1, 3)) / l
    return o.view(B, Hq, d).to(q.dtype), (m + l.log()).view(B, Hq)


def _plain_append(case, s):
    table, lens, refcount, page = s["table"], s["lens"], s["refcount"], case["page"]
    kc, vc = s["caches"]
    seqs, n_new = s["seqs"].long(), s["n_new"].long()
    old = lens[seqs].long()
    have = (old + page - 1) // page
    need = (old + n_new + page - 1) // page - have
    free = (refcount == 0).nonzero().squeeze(1)[: table.numel()]
    end = need.cumsum(0)
    ok = (end <= free.numel()) | (need == 0)
    i = torch.repeat_interleave(torch.arange(seqs.numel(), device=seqs.device), torch.where(ok, need, 0))
    nth = torch.arange(i.numel(), device=i.device) - (end - need)[i]
    got = free[: i.numel()]
    table[seqs[i], have[i] + nth] = got.to(torch.int32)
    refcount[got] = 1
    lens[seqs] += torch.where(ok, n_new, 0).to(torch.int32)
    row = torch.repeat_interleave(torch.arange(seqs.numel(), device=seqs.device), n_new)
    pos = old[row] + torch.arange(row.numel(), device=row.device) - s["cu"][row].long()
    keep = ok[row]
    pages = table[seqs[row], pos // page].long()
    kc[pages[keep], (pos % page)[keep]] = s["k_new"][keep]
    vc[pages[keep], (pos % page)[keep]] = s["v_new"][keep]
    return [torch.where(ok, old, -1).to(torch.int32), table, lens, refcount, *s["caches"]]


def _plain_fork(case, s):
    table, lens, refcount, page = s["table"], s["lens"], s["refcount"], case["page"]
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src].long()
    full, tail = n // page, (n % page) != 0
    end = tail.long().cumsum(0)
    free = (refcount == 0).nonzero().squeeze(1)
    ok = ~tail | (end <= free.numel())
    at = torch.arange(table.shape[1], device=table.device)
    shared = (at < full[:, None]) & ok[:, None]
    rows = torch.where(shared, table[src], -1)
    refcount += torch.bincount(rows[shared].long(), minlength=refcount.numel()).to(torch.int32)
    fresh = free[(end - 1).clamp(min=0, max=max(0, free.numel() - 1))]
    part = tail & ok
    old = table[src, full.clamp(max=table.shape[1] - 1)].long()
    rows[part, full[part]] = fresh[part].to(torch.int32)
    refcount[fresh[part]] = 1
    table[dst[ok]] = rows[ok]
    lens[dst[ok]] = lens[src[ok]]
    moved = [(c, c[old[part]]) for c in s["caches"]]
    [c.index_copy_(0, fresh[part], x) for c, x in moved]
    return [ok.to(torch.int32), table, lens, refcount, *s["caches"]]


def _plain_free(case, s):
    table, lens, refcount, seqs = s["table"], s["lens"], s["refcount"], s["seqs"].long()
    held = table[seqs]
    refcount -= torch.bincount(held[held >= 0].long(), minlength=refcount.numel()).to(torch.int32)
    table[seqs] = -1
    lens[seqs] = 0
    return [table, lens, refcount]


def _plain_compact(case, s):
    table, refcount = s["table"], s["refcount"]
    live = refcount > 0
    n_live = live.sum()
    ids = torch.arange(refcount.numel(), device=refcount.device)
    src = (live & (ids >= n_live)).nonzero().squeeze(1)
    dst = (~live & (ids < n_live)).nonzero().squeeze(1)
    new = ids.clone()
    new[src] = dst
    table.copy_(torch.where(table >= 0, new[table.long().clamp(min=0)].to(torch.int32), table))
    refcount[dst] = refcount[src]
    refcount[src] = 0
    [c.index_copy_(0, dst, c[src]) for c in s["caches"]]
    return [n_live.to(torch.int32).view(1), table, refcount, *s["caches"]]


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """The definition in 64 bits, one sequence and block of queries at a time with a whole mask; the page operations compute no numbers."""
    kind = case["kind"]
    if kind == "decode":
        s = prepare(case, seed)
        lens, d = _lens(case), case["d"]
        o, lse = [], []
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            if case["window"]:
                j = j[(j > n - 1 - case["window"]) | (j < case["sinks"])]
            pages, slots = s["table"][b, j // case["page"]].long(), j % case["page"]
            k, v = (s[x][pages, slots].double().repeat_interleave(case["Hq"] // case["Hkv"], 1) for x in "kv")
            z = torch.einsum("hd,jhd->hj", s["q"][b].double(), k) / math.sqrt(d)
            lse.append(torch.logsumexp(z, 1))
            o.append(torch.einsum("hj,jhd->hd", torch.softmax(z, 1), v))
        return torch.stack(o), torch.stack(lse)
    if kind not in ("fwd", "bwd"):
        return None
    s = prepare(case, seed)
    ql, kl = _query_lens(case)
    G, d, window, sinks = case["Hq"] // case["Hkv"], case["d"], case["window"], case["sinks"]
    grads = kind == "bwd"
    q, k, v = (s[x].double() for x in "qkv")
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:-1], dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros_like(x) if grads else None for x in (q, k, v))
    q0 = k0 = 0
    step = max(16, min(1024, (1 << 26) // (case["Hq"] * (min(window, max(kl)) + sinks + 1024))))
    for b, (nq, nk) in enumerate(zip(ql, kl)):
        at = (slice(q0, q0 + nq) if case["packed"] else b), (slice(k0, k0 + nk) if case["packed"] else b)
        qs, ks, vs = q[at[0]], k[at[1]], v[at[1]]
        for t in range(0, nq, step):
            n = min(step, nq - t)
            p = torch.arange(t, t + n, device="cuda") + nk - nq
            lo = max(0, int(t + nk - nq - window + 1))
            j = torch.arange(lo, t + n + nk - nq, device="cuda")
            if min(sinks, lo):
                j = torch.cat([torch.arange(min(sinks, lo), device="cuda"), j])
            see = (j <= p[:, None]) & ((p[:, None] - j < window) | (j < sinks))
            kj, vj = ks[j], vs[j]
            qt = qs[t:t + n].unflatten(1, (-1, G))
            z = torch.einsum("tgid,jgd->gitj", qt, kj) / math.sqrt(d)
            z.masked_fill_(~see, -math.inf)
            big = torch.logsumexp(z, -1, keepdim=True)
            P = torch.exp(z - big)
            ot = torch.einsum("gitj,jgd->tgid", P, vj)
            o[at[0]][t:t + n] = ot.flatten(1, 2)
            lse[at[0]][t:t + n] = big.squeeze(-1).permute(2, 0, 1).flatten(1)
            if grads:
                g = s["dout"][at[0]][t:t + n].double().unflatten(1, (-1, G))
                D = torch.einsum("tgid,tgid->git", g, ot)[..., None]
                dS = P * (torch.einsum("tgid,jgd->gitj", g, vj) - D) / math.sqrt(d)
                dq[at[0]][t:t + n] = torch.einsum("gitj,jgd->tgid", dS, kj).flatten(1, 2)
                dk[at[1]].index_add_(0, j, torch.einsum("gitj,tgid->jgd", dS, qt))
                dv[at[1]].index_add_(0, j, torch.einsum("gitj,tgid->jgd", P, g))
        q0, k0 = q0 + nq, k0 + nk
    return (dq, dk, dv) if grads else (o, lse)

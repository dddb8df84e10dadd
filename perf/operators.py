"""The bounded-cache operators as a serving program calls them, for timing and comparison.

Four operators that hold a paged key-value cache to a bounded size:
  window_decode   one new token per sequence over the first tokens and a sliding window
  window_prefill  the same visibility for every sequence's newest tokens (prompts, chunks)
  score_decode    one new token over the whole context, adding each token's attention weight to its score
  evict           keep the first, the newest and the highest-scored tokens and close the gaps

With `own` false, `run` computes them from elementary torch operations in 32 bits; with `own` true it
calls this package's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, seqs, heads, kv_heads, dim, block, dtype, lo, hi, **more):
    """lo, hi: context lengths spread evenly over [lo, hi], in an order of their own."""
    return dict(name=name, op=op, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype,
                lo=lo, hi=hi, **more)


def listed():
    return [
        # a single conversation far past its window: what counts is the latency of one call
        _case("window_decode_single", "window_decode", 1, 32, 8, 128, 16, "f16", 7001, 7001, window=1024, sinks=4),
        # a full batch of full-head attention, most contexts longer than the window, some shorter
        _case("window_decode_batch", "window_decode", 128, 40, 40, 128, 16, "bf16", 17, 2048, window=1000, sinks=4),
        # long contexts with shared heads; blocks that left the window have been given back
        _case("window_decode_long", "window_decode", 64, 64, 8, 128, 32, "bf16", 4097, 32768, window=4096, sinks=64),
        # one chunk of a prompt behind a cached context
        _case("window_prefill_chunk", "window_prefill", 1, 32, 8, 128, 16, "bf16", 2777, 2777, window=1024, sinks=4,
              new_lo=100, new_hi=100),
        # a batch of prompts of unequal lengths
        _case("window_prefill_batch", "window_prefill", 8, 40, 40, 64, 8, "f16", 300, 1500, window=500, sinks=1,
              new_lo=256, new_hi=1500),
        # one long prompt
        _case("window_prefill_long", "window_prefill", 1, 32, 8, 128, 16, "bf16", 8192, 8192, window=2048, sinks=4,
              new_lo=8192, new_hi=8192),
        # a small 32-bit model's step
        _case("score_decode_small", "score_decode", 4, 8, 8, 64, 16, "f32", 1, 1000),
        # a full batch of full-head attention
        _case("score_decode_batch", "score_decode", 128, 40, 40, 128, 16, "bf16", 17, 2048),
        # few sequences of long contexts with shared heads
        _case("score_decode_long", "score_decode", 8, 32, 8, 128, 32, "f16", 16385, 32768),
        # one sequence over its budget
        _case("evict_single", "evict", 1, 8, 8, 128, 16, "bf16", 2001, 2001, budget=1024, sinks=4, recent=256),
        # a batch, some sequences still within the budget
        _case("evict_batch", "evict", 64, 8, 8, 128, 8, "f16", 700, 4000, budget=1001, sinks=4, recent=100),
        # long contexts cut to a quarter
        _case("evict_long", "evict", 8, 32, 32, 128, 16, "f16", 16385, 32768, budget=8192, sinks=64, recent=1024),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_decode", "window_prefill", "score_decode", "evict"])
    dtype = rng.choice(["f16", "bf16"] if op == "window_prefill" else ["f16", "bf16", "f16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32, 40])
    group = 1 if op == "evict" else rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 12])
    group = min(group, max(1, 64 // kv_heads))
    dim, block = rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32])
    if op == "window_prefill":
        seqs = _spread(rng, 1, 8)
        hi = _spread(rng, 200, 4000 // seqs)
        lo = _spread(rng, max(1, hi // 4), hi)
        new_hi = _spread(rng, max(1, hi // 32), hi)
        more = dict(new_lo=_spread(rng, 1, min(new_hi, lo)), new_hi=new_hi, window=_spread(rng, 16, 2048),
                    sinks=rng.choice([0, 1, 4, 17, 64]))
    else:
        seqs = _spread(rng, 1, 128)
        # total cached rows over all sequences and kv heads, bounded by the largest listed cases
        rows = _spread(rng, 2000, 2_000_000)
        hi = max(16, min(32768, rows // (seqs * kv_heads)))
        lo = _spread(rng, max(1, hi // 8), hi)
        if op == "window_decode":
            more = dict(window=_spread(rng, max(1, hi // 16), min(4096, 2 * hi)), sinks=rng.choice([0, 1, 4, 17, 64]))
        elif op == "evict":
            budget = _spread(rng, max(1, hi // 8), hi)
            sinks = min(rng.choice([0, 1, 4, 64]), budget)
            more = dict(budget=budget, sinks=sinks, recent=rng.randint(0, (budget - sinks + 1) // 2))
        else:
            more = {}
    case = _case("", op, seqs, kv_heads * group, kv_heads, dim, block, dtype, lo, hi, **more)
    del case["name"]
    return case


# ---- sizes of a case ---------------------------------------------------------------------------------------


def _lengths(case):
    """The sequences' context lengths (a matter of the case, not of the seed)."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    lens = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(17).shuffle(lens)
    return lens


def _new(case, lens):
    """window_prefill: each sequence's number of newest tokens."""
    n, lo, hi = case["seqs"], case["new_lo"], case["new_hi"]
    new = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(18).shuffle(new)
    return [min(a, b) for a, b in zip(new, lens)]


def _es(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    lens, es, H, G, D = _lengths(case), _es(case), case["heads"], case["kv_heads"], case["dim"]
    bs = case["block"]
    n = len(lens)
    if case["op"] == "window_decode":
        seen = sum(min(L, case["sinks"] + case["window"]) for L in lens)
        return {"bytes": 2 * seen * G * D * es + 2 * n * H * D * es + 4 * (seen // bs + n), "flops": 4 * seen * H * D}
    if case["op"] == "score_decode":
        seen = sum(lens)
        return {"bytes": 2 * seen * G * D * es + 2 * n * H * D * es + 8 * seen * G + 4 * (seen // bs + n),
                "flops": 4 * seen * H * D}
    if case["op"] == "window_prefill":
        W, S = case["window"], case["sinks"]
        new = _new(case, lens)
        rows = sum(min(L, min(S, L) + W + q - 1) for L, q in zip(lens, new) if q)
        pairs = 0
        for L, q in zip(lens, new):
            for P in range(L - q, L):
                pairs += min(P + 1, S + W)
        return {"bytes": 2 * sum(new) * H * D * es + 2 * rows * G * D * es, "flops": 4 * pairs * H * D}
    kept = [min(L, case["budget"]) for L in lens]
    # reads the scores, reads and writes the kept rows, their scores and indices
    return {"bytes": G * sum(4 * L + k * (4 * D * es + 8) for L, k in zip(lens, kept)), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------------------


def _tables(case, lens, counts, gen, more_blocks=0):
    """Block tables over a pool of scattered blocks: counts[s] is the set of logical blocks of sequence s that
    are held; -1 elsewhere. Returns (tables, number of blocks, the pool's blocks left over)."""
    bs = case["block"]
    width = max(1, -(-max(lens) // bs))
    total = sum(len(c) for c in counts)
    perm = torch.randperm(total + more_blocks, generator=gen).to(torch.int32)
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for s, c in enumerate(counts):
        if c:
            tables[s, torch.tensor(c)] = perm[at:at + len(c)]
        at += len(c)
    return tables, total + more_blocks, perm[at:]


def prepare(case, seed):
    lens, bs, op = _lengths(case), case["block"], case["op"]
    B, H, G, D, dt = len(lens), case["heads"], case["kv_heads"], case["dim"], _DTYPES[case["dtype"]]
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gpu, dtype=dt)

    held = []
    for L in lens:
        blocks = range(-(-L // bs))
        if op == "window_decode":  # blocks wholly outside the sinks and the window have been given back
            first = max(0, L - case["window"]) // bs
            blocks = [j for j in blocks if j * bs < case["sinks"] or j >= first]
        held.append(list(blocks))
    extra = sum(-(-min(L, case["budget"]) // bs) for L in lens) if op == "evict" else 0
    tables, nb, spare = _tables(case, lens, held, cpu, extra)
    st = dict(case=case, scale=1.0 / math.sqrt(D), max_len=max(lens), tables=tables.cuda(),
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              k=normal(nb, G, bs, D), v=normal(nb, G, bs, D))
    rows = B
    if op == "window_prefill":
        new = _new(case, lens)
        starts = [0]
        for q in new:
            starts.append(starts[-1] + q)
        rows = starts[-1]
        st.update(starts=torch.tensor(starts, dtype=torch.int32, device="cuda"), max_new=max(new))
    if op != "evict":
        st.update(q=normal(rows, H, D), out=torch.zeros(rows, H, D, device="cuda", dtype=dt))
    if op == "score_decode":
        # scores after some ten steps: a few large, most small
        old = torch.rand(B, G, st["max_len"], device="cuda", generator=gpu)
        st.update(scores=H // G / st["max_len"] / (old + 0.05), scores_out=torch.zeros(B, G, st["max_len"], device="cuda"))
    if op == "evict":
        budget = case["budget"]
        # scores of tokens that have been attended to for a while: a few large, most small
        old = torch.rand(B, G, st["max_len"], device="cuda", generator=gpu)
        dst = torch.full((B, tables.shape[1]), -1, dtype=torch.int32)
        at = 0
        for s, L in enumerate(lens):
            n = -(-min(L, budget) // bs)
            dst[s, :n] = spare[at:at + n]
            at += n
        st.update(scores=0.05 / (old + 0.01), scores_out=torch.zeros(B, G, budget, device="cuda"), dst=dst.cuda(),
                  new_lens=torch.zeros(B, dtype=torch.int32, device="cuda"),
                  kept=torch.full((B, G, budget), -1, dtype=torch.int32, device="cuda"))
    if own:
        import paged_kv_cache_204_gb300 as pkv
        st["pkv"] = pkv
        if op == "window_decode":
            st["ws"] = pkv.new_window_workspace(B, H, G, D)
        if op == "score_decode":
            st["ws"] = pkv.new_scores_workspace(B, H, G, D, st["max_len"])
    return st


# ---- one pass --------------------------------------------------------------------------------------------------


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st, op)
    if op == "window_decode":
        return _plain_window_decode(st)
    if op == "window_prefill":
        return _plain_window_prefill(st)
    if op == "score_decode":
        return _plain_score_decode(st)
    return _plain_evict(st)


def _own(st, op):
    pkv, c = st["pkv"], st["case"]
    if op == "window_decode":
        pkv.paged_attention_decode_window(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["scale"],
                                          c["window"], c["sinks"], st["max_len"], st["ws"])
        return st["out"]
    if op == "window_prefill":
        pkv.paged_attention_prefill_window(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"],
                                           st["starts"], st["scale"], c["window"], c["sinks"], st["max_new"])
        return st["out"]
    if op == "score_decode":
        pkv.paged_attention_decode_scores(st["out"], st["scores_out"], st["q"], st["k"], st["v"], st["tables"],
                                          st["lens"], st["scale"], st["max_len"], st["ws"], scores=st["scores"])
        return st["out"], st["scores_out"]
    pkv.evict_tokens(st["k"], st["v"], st["scores"], st["scores_out"], st["tables"], st["dst"], st["lens"],
                     st["new_lens"], st["kept"], c["sinks"], c["recent"], st["max_len"])
    return st["k"], st["v"], st["scores_out"], st["new_lens"], st["kept"]


def _rows(st, pool, pos, ok):
    """Cache rows of the positions pos [B, T] as [B, T, kv heads, dim] in 32 bits (zeros where not ok)."""
    bs = st["case"]["block"]
    block = st["tables"].gather(1, torch.where(ok, pos // bs, 0)).long()
    block = torch.where(ok, block, 0)
    got = pool[block, :, torch.where(ok, pos % bs, 0)].float()
    return torch.where(ok[:, :, None, None], got, 0.0)


def _attend(q, k, v, seen, scale):
    """q [B, N, H, D], k and v [B, T, G, D], seen [B, N, T] -> out [B, N, H, D], weights [B, G, H/G, N, T]."""
    B, N, H, D = q.shape
    G = k.shape[2]
    x = torch.einsum("bngrd,btgd->bgrnt", q.reshape(B, N, G, H // G, D), k) * scale
    x = torch.where(seen[:, None, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    w = e / e.sum(-1, keepdim=True).clamp_min(1e-38)
    return torch.einsum("bgrnt,btgd->bngrd", w, v).reshape(B, N, H, D), w


def _plain_window_decode(st):
    c, L = st["case"], st["lens"].long()[:, None]
    S, n = c["sinks"], torch.clamp(L, max=c["sinks"] + c["window"])
    j = torch.arange(min(st["max_len"], S + c["window"]), device=L.device)[None]
    pos, ok = torch.where(j < S, j, L - n + j), j < n
    k, v = _rows(st, st["k"], pos, ok), _rows(st, st["v"], pos, ok)
    out, _ = _attend(st["q"].float()[:, None], k, v, ok[:, None], st["scale"])
    st["out"].copy_(out[:, 0])
    return st["out"]


def _plain_window_prefill(st):
    c, L = st["case"], st["lens"].long()
    first = st["starts"].long()[:-1]
    n = st["starts"].long()[1:] - first
    i = torch.arange(st["max_new"], device=L.device)[None]
    live = i < n[:, None]
    row = torch.where(live, first[:, None] + i, 0)
    at = (L - n)[:, None] + i                                    # positions of the queries
    t = torch.arange(st["max_len"], device=L.device)
    ok = t[None] < L[:, None]
    k, v = _rows(st, st["k"], t.expand_as(ok), ok), _rows(st, st["v"], t.expand_as(ok), ok)
    seen = (t <= at[..., None]) & ((t < c["sinks"]) | (t > at[..., None] - c["window"])) & ok[:, None]
    out, _ = _attend(st["q"].float()[row], k, v, seen, st["scale"])
    st["out"][row[live]] = out[live].to(st["out"].dtype)
    return st["out"]


def _plain_score_decode(st):
    L = st["lens"].long()[:, None]
    t = torch.arange(st["max_len"], device=L.device)[None]
    ok, t = t < L, t.expand(L.shape[0], -1)
    k, v = _rows(st, st["k"], t, ok), _rows(st, st["v"], t, ok)
    out, w = _attend(st["q"].float()[:, None], k, v, ok[:, None], st["scale"])
    st["out"].copy_(out[:, 0])
    old = torch.where((t < L - 1)[:, None], st["scores"], 0.0)
    st["scores_out"].copy_(torch.where(ok[:, None], old + w[:, :, :, 0].sum(2), st["scores_out"]))
    return st["out"], st["scores_out"]


def _plain_evict(st):
    c, L = st["case"], st["lens"].long()[:, None]
    budget, bs = c["budget"], c["block"]
    t = torch.arange(st["max_len"], device=L.device)[None]
    ok = t < L
    safe = ok & ((t < c["sinks"]) | (t >= L - c["recent"]))
    s = st["scores"].nan_to_num(nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf)
    order = torch.sort(s, dim=-1, descending=True, stable=True).indices
    kind = torch.where(safe, 0, torch.where(ok, 1, 2))[:, None].expand_as(order).gather(2, order)
    order = order.gather(2, torch.sort(kind, dim=-1, stable=True).indices)[:, :, :budget]
    n = torch.clamp(L, max=budget)
    i = torch.arange(order.shape[2], device=L.device)
    live = (i < n)[:, None].expand_as(order)
    pos = torch.sort(torch.where(live, order, st["max_len"]), dim=-1).values
    pos = torch.where(live, pos, 0)
    B, G, K = pos.shape
    g = torch.arange(G, device=L.device)[None, :, None].expand_as(pos)
    src = st["tables"].long()[:, None].expand(B, G, -1).gather(2, pos // bs)
    to = i.expand(B, G, K)
    dst = st["dst"].long()[:, None].expand(B, G, -1).gather(2, to // bs)
    src, dst, off, to_off, g = src[live], dst[live], (pos % bs)[live], (to % bs)[live], g[live]
    st["k"][dst, g, to_off] = st["k"][src, g, off]
    st["v"][dst, g, to_off] = st["v"][src, g, off]
    st["scores_out"][:, :, :K] = torch.where(live, st["scores"].gather(2, pos), st["scores_out"][:, :, :K])
    st["kept"][:, :, :K] = torch.where(live, pos.int(), st["kept"][:, :, :K])
    st["new_lens"].copy_(n[:, 0])
    return st["k"], st["v"], st["scores_out"], st["new_lens"], st["kept"]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------


def exact(case, seed):
    """Each sequence by itself, from the definition, in 64 bits."""
    st = prepare(case, seed)
    lens, bs, H, G, D = _lengths(case), case["block"], case["heads"], case["kv_heads"], case["dim"]
    k, v, tables = st["k"], st["v"], st["tables"].long()
    if case["op"] == "evict":
        k, v = k.clone(), v.clone()
        scores_out, kept = st["scores_out"].double(), st["kept"].long()
        new_lens = torch.tensor([min(L, case["budget"]) for L in lens])
        if sum(lens) * G > 4_000_000:
            return [None, None, None, new_lens, None]
        for s, L in enumerate(lens):
            n, lo, hi = min(L, case["budget"]), case["sinks"], L - case["recent"]
            for h in range(G):
                row = st["scores"][s, h, :L].double().cpu().tolist()
                keep = list(range(L))
                if n < L:
                    middle = sorted(range(lo, hi), key=lambda a: (-row[a], a))[:n - lo - case["recent"]]
                    keep = list(range(lo)) + sorted(middle) + list(range(hi, L))
                a = torch.tensor(keep, device="cuda")
                b = torch.arange(n, device="cuda")
                to, frm = st["dst"][s].long()[b // bs], tables[s, a // bs]
                k[to, h, b % bs], v[to, h, b % bs] = st["k"][frm, h, a % bs], st["v"][frm, h, a % bs]
                scores_out[s, h, :n], kept[s, h, :n] = st["scores"][s, h, a].double(), a
        return [k.double(), v.double(), scores_out, new_lens, kept]

    def dense(pool, s, L):  # [heads, L, D] of one sequence; rows in blocks not held are never seen
        rows = pool[tables[s, :-(-L // bs)].clamp_min(0)].transpose(0, 1).reshape(G, -1, D)[:, :L]
        return rows.double().repeat_interleave(H // G, 0)

    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "score_decode":
        total = st["scores_out"].double()
    new = _new(case, lens) if case["op"] == "window_prefill" else [1] * len(lens)
    first = 0
    for s, L in enumerate(lens):
        kd, vd = dense(k, s, L), dense(v, s, L)
        for a in range(0, new[s], 512):
            b = min(a + 512, new[s])
            q = st["q"][first + a:first + b].double().transpose(0, 1)
            last = torch.arange(L - new[s] + a, L - new[s] + b, device="cuda")[:, None]
            t = torch.arange(L, device="cuda")[None]
            see = t <= last
            if "window" in case:
                see = see & ((last - t < case["window"]) | (t < case["sinks"]))
            p = (q @ kd.transpose(1, 2) * st["scale"]).masked_fill(~see, float("-inf")).softmax(-1)
            out[first + a:first + b] = (p @ vd).transpose(0, 1)
            if case["op"] == "score_decode":
                total[s, :, :L] = p[:, 0].reshape(G, H // G, L).sum(1)
                total[s, :, :L - 1] += st["scores"][s, :, :L - 1].double()
        first += new[s]
    return [out, total] if case["op"] == "score_decode" else out

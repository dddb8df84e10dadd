"""Filling a paged key-value cache with rotated keys, and prompts over caches held in 8 and 4 bits, as a
serving program calls them, for timing and comparison.

Operators:
  append         the step's new tokens: queries and keys turned by their positions, keys and values stored in the
                 slots of a paged cache of 16 or 32 bits
  append_quant   the same into a cache of e4m3 codes or of q4_0 blocks
  append_axes    the same with positions of several axes (time, height, width): each pair of a row turns by the
                 position on its own axis
  prefill_q4     causal attention of every sequence's newest tokens (drafted tokens, chunks, prompts) over a cache of
                 q4_0 blocks
  prefill_fp8    the same over a cache of e4m3 codes

With `own` false, `run` computes them from elementary torch operations in 32 bits; with `own` true it
calls this package's entry points.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_FP8 = torch.float8_e4m3fn


def _append(name, op, tokens, heads, kv_heads, dim, block, dtype, cache, rot, layout="half", sections="", step=False, pad=0):
    """rot: values of a row that turn; layout "half" pairs value i with i + rot / 2, "pairs" 2 i with 2 i + 1;
    sections: pairs of each axis in turn, "" for one axis; step: one token of each of `tokens` sequences, else one
    prompt; pad: idle rows at the end."""
    return dict(name=name, op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype,
                cache=cache, rot=rot, layout=layout, sections=sections, step=step, pad=pad)


def _prefill(name, op, seqs, heads, kv_heads, dim, block, dtype, lo, hi, new_lo, new_hi):
    """Context lengths spread evenly over [lo, hi] and numbers of new tokens over [new_lo, new_hi], each in an order
    of its own."""
    return dict(name=name, op=op, seqs=seqs, heads=heads, kv_heads=kv_heads, dim=dim, block=block, dtype=dtype, lo=lo,
                hi=hi, new_lo=new_lo, new_hi=new_hi)


def listed():
    return [
        # one conversation's next token: the latency of a call
        _append("append_single", "append", 1, 32, 8, 128, 16, "f16", "same", 128, step=True),
        # a full batch's next tokens, full heads, three rows of the fixed batch idle
        _append("append_batch", "append", 128, 40, 40, 128, 16, "bf16", "same", 128, step=True, pad=3),
        # a long prompt with shared heads
        _append("append_prompt", "append", 8192, 32, 8, 128, 16, "bf16", "same", 128),
        # a batch's next tokens into an 8-bit cache; a model that turns half of each row, neighbours as pairs
        _append("append_fp8_batch", "append_quant", 64, 64, 8, 128, 32, "bf16", "fp8", 64, "pairs", step=True),
        # a prompt into a 4-bit cache (the cache is read back as the values that its codes stand for)
        _append("append_q4_prompt", "append_quant", 2777, 32, 8, 128, 16, "f16", "q4", 128),
        # next tokens of conversations about pictures
        _append("append_axes_batch", "append_axes", 100, 32, 8, 128, 16, "bf16", "same", 128, sections="16,24,24", step=True),
        # a prompt of text and pictures
        _append("append_axes_prompt", "append_axes", 4099, 40, 40, 64, 8, "f16", "same", 64, sections="8,12,12"),
        # drafted tokens checked against long 4-bit contexts
        _prefill("prefill_q4_draft", "prefill_q4", 16, 32, 8, 128, 16, "bf16", 4097, 32768, 5, 5),
        # prompts of unequal lengths, full heads
        _prefill("prefill_q4_batch", "prefill_q4", 8, 40, 40, 64, 8, "f16", 300, 1500, 256, 1500),
        # one long prompt, shared heads
        _prefill("prefill_q4_long", "prefill_q4", 1, 32, 8, 128, 16, "bf16", 8192, 8192, 8192, 8192),
        # one chunk of a prompt behind a cached context
        _prefill("prefill_fp8_chunk", "prefill_fp8", 1, 32, 8, 128, 32, "f16", 2777, 2777, 100, 100),
        # chunks of several long prompts
        _prefill("prefill_fp8_batch", "prefill_fp8", 4, 64, 8, 128, 16, "bf16", 1000, 6001, 512, 1024),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append_quant", "append_axes", "prefill_q4", "prefill_q4", "prefill_fp8"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16, 32, 40])
    group = min(rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 12]), max(1, 64 // kv_heads))
    heads, dim, block = kv_heads * group, rng.choice([64, 128, 128]), rng.choice([8, 16, 16, 32])
    if op.startswith("append"):
        cache = rng.choice(["fp8", "q4"]) if op == "append_quant" else "same"
        step = cache != "q4" and rng.random() < 0.4
        tokens = _spread(rng, 1, min(256 if step else 8192, 8192 * 48 * 128 // ((heads + 2 * kv_heads) * dim)))
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        sections = ""
        if op == "append_axes":
            first = rng.randint(1, rot // 2 - 2)
            second = rng.randint(1, rot // 2 - first - 1)
            sections = "%d,%d,%d" % (first, second, rot // 2 - first - second)
        dtype = rng.choice(["f16", "bf16"] if cache != "same" else ["f16", "bf16", "f16", "bf16", "f32"])
        case = _append("", op, tokens, heads, kv_heads, dim, block, dtype, cache, rot, rng.choice(["half", "half", "pairs"]),
                       sections, step, rng.randint(0, 3) if step and tokens > 8 else 0)
    else:
        seqs = _spread(rng, 1, 16)
        if rng.random() < 0.4:  # a few drafted tokens behind long contexts
            new_hi, most = rng.randint(1, 8), min(32768, 400_000_000 // (seqs * kv_heads * dim))
            hi = _spread(rng, 16, most)
        else:
            new_hi = _spread(rng, 9, max(9, min(8192, int(math.sqrt(400_000_000 / (seqs * heads))))))
            hi = _spread(rng, new_hi, max(new_hi, min(32768, 400_000_000 // (seqs * max(heads * new_hi, kv_heads * dim)))))
        lo = _spread(rng, max(1, hi // 8), hi)
        case = _prefill("", op, seqs, heads, kv_heads, dim, block, rng.choice(["f16", "bf16"]), lo, hi, rng.randint(0, new_hi),
                        new_hi)
    del case["name"]
    return case


# ---- sizes of a case ---------------------------------------------------------------------------------------


def _evenly(lo, hi, n, seed):
    got = [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]
    random.Random(seed).shuffle(got)
    return got


def _lengths(case):
    """Context lengths and numbers of new tokens of a prefill (a matter of the case, not of the seed)."""
    lens = _evenly(case["lo"], case["hi"], case["seqs"], 17)
    return lens, [min(a, b) for a, b in zip(_evenly(case["new_lo"], case["new_hi"], case["seqs"], 18), lens)]


def _axes(case):
    return case["sections"].count(",") + 1


def _row_bytes(case):
    cache = {"prefill_q4": "q4", "prefill_fp8": "fp8"}.get(case["op"]) or case["cache"]
    return {"same": (4 if case["dtype"] == "f32" else 2) * case["dim"], "fp8": case["dim"], "q4": case["dim"] // 16 * 9}[cache]


def work(case):
    H, G, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"].startswith("append"):
        T, es = case["tokens"] - case["pad"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * ((2 * H + 2 * G) * D * es + 2 * G * _row_bytes(case) + 4 * case["rot"] + 8 + 4 * _axes(case)),
                "flops": 3 * T * (H + G) * case["rot"]}
    lens, new = _lengths(case)
    pairs = sum(q * (L - q) + q * (q + 1) // 2 for L, q in zip(lens, new))
    rows = sum(L for L, q in zip(lens, new) if q)
    return {"bytes": 4 * sum(new) * H * D + 2 * rows * G * _row_bytes(case) + 4 * (rows // case["block"] + case["seqs"]),
            "flops": 4 * pairs * H * D}


# ---- q4_0 rows -----------------------------------------------------------------------------------------------


def _to_q4(x):
    """Rows of 32-bit values as q4_0 rows: every 32 values share a scale, the first value of largest magnitude over
    -8, stored in binary16 (the scales first); a code is trunc(x / scale + 8.5), at most 15; byte j of a block holds
    the codes j (low half) and j + 16."""
    x = x.float().unflatten(-1, (-1, 32))
    m = x.gather(-1, x.abs().argmax(-1, keepdim=True))
    d = m / -8.0
    inv = torch.where(d == 0, 0.0, 1.0 / torch.where(d == 0, 1.0, d))
    code = (x * inv + 8.5).clamp(0, 15).to(torch.uint8)
    code = (code[..., :16] | (code[..., 16:] << 4)).flatten(-2)
    return torch.cat([d[..., 0].half().view(torch.uint8), code], -1)


def _from_q4(rows):
    """The values that q4_0 rows of 9 D / 16 bytes stand for."""
    n = rows.shape[-1] // 9
    d = rows[..., :n].contiguous().view(torch.float16)
    code = rows[..., n:].unflatten(-1, (-1, 16))
    code = torch.cat([code & 15, code >> 4], -1).float() - 8.0
    return (code * d[..., None].float()).flatten(-2)


# ---- inputs --------------------------------------------------------------------------------------------------


def _table(positions, rot):
    """Cosines, then sines of position * 10000^(-2 i / rot): angles in 64 bits, as far positions need."""
    turn = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * turn
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _prepare_append(case, cpu, gpu):
    T, live, H, G, D, bs = case["tokens"], case["tokens"] - case["pad"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    dt = _DTYPES[case["dtype"]]
    if case["step"]:  # every sequence's newest token somewhere in a block of its own
        nb = 2 * T + 1
        pos = torch.randint(16, 2049, (live,), generator=cpu)
        slots = torch.randperm(nb, generator=cpu)[:live] * bs + pos % bs
    else:             # a prompt's tokens in scattered blocks
        nb = -(-T // bs) + 1
        pos = torch.arange(live)
        slots = torch.randperm(nb, generator=cpu)[pos // bs] * bs + pos % bs
    pos = pos.repeat(_axes(case), 1)
    if _axes(case) > 1 and not case["step"]:
        # text, then pictures of 24 x 32 patches in turn: time stands still, rows and columns run
        patch = torch.arange(live) - 64
        picture = patch.clamp_min(0) // 768
        inside = torch.stack([torch.zeros_like(patch), patch % 768 // 32, patch % 32])
        pos = torch.where(patch < 0, pos, 64 + 33 * picture + inside)
    idle = torch.full((case["pad"],), -1)
    positions = torch.cat([pos, idle.repeat(_axes(case), 1)], 1).int()
    # queries, keys and values lie side by side, as one product gives them
    qkv = torch.randn(T, H + 2 * G, D, device="cuda", generator=gpu, dtype=dt)
    st = dict(q=qkv[:, :H], k=qkv[:, H:H + G], v=qkv[:, H + G:], q_out=torch.zeros(T, H, D, device="cuda", dtype=dt),
              slots=torch.cat([slots, idle]).cuda(), positions=positions.cuda(),
              table=_table(max(4096, T), case["rot"]))
    if case["sections"]:
        st["axis"] = [a for a, n in enumerate(case["sections"].split(",")) for _ in range(int(n))]
    for name in ("k_cache", "v_cache"):
        old = torch.randn(nb, G, bs, D, device="cuda", generator=gpu, dtype=dt)
        st[name] = {"same": lambda: old, "fp8": lambda: (old / 0.02).to(_FP8).view(torch.uint8), "q4": lambda: _to_q4(old)}[case["cache"]]()
    if case["cache"] == "fp8":
        st.update(k_scale=0.02, v_scale=0.015)
    return st


def _prepare_prefill(case, cpu, gpu):
    lens, new = _lengths(case)
    B, H, G, D, bs, dt = len(lens), case["heads"], case["kv_heads"], case["dim"], case["block"], _DTYPES[case["dtype"]]
    counts = [-(-L // bs) for L in lens]
    nb = sum(counts) + 1
    perm = torch.randperm(nb, generator=cpu).int()
    tables = torch.full((B, max(counts)), -1, dtype=torch.int32)
    starts, at = [0], 0
    for s, c in enumerate(counts):
        tables[s, :c] = perm[at:at + c]
        at += c
        starts.append(starts[-1] + new[s])
    st = dict(scale=1.0 / math.sqrt(D), max_len=max(lens), max_new=max(new), tables=tables.cuda(),
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
              q=torch.randn(starts[-1], H, D, device="cuda", generator=gpu, dtype=dt),
              out=torch.zeros(starts[-1], H, D, device="cuda", dtype=dt))
    for name in ("k_cache", "v_cache"):
        rows = torch.randn(nb, G, bs, D, device="cuda", generator=gpu, dtype=dt)
        st[name] = _to_q4(rows) if case["op"] == "prefill_q4" else (rows / 0.02).to(_FP8).view(torch.uint8)
    if case["op"] == "prefill_fp8":
        st.update(k_scale=0.02, v_scale=0.02)
    return st


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gpu = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"].startswith("append"):
        st = _prepare_append(case, cpu, gpu)
    else:
        st = _prepare_prefill(case, cpu, gpu)
    st["case"] = case
    if own:
        import paged_kv_cache_204_gb300 as pkv
        st["pkv"] = pkv
        if "axis" in st:
            st["axis"] = bytes(st["axis"])
        if case["op"].startswith("prefill"):
            st["ws"] = pkv.new_prefill_workspace(case["dim"])
    elif "axis" in st:
        st["axis"] = torch.tensor(st["axis"], device="cuda")
    return st


# ---- one pass --------------------------------------------------------------------------------------------------


def run(st):
    append = st["case"]["op"].startswith("append")
    if own:
        return _own_append(st) if append else _own_prefill(st)
    return _plain_append(st) if append else _plain_prefill(st)


def _filled(st):
    """The caches as the values that they stand for."""
    cache, k, v = st["case"]["cache"], st["k_cache"], st["v_cache"]
    if cache == "fp8":
        return st["q_out"], k.view(_FP8), v.view(_FP8)
    if cache == "q4":
        return st["q_out"], _from_q4(k).half(), _from_q4(v).half()
    return st["q_out"], k, v


def _own_append(st):
    pkv, c = st["pkv"], st["case"]
    more = dict(pair_axis=st.get("axis"), interleaved=c["layout"] == "pairs")
    args = [st[n] for n in ("q_out", "q", "k", "v", "k_cache", "v_cache", "slots", "positions", "table")]
    if c["cache"] == "fp8":
        pkv.rope_and_cache_fp8(*args, st["k_scale"], st["v_scale"], **more)
    elif c["cache"] == "q4":
        pkv.rope_and_cache_q4_0(*args, **more)
    else:
        pkv.rope_and_cache(*args, **more)
    return _filled(st)


def _own_prefill(st):
    pkv = st["pkv"]
    args = [st[n] for n in ("out", "q", "k_cache", "v_cache", "tables", "lens", "starts", "scale")]
    if st["case"]["op"] == "prefill_fp8":
        pkv.paged_attention_prefill_fp8(*args, st["k_scale"], st["v_scale"], st["max_new"], st["ws"])
    else:
        pkv.paged_attention_prefill_q4_0(*args, st["max_new"], st["ws"])
    return st["out"]


def _turned(x, cos, sin, rot, layout):
    """x [T, heads, D] in 32 bits with its first rot values turned; cos, sin [T, 1, rot / 2]."""
    a, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = a[..., :rot // 2], a[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = a[..., 0::2], a[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_append(st):
    c, bs, half = st["case"], st["case"]["block"], st["case"]["rot"] // 2
    live = st["positions"][0] >= 0
    pos = st["positions"].long().clamp_min(0)
    cos, sin = st["table"][:, :half], st["table"][:, half:]
    if "axis" in st:
        pair = torch.arange(half, device=pos.device)
        pos = pos[st["axis"]].T                      # [T, pairs]
        cos, sin = cos[pos, pair][:, None], sin[pos, pair][:, None]
    else:
        cos, sin = cos[pos[0]][:, None], sin[pos[0]][:, None]
    q = _turned(st["q"].float(), cos, sin, c["rot"], c["layout"])
    k, v = _turned(st["k"].float(), cos, sin, c["rot"], c["layout"]), st["v"].float()
    st["q_out"].copy_(torch.where(live[:, None, None], q, st["q_out"]))
    slots = st["slots"]
    if c["pad"]:
        slots, k, v = slots[live], k[live], v[live]
    for pool, x, scale in ((st["k_cache"], k, st.get("k_scale")), (st["v_cache"], v, st.get("v_scale"))):
        if c["cache"] == "fp8":
            x = (x / torch.tensor(scale, dtype=torch.float32, device=x.device)).clamp(-448, 448).to(_FP8).view(torch.uint8)
        elif c["cache"] == "q4":
            x = _to_q4(x)
        pool[slots // bs, :, slots % bs] = x.to(pool.dtype)
    return _filled(st)


def _plain_prefill(st):
    c, L = st["case"], st["lens"].long()
    B, H, G, D, bs = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["block"]
    first = st["starts"].long()[:-1]
    n = st["starts"].long()[1:] - first
    i = torch.arange(st["max_new"], device=L.device)[None]
    live = i < n[:, None]
    row = torch.where(live, first[:, None] + i, 0)
    at = (L - n)[:, None] + i                        # positions of the queries
    t = torch.arange(st["max_len"], device=L.device)
    held = t[None] < L[:, None]
    block = torch.where(held, st["tables"].long().gather(1, (t // bs)[None].expand(B, -1)), 0)

    def rows(pool, scale):  # [B, T, G, D]
        got = pool[block, :, t % bs]
        got = _from_q4(got) if scale is None else got.view(_FP8).float() * scale
        return torch.where(held[:, :, None, None], got, 0.0)

    k, v = rows(st["k_cache"], st.get("k_scale")), rows(st["v_cache"], st.get("v_scale"))
    q = st["q"].float()[row].reshape(B, -1, G, H // G, D)
    x = torch.einsum("bngrd,btgd->bgrnt", q, k) * st["scale"]
    seen = (t <= at[..., None]) & held[:, None] & live[..., None]
    x = torch.where(seen[:, None, None], x, -torch.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -torch.inf, 0.0, top))
    x = x / x.sum(-1, keepdim=True).clamp_min(1e-38)
    out = torch.einsum("bgrnt,btgd->bngrd", x, v).reshape(B, -1, H, D)
    st["out"][row[live]] = out[live].to(st["out"].dtype)
    return st["out"]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------


def _exact_append(case, st):
    D, G, rot, bs = case["dim"], case["kv_heads"], case["rot"], case["block"]
    positions, table, slots = st["positions"].tolist(), st["table"].double(), st["slots"].tolist()
    counts = [int(n) for n in case["sections"].split(",")] if case["sections"] else [rot // 2]
    axis = sum(([a] * n for a, n in enumerate(counts)), [])
    alive = [t for t in range(case["tokens"]) if positions[0][t] >= 0]
    # the angle of pair i of token t as a complex number
    turn = torch.empty(len(alive), 1, rot // 2, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(axis):
        p = torch.tensor([positions[a][t] for t in alive], device="cuda")
        turn[:, 0, i] = torch.complex(table[p, i], table[p, rot // 2 + i])

    def turned(x):
        x = x[alive].double().clone()
        pairs = x[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else x[..., :rot].unflatten(-1, (-1, 2))
        got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        x[..., :rot] = got.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else got.flatten(-2)
        return x

    q_out = st["q_out"].double()
    q_out[alive] = turned(st["q"])
    at = torch.tensor([slots[t] for t in alive], device="cuda")
    outs = [q_out]
    for name, x in (("k", turned(st["k"])), ("v", st["v"][alive].double())):
        pool = st[name + "_cache"]
        if case["cache"] == "same":
            pool = pool.double()
        elif case["cache"] == "fp8":
            pool = pool.view(_FP8).double()
            x = (x / st[name + "_scale"]).clamp(-448.0, 448.0)
            # steps of 2^-3 of the value's power of two, 2^-9 below 2^-6; torch.round takes halves to even
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
            x = torch.round(x / step) * step
        else:
            bits = pool.reshape(-1, pool.shape[-1])
            d = bits[:, :D // 16].contiguous().view(torch.float16).double()
            low, high = (bits[:, D // 16:] % 16).double(), (bits[:, D // 16:] // 16).double()
            old = torch.empty(bits.shape[0], D // 32, 2, 16, dtype=torch.float64, device="cuda")
            old[:, :, 0], old[:, :, 1] = low.view(-1, D // 32, 16), high.view(-1, D // 32, 16)
            pool = ((old - 8) * d[:, :, None, None]).view(*pool.shape[:-1], D)
            x = x.view(*x.shape[:-1], D // 32, 32)
            big = x.abs().amax(-1, keepdim=True)
            firsts = (x.abs() == big).long().argmax(-1, keepdim=True)
            d = -torch.take_along_dim(x, firsts, -1) / 8
            code = torch.where(d == 0, 8.0, torch.floor(x / torch.where(d == 0, 1.0, d) + 8.5).clamp(0, 15))
            x = ((code - 8) * d.half().double()).flatten(-2)
        pool[at // bs, :, at % bs] = x
        outs.append(pool)
    return outs


def _exact_prefill(case, st):
    lens, new = _lengths(case)
    H, G, D, bs = case["heads"], case["kv_heads"], case["dim"], case["block"]

    def dense(name, s, L):  # [heads, L, D] of one sequence
        rows = st[name + "_cache"][st["tables"][s, :-(-L // bs)].long()].transpose(0, 1).flatten(1, 2)[:, :L]
        if case["op"] == "prefill_fp8":
            rows = rows.contiguous().view(_FP8).double() * st[name + "_scale"]
        else:
            d = rows[..., :D // 16].contiguous().view(torch.float16).double().repeat_interleave(16, -1)
            codes = rows[..., D // 16:].long()
            low, high = ((codes % 16 - 8) * d).unflatten(-1, (-1, 16)), ((codes // 16 - 8) * d).unflatten(-1, (-1, 16))
            rows = torch.stack([low, high], -2).flatten(-3)
        return rows.repeat_interleave(H // G, 0)

    out, first = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), 0
    for s, L in enumerate(lens):
        k, v = dense("k", s, L), dense("v", s, L)
        for a in range(0, new[s], 512):
            b = min(a + 512, new[s])
            q = st["q"][first + a:first + b].double().transpose(0, 1)
            last = torch.arange(L - new[s] + a, L - new[s] + b, device="cuda")[:, None]
            p = q @ k.transpose(1, 2) * st["scale"]
            p = p.masked_fill(torch.arange(L, device="cuda")[None] > last, float("-inf")).softmax(-1)
            out[first + a:first + b] = (p @ v).transpose(0, 1)
        first += new[s]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(case, st) if case["op"].startswith("append") else _exact_prefill(case, st)

"""Prefill over fp8 and q4_0 caches on the GPU against plain 64-bit attention:
every type, head layout and block size, lengths at tile, block and split
borders, poison in every place that must not be read, values at the ends of
the types' ranges, the device error word, streams, graphs, and sessions that
write, attend and decode together."""
import numpy as np
import pytest
import torch

from quant_helpers import DEV, TD, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_204_gb300 as m
    return m


def new_err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


COMBOS = [  # kind, dtype, head_dim, block_size, kv heads, group
    ("q4", "bf16", 128, 16, 2, 4), ("q4", "f16", 128, 8, 1, 1), ("q4", "bf16", 64, 32, 1, 3), ("q4", "f16", 64, 16, 2, 8),
    ("q4", "f16", 128, 32, 1, 12), ("q4", "bf16", 64, 8, 3, 1), ("q4", "bf16", 128, 16, 1, 19),
    ("fp8", "bf16", 128, 16, 2, 4), ("fp8", "f16", 128, 32, 1, 1), ("fp8", "bf16", 64, 8, 1, 5), ("fp8", "f16", 64, 16, 2, 7),
    ("fp8", "f16", 128, 8, 3, 2), ("fp8", "bf16", 64, 32, 1, 16),
]
BATCHES = {
    "short": [(0, 0), (1, 1), (2, 1), (7, 7), (8, 0), (9, 3), (16, 16), (31, 30), (33, 1)],
    "tiles": [(127, 127), (128, 128), (129, 129), (128, 1), (129, 1), (257, 2), (255, 255), (385, 130)],
    "long": [(1000, 257), (513, 513), (2047, 100), (3000, 5), (0, 0), (1537, 1)],
    "one": [(700, 700)],
    "far": [(20011, 3)],
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("combo", COMBOS, ids=lambda c: "_".join(map(str, c)))
def test_against_64_bits(pkv, combo, batch):
    kind, dtype, D, bs, Hkv, G = combo
    b = Batch(BATCHES[batch], Hkv, G, D, bs, dtype, kind, seed=len(batch))
    err = new_err()
    out = b.run(pkv, err=err)
    b.check(out, batch)
    assert err.item() == 0


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_ragged_batches(pkv, kind):
    """Many sequences, many of them idle, of lengths apart by orders; a table far wider than any of them."""
    rng = np.random.default_rng(5)
    for dtype, D, Hkv, G in (("bf16", 128, 2, 2), ("f16", 64, 1, 4)):
        seqs = []
        for _ in range(300):
            L = int(np.exp(rng.uniform(0, np.log(1500))))
            seqs.append((L, int(rng.integers(0, L + 1)) if rng.random() < 0.1 else int(rng.integers(0, 3)) if L > 3 else 0))
        b = Batch(seqs, Hkv, G, D, 16, dtype, kind, seed=D)
        b.bt = np.concatenate([b.bt, np.full((len(seqs), 5000), -1, np.int32)], 1)
        b.tables = torch.from_numpy(b.bt).to(DEV)
        err = new_err()
        out = b.run(pkv, err=err, max_new=40000)
        b.check(out)
        assert err.item() == 0


@pytest.mark.parametrize("kind", ["q4", "fp8"])
@pytest.mark.parametrize("scale", [0.0, -0.11, 1e-30, 1.7])
def test_scales(pkv, kind, scale):
    for dtype, D in (("bf16", 128), ("f16", 64)):
        b = Batch([(300, 70), (129, 2), (1, 1)], 2, 3, D, 16, dtype, kind, seed=3, scale=scale, q_sigma=0.3)
        b.check(b.run(pkv), scale)


@pytest.mark.parametrize("kind", ["q4", "fp8"])
@pytest.mark.parametrize("sigma,q_sigma", [(3e-3, 1.0), (400.0, 0.01), (1.0, 1e-3), (1.0, 8.0)])
def test_magnitudes(pkv, kind, sigma, q_sigma):
    for dtype in TD:
        b = Batch([(600, 100), (2000, 2)], 1, 4, 128, 16, dtype, kind, seed=4, sigma=sigma, q_sigma=q_sigma)
        b.check(b.run(pkv), (sigma, q_sigma))


@pytest.mark.parametrize("kind", ["q4", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sigma,q_sigma", [(1.0, 0.5), (1.0, 2.0), (0.03, 60.0)])
def test_size_of_the_error(pkv, kind, D, sigma, q_sigma):
    """Over many binary16 outputs the error is within 1.5 times what rounding the exact result leaves. One operand of
    P V is rounded to binary16 on the way (V of q4_0, P over e4m3), by the same 2^-11 / 3^.5 times the rms of the
    values' 1 / mantissa (0.74 where mantissas are spread evenly over their logarithm) as the outputs are; its signs are
    independent, so that it is as large again relative to the output: a factor of 2^.5. The other
    errors are 2^-20 of a weight or less. One more such operand would make it 3^.5. (Keys of 0.03: what their rounding
    leaves is below binary16's normal range, and counts all the same.)"""
    b = Batch([(1500, 200), (333, 333), (900, 1)], 2, 3, D, 16, "f16", kind, seed=12, sigma=sigma, q_sigma=q_sigma)
    out, err, own = b.run(pkv).double(), 0.0, 0.0
    for s, n in enumerate(b.new):
        want, _ = b.exact(s, 0, n)
        err += (out[b.first[s]:b.first[s] + n] - want).square().sum()
        own += (want.half().double() - want).square().sum()
    assert err <= 1.5 ** 2 * own, f"{(err / own).sqrt().item():.3f} times the rounding"


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_bfloat16_queries_beyond_binary16(pkv, kind):
    """Rows of 1e30 and of 1e-30 beside ordinary ones, each scaled by itself."""
    b = Batch([(400, 40)], 2, 2, 64, 16, "bf16", kind, seed=6)
    b.q[::3] *= 2.0 ** 100
    b.q[1::3] *= 2.0 ** -100
    b.scale = 2.0 ** -103
    out = b.run(pkv)
    b.check(out)
    b.q[:] = 0
    b.check(b.run(pkv))


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_one_token_far_above_the_rest(pkv, kind):
    """A weight near 1 beside thousands some 2^-20 of it, which add up."""
    b = Batch([(9000, 2)], 1, 1, 64, 16, "f16", kind, seed=7)
    q = b.q.double()
    x = (q.transpose(0, 1) @ b.k_rows[0].transpose(1, 2))[0, :, :8000]
    b.scale = float(20 * np.log(2) / (x.amax() - x.mean()))
    b.check(b.run(pkv))


def test_infinite_and_nan_keys_and_values_outside(pkv):
    """Rows behind the last token hold NaN (the poison of every batch); here the last block's rows too, block sizes
    where they share a tile's boxes with seen rows."""
    for kind in ("q4", "fp8"):
        for bs in (8, 16, 32):
            b = Batch([(L, min(L, 3)) for L in (1, 5, 9, 17, 33, 65, 121, 131)], 1, 2, 128, bs, "bf16", kind, seed=bs)
            b.check(b.run(pkv), bs)


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_bad_lengths_and_blocks(pkv, kind):
    b = Batch([(100, 10), (50, 5), (200, 20), (60, 6), (70, 7)], 2, 2, 128, 16, "bf16", kind)
    out = torch.full_like(b.q, 7.0)
    err = new_err()
    good = b.run(pkv)
    for bad in (4, 16 * b.bt.shape[1] + 1, -1, (1 << 31) - 1, -(1 << 31)):
        b.context[1] = bad
        out.fill_(7.0)
        err.zero_()
        b.run(pkv, err=err, out=out)
        assert err.item() == pkv.DEV_ERR_CONTEXT_LEN
        assert (out[10:15] == 7).all() and torch.equal(out[:10], good[:10]) and torch.equal(out[15:], good[15:])
    b.context[1] = 50
    err.zero_()
    out.fill_(7.0)
    b.run(pkv, err=err, out=out, max_new=19)  # the third has 20
    assert err.item() == pkv.DEV_ERR_CONTEXT_LEN
    assert (out[15:35] == 7).all() and torch.equal(out[:15], good[:15]) and torch.equal(out[35:], good[35:])
    starts = b.starts.clone()
    b.starts[2] = 8  # the second's queries run backwards, the third's are 27
    err.zero_()
    out.fill_(7.0)
    b.run(pkv, err=err, out=out, max_new=20)
    assert err.item() == pkv.DEV_ERR_CONTEXT_LEN and torch.equal(out[35:], good[35:])
    b.starts = starts
    for bad in (-1, b.nb, 1 << 30, -(1 << 31)):
        b.tables = torch.from_numpy(b.bt).to(DEV)
        b.tables[2, 3] = bad
        err.zero_()
        out.fill_(float("nan"))
        b.run(pkv, err=err, out=out)
        assert err.item() == pkv.DEV_ERR_BLOCK_ID
        # its rows count as zeros
        keep = b.k_rows[2].clone(), b.v_rows[2].clone()
        b.k_rows[2][:, 48:64] = 0
        b.v_rows[2][:, 48:64] = 0
        b.check(out)
        b.k_rows[2], b.v_rows[2] = keep


def test_one_workspace_serves_all_sizes(pkv):
    ws = pkv.new_prefill_workspace(128)
    ws.fill_(0xFF)
    for i, (kind, D, batch) in enumerate([("q4", 128, "far"), ("fp8", 64, "long"), ("q4", 64, "tiles"), ("fp8", 128, "far"),
                                          ("q4", 128, "one"), ("fp8", 128, "short"), ("q4", 128, "far")]):
        b = Batch(BATCHES[batch], 2, 2, D, 16, "bf16", kind, seed=i)
        b.check(b.run(pkv, ws=ws), (i, batch))


@pytest.mark.parametrize("kind", ["q4", "fp8"])
@pytest.mark.parametrize("batch", ["far", "long"])
def test_equal_calls_give_equal_bits(pkv, kind, batch):
    b = Batch(BATCHES[batch], 2, 4, 128, 16, "f16", kind)
    ws = pkv.new_prefill_workspace(128)
    first = b.run(pkv, ws=ws)
    for _ in range(10):
        assert torch.equal(b.run(pkv, ws=ws), first)


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_streams_and_graphs(pkv, kind):
    """Two streams with a workspace each; a graph replayed with other lengths and queries."""
    a, b = Batch([(5000, 5), (300, 300)], 2, 4, 128, 16, "bf16", kind, seed=1), Batch([(9000, 2)], 4, 1, 64, 8, "f16", kind, seed=2)
    wa, wb = pkv.new_prefill_workspace(128), pkv.new_prefill_workspace(64)
    oa, ob = torch.empty_like(a.q), torch.empty_like(b.q)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.run(pkv, ws=wa, out=oa, stream=s)
        b.run(pkv, ws=wb, out=ob, stream=t)
    torch.cuda.synchronize()
    a.check(oa)
    b.check(ob)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(pkv, ws=wa, out=oa, max_new=300)
    a.context.copy_(torch.tensor([4000, 280], dtype=torch.int32))
    a.starts.copy_(torch.tensor([0, 9, 250], dtype=torch.int32))
    a.seqs, a.first = [(4000, 9), (280, 241)], np.array([0, 9, 250])
    a.k_rows = [a.k_rows[0][:, :4000], a.k_rows[1][:, :280]]
    a.v_rows = [a.v_rows[0][:, :4000], a.v_rows[1][:, :280]]
    a.q.mul_(0.5)
    oa.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    a.check(oa)
    assert (oa[250:] == 7).all()  # rows behind the last sequence stay as they were


@pytest.mark.parametrize("kind,dtype,D,bs", [("fp8", "bf16", 128, 16), ("q4", "f16", 128, 32), ("q4", "bf16", 64, 8)])
def test_session(pkv, kind, dtype, D, bs):
    """Prompts written with their rotation and attended in chunks, then drafted tokens, then single ones, over blocks
    that the block manager hands out: a chunked prefill gives what one call gives, and a prefill of one token what
    decode gives, up to their roundings."""
    from paged_kv_cache_204_gb300.block_manager import BlockManager
    H, G, lens = 8, 2, [150, 37, 300]
    width = D if kind == "fp8" else D // 16 * 9
    gen = torch.Generator(device=DEV).manual_seed(1)
    table, ws = pkv.rope_table(1000, D), pkv.new_prefill_workspace(D)
    scale, scales = D ** -0.5, (0.02, 0.02)
    write, prefill, decode = ((pkv.rope_and_cache_fp8, pkv.paged_attention_prefill_fp8, pkv.paged_attention_decode_fp8) if kind == "fp8" else
                              (pkv.rope_and_cache_q4_0, pkv.paged_attention_prefill_q4_0, pkv.paged_attention_decode_q4_0))
    more = scales if kind == "fp8" else ()
    with BlockManager(200, bs, seed=1) as bm:
        nb = 200
        k, v = (torch.full((nb, G, bs, width), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2))
        ids, held = [bm.add_seq() for _ in lens], [0] * 3
        rows = [torch.randn(320, H + 2 * G, D, device=DEV, generator=gen).to(TD[dtype]) for _ in lens]

        def step(new):
            slots = np.concatenate([bm.append(s, n)[0] for s, n in zip(ids, new) if n])
            pos = np.concatenate([np.arange(a, a + n) for a, n in zip(held, new)]).astype(np.int32)
            x = torch.cat([r[a:a + n] for r, a, n in zip(rows, held, new)])
            q = torch.empty(len(pos), H, D, device=DEV, dtype=TD[dtype])
            err = new_err()
            write(q, x[:, :H], x[:, H:H + G], x[:, H + G:], k, v, torch.from_numpy(slots.astype(np.int64)).to(DEV),
                  torch.from_numpy(pos).to(DEV), table, *more, dev_err=err)
            for i, n in enumerate(new):
                held[i] += n
            tables, context = bm.export(ids, 320 // bs + 1)
            tables, context = torch.from_numpy(tables).to(DEV), torch.from_numpy(context).to(DEV)
            starts = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(DEV)
            out = torch.empty_like(q)
            prefill(out, q, k, v, tables, context, starts, scale, *more, max(new), ws, dev_err=err)
            assert err.item() == 0 and context.tolist() == held
            return q, out, tables, context, starts

        chunks = [step([100, 37, 100]), step([50, 0, 200])]
        q = torch.cat([chunks[0][0][:100], chunks[1][0][:50], chunks[0][0][100:137], chunks[0][0][137:], chunks[1][0][50:]])
        got = torch.cat([chunks[0][1][:100], chunks[1][1][:50], chunks[0][1][100:137], chunks[0][1][137:], chunks[1][1][50:]])
        whole = torch.empty_like(q)
        _, _, tables, context, _ = chunks[1]
        prefill(whole, q, k, v, tables, context, torch.tensor([0, 150, 187, 487], dtype=torch.int32, device=DEV), scale,
                *more, 300, ws)
        # twice the bound of one against 64 bits: weights and V off by 2^-11 each, logits by some 2^-10 at these
        # sizes, the output's half step; values of some 1 to 3
        tol = 2 * (2.0 ** -8 * 4 + torch.finfo(TD[dtype]).eps / 2 * 4)
        assert (got.double() - whole.double()).abs().max() <= tol
        step([4, 3, 5])
        for _ in range(3):
            q, out, tables, context, _ = step([1, 1, 1])
            want = torch.empty_like(out)
            decode(want, q, k, v, tables, context, scale, *more, 320, pkv.new_workspace(3, H, D, 320))
            assert (out.double() - want.double()).abs().max() <= tol


@pytest.mark.parametrize("kind,batch", [("q4", "long"), ("fp8", "far"), ("q4", "short")])
def test_gives_up_on_a_wait(pkv, kind, batch):
    """With a limit of 0 any wait not over at its first test gives up: the call reports it and the next one works."""
    b = Batch(BATCHES[batch], 2, 4, 128, 16, "bf16", kind)
    ws = pkv.new_prefill_workspace(128)
    good = b.run(pkv, ws=ws)
    old, err = pkv.get_wait_timeout_ns(), new_err()
    try:
        pkv.set_wait_timeout_ns(0)
        b.run(pkv, ws=ws, err=err)
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_timeout_ns(old)
    assert int(err.item()) == pkv.DEV_ERR_TIMEOUT
    err.zero_()
    got = b.run(pkv, ws=ws, err=err)
    assert int(err.item()) == 0
    live = torch.isfinite(good.float())
    assert torch.equal(got[live], good[live])


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_blocks_past_four_gigabytes(pkv, kind):
    """Blocks at the far end of pools of more than 2^32 bytes."""
    b = Batch([(300, 40), (77, 1)], 8, 2, 128, 16, "bf16", kind, seed=9)
    row = 128 if kind == "fp8" else 72
    nb = (1 << 32) // (8 * 16 * row) + 1000
    far = nb - b.nb
    for name in ("k", "v"):
        pool = torch.empty(nb, 8, 16, row, dtype=torch.uint8, device=DEV)
        pool[far:] = getattr(b, name)
        setattr(b, name, pool)
    b.tables = torch.where(b.tables >= 0, b.tables + far, b.tables)
    b.nb = nb
    err = new_err()
    b.check(b.run(pkv, err=err))
    assert err.item() == 0


def test_extra_rows_of_queries_and_wide_tables(pkv):
    """Output rows behind the last sequence and table entries behind a sequence's blocks are left alone."""
    b = Batch([(500, 60), (40, 3)], 2, 2, 64, 8, "f16", "q4", seed=11)
    q = torch.cat([b.q, torch.full((9, b.H, 64), float("nan"), device=DEV, dtype=b.dtype)])
    out = torch.full_like(q, 3.0)
    b.q = q
    b.bt[0, 500 // 8 + 1:] = 1 << 30
    b.tables = torch.from_numpy(b.bt).to(DEV)
    err = new_err()
    b.run(pkv, err=err, out=out)
    b.check(out)
    assert err.item() == 0 and (out[63:] == 3).all()


def test_binding_refusals(pkv):
    b = Batch([(100, 10)], 2, 2, 64, 16, "bf16", "q4")
    ws, out = pkv.new_prefill_workspace(64), torch.empty_like(b.q)
    good = dict(out=out, q=b.q, k_cache=b.k, v_cache=b.v, block_tables=b.tables, context_lens=b.context, query_start=b.starts,
                scale=b.scale, max_query_len=10, workspace=ws)
    for name, bad in (("q", b.q.transpose(0, 1)), ("q", b.q.cpu()), ("q", b.q[0]), ("out", out.half()), ("out", out[:5]),
                      ("k_cache", b.k.bfloat16()), ("v_cache", b.v[:1]), ("k_cache", b.k.cpu()), ("block_tables", b.tables.long()),
                      ("block_tables", b.tables[0]), ("context_lens", b.context.long()), ("context_lens", b.starts),
                      ("query_start", b.context), ("workspace", ws.cpu()), ("workspace", None), ("max_query_len", 1 << 40)):
        with pytest.raises((ValueError, TypeError)):
            pkv.paged_attention_prefill_q4_0(**{**good, name: bad})
    with pytest.raises(ValueError):  # e4m3 rows are head_dim bytes
        pkv.paged_attention_prefill_fp8(**{k: v for k, v in good.items()}, k_scale=1.0, v_scale=1.0)
    both = torch.empty(15, b.H, 64, device=DEV, dtype=b.dtype)
    for q, o in ((b.q, b.q), (both[:10], both[5:])):
        with pytest.raises(ValueError, match="overlap"):
            pkv.paged_attention_prefill_q4_0(**{**good, "q": q, "out": o})
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_attention_prefill_q4_0(**{**good, "workspace": ws[:100]})
    assert e.value.status == pkv.PKV_ERR_WORKSPACE


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_every_negative_block_id_is_reported(pkv, kind):
    """A visible entry of any negative value, in a sequence's first, middle and last tile and in a last block of one
    token; entries that no query of the call sees may have any value."""
    for dtype, D in (("bf16", 128), ("f16", 128), ("f16", 64)):
        b = Batch([(400, 10), (50, 5), (257, 3)], 2, 2, D, 16, dtype, kind, seed=13)
        for bad in (-2, -1, -3, -17, -(1 << 31), b.nb):
            for s, at in ((0, 0), (0, 11), (0, 24), (1, 3), (2, 16)):
                b.tables = torch.from_numpy(b.bt).to(DEV)
                b.tables[s, at] = bad
                b.tables[s, -(-b.lens[s] // 16):] = bad
                err = new_err()
                out = b.run(pkv, err=err)
                assert err.item() == pkv.DEV_ERR_BLOCK_ID, (bad, s, at)
                keep = b.k_rows[s], b.v_rows[s]
                b.k_rows[s], b.v_rows[s] = keep[0].clone(), keep[1].clone()
                b.k_rows[s][:, 16 * at:16 * at + 16] = 0  # its rows count as zeros
                b.v_rows[s][:, 16 * at:16 * at + 16] = 0
                b.check(out, (bad, s, at))
                b.k_rows[s], b.v_rows[s] = keep
        b.tables = torch.from_numpy(b.bt).to(DEV)
        for s, L in enumerate(b.lens):
            b.tables[s, -(-L // 16):] = -2
        err = new_err()
        b.check(b.run(pkv, err=err))
        assert err.item() == 0


@pytest.mark.parametrize("kind,dtype", [("q4", "f16"), ("fp8", "bf16")])
@pytest.mark.parametrize("seqs", [[(16384, 16384)], [(16384, 16000), (1, 1), (16000, 3), (9000, 9000)]], ids=["one", "four"])
def test_costs_beyond_30_bits(pkv, kind, dtype, seqs):
    """Batches of more than 2^30 in tokens of walks x query heads of a kv head, whose stretches are measured in coarser steps:
    every row is written, and rows at borders of pairs and all over the walk hold what they should."""
    b = Batch(seqs, 1, 64, 64, 16, dtype, kind, seed=15)
    err = new_err()
    out = b.run(pkv, err=err)
    assert err.item() == 0
    rng = np.random.default_rng(16)
    for s, (L, n) in enumerate(b.seqs):
        for a in range(b.first[s], b.first[s + 1], 1024):
            assert torch.isfinite(out[a:min(a + 1024, b.first[s + 1])]).all()
        # a pair is 4 queries
        at = {0, n - 1} | {int(i) // 4 * 4 + d for i in rng.integers(4, max(n - 4, 5), 40) for d in (-1, 0)}
        # where the 152 stretches of one long prompt end, each of the same area
        at |= {int(n * (c / 152) ** 0.5) for c in range(0, 153, 8)}
        for i in sorted(i for i in at if 0 <= i < n):
            want, tol = b.exact(s, i, i + 1)
            got = out[b.first[s] + i:b.first[s] + i + 1].double()
            assert ((got - want).abs() <= tol).all(), (s, i)


@pytest.mark.parametrize("kind", ["q4", "fp8"])
def test_queries_outside_the_batch(pkv, kind):
    """query_start that begins below 0, or goes beyond its last entry: the sequences whose rows would lie outside are
    left out and reported, the others are done."""
    b = Batch([(100, 10), (50, 5), (200, 20), (60, 6)], 2, 2, 128, 16, "bf16", kind, seed=14)
    good, err, starts = b.run(pkv), new_err(), b.starts.clone()
    room = torch.full((b.q.shape[0] + 64, b.H, b.D), 7.0, device=DEV, dtype=b.dtype)
    out = room[32:-32]
    for bad, done in (([-3, 10, 15, 35, 41], [1, 2, 3]), ([0, 10, 15, 35, 30], [0, 1]), ([0, 10, 15, 35, 14], [0]),
                      ([-(1 << 31), 10, 15, 35, 41], [1, 2, 3]), ([0, 10, 15, 35, -1], []), ([0, 10, 15, 35, -(1 << 31)], [])):
        b.starts = torch.tensor(bad, dtype=torch.int32, device=DEV)
        room.fill_(7.0)
        err.zero_()
        b.run(pkv, err=err, out=out, max_new=40)
        assert err.item() == pkv.DEV_ERR_CONTEXT_LEN
        for s in range(4):
            rows = slice(int(starts[s]), int(starts[s + 1]))
            if s in done:
                b.check(out, bad, [s])
            else:
                assert (out[rows] == 7).all(), (bad, s)
        assert (room[:32] == 7).all() and (room[-32:] == 7).all()
    b.starts = starts
    assert torch.equal(b.run(pkv), good)

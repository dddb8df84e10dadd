"""Prefill over q4_0 caches whose values exceed binary16's largest, 65504: a scale of up to 65504 times codes of up to 8,
as rows of bfloat16 give them, and keys of binary16 that were turned before they were quantised. The bounds are those of
any other values."""
import numpy as np
import pytest
import torch

from quant_helpers import DEV, TD, Batch
from rope_helpers import q4_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_204_gb300 as m
    return m


class Wide(Batch):
    """Sequences whose K and V scales are spread up to binary16's largest, in all tokens or in the named ones."""

    def __init__(self, seqs, Hkv, G, D, bs, dtype, seed, k_tokens=None, v_tokens=None, **more):
        super().__init__(seqs, Hkv, G, D, bs, dtype, "q4", seed=seed, **more)
        gen = torch.Generator(device=DEV).manual_seed(seed + 1)
        for pool, rows, tokens in ((self.k, self.k_rows, k_tokens), (self.v, self.v_rows, v_tokens)):
            for s, L in enumerate(self.lens):
                raw = self.random_rows(gen, L, 1.0)
                d = (torch.rand(self.Hkv, L, self.D // 32, device=DEV, generator=gen) * 131008 - 65504).half()
                wide = torch.cat([d.view(torch.uint8), raw[..., self.D // 16:]], -1)
                if tokens is not None:  # the others stay small
                    at = torch.tensor([t for t in tokens if t < L], dtype=torch.long, device=DEV)
                    raw[:, at] = wide[:, at]
                else:
                    raw = wide
                self.put(pool, s, raw)
                rows[s] = self.values(raw, 1.0)


@pytest.mark.parametrize("dtype", TD)
@pytest.mark.parametrize("D", [64, 128])
def test_values_beyond_binary16(pkv, dtype, D):
    """Every K and V row has such values; few and many tokens, cut and whole pairs, ends within 32 tokens."""
    for i, seqs in enumerate([[(300, 40), (1, 1), (129, 2), (33, 33)], [(1000, 257), (2047, 3)], [(5000, 5)]]):
        for Hkv, G, bs in ((1, 2, 16), (2, 5, 8), (1, 8, 32)):
            # small V beside binary16 outputs, which could not hold a wide row by itself
            v_tokens = None if dtype == "bf16" else ()
            b = Wide(seqs, Hkv, G, D, bs, dtype, seed=10 * i + G, q_sigma=2.0 ** -19 if i else 2.0 ** -17, v_tokens=v_tokens)
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            b.check(b.run(pkv, err=err), (i, Hkv, G))
            assert err.item() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_wide_values_beside_binary16_outputs(pkv, D):
    """V rows beyond binary16 that outputs of binary16 can hold all the same: weights of 1/257 and less."""
    b = Wide([(400, 100), (600, 50)], 2, 3, D, 16, "f16", seed=4, q_sigma=1.0, k_tokens=(), v_tokens=(3, 200), scale=0.0)
    assert max(v.abs().max().item() for v in b.v_rows) > 65504
    b.check(b.run(pkv))


@pytest.mark.parametrize("dtype", TD)
@pytest.mark.parametrize("D", [64, 128])
def test_few_wide_tokens(pkv, dtype, D):
    """Some tokens' rows are wide. Queries that do not see them (they are the newest) have outputs as if they were not
    there."""
    b = Wide([(200, 100), (400, 300)], 2, 2, D, 16, dtype, seed=7, k_tokens=(190, 385), v_tokens=(195, 386), q_sigma=0.1)
    out = b.run(pkv)
    for s, (first, seen) in enumerate(((100, 190), (100, 190))):  # queries of positions first .. seen - 1
        want, tol = b.exact(s, 0, seen - first)
        assert want.abs().max() < 16
        got = out[b.first[s]:b.first[s] + seen - first].double()
        assert torch.isfinite(got).all() and ((got - want).abs() <= tol).all()
    # from binary16 outputs only those can be held that see no wide V row, or in a row's average
    for s, (L, n) in enumerate(b.seqs):
        want, tol = b.exact(s, 0, n)
        got = out[b.first[s]:b.first[s] + n].double()
        held = want.abs() + tol < torch.finfo(b.dtype).max
        assert held.any() and torch.isfinite(got[held]).all() and ((got - want).abs()[held] <= tol[held]).all()


def test_turned_binary16_keys(pkv):
    """Keys of up to 65504 a value, turned on their way into the pool: what the pool holds exceeds 65504, and
    prefill attends over it as decode does."""
    H, G, D, T, bs = 8, 2, 128, 96, 16
    gen = torch.Generator(device=DEV).manual_seed(2)
    q = (torch.randn(T, H, D, device=DEV, generator=gen) * 2.0 ** -18).half()
    k = (torch.rand(T, G, D, device=DEV, generator=gen) * 131008 - 65504).half()
    v = torch.randn(T, G, D, device=DEV, generator=gen).half()
    kc, vc = (torch.zeros(T // bs, G, bs, 72, dtype=torch.uint8, device=DEV) for _ in range(2))
    turned = torch.empty_like(q)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.rope_and_cache_q4_0(turned, q, k, v, kc, vc, torch.arange(T, device=DEV),
                            torch.arange(T, dtype=torch.int32, device=DEV), pkv.rope_table(T, D), dev_err=err)
    b = Wide([(T, T)], G, H // G, D, bs, "f16", seed=0)
    b.bt[0, :T // bs] = np.arange(T // bs)
    b.tables = torch.from_numpy(b.bt).to(DEV)
    b.nb, b.k, b.v, b.q = T // bs, kc, vc, turned
    for rows, pool in ((b.k_rows, kc), (b.v_rows, vc)):
        rows[0] = torch.from_numpy(q4_values(pool.transpose(0, 1).reshape(G, T, 72).cpu().numpy())).to(DEV)
    assert b.k_rows[0].abs().max() > 65504
    out = b.run(pkv, err=err)
    b.check(out)
    want = torch.empty_like(out[-1:])
    pkv.paged_attention_decode_q4_0(want, turned[-1:], kc, vc, b.tables, b.context, b.scale, T,
                                    pkv.new_workspace(1, H, D, T), dev_err=err)
    _, tol = b.exact(0, T - 1, T)
    # decode's outputs are one rounding and 32-bit sums away from 64 bits: within the same bound
    assert ((out[-1:].double() - want.double()).abs() <= 2 * tol).all() and err.item() == 0


@pytest.mark.parametrize("dtype", TD)
def test_batches_with_one_wide_sequence(pkv, dtype):
    """Sequences that share CTAs with one that has wide keys, pairs cut by borders among them; a workspace that held
    other calls' results."""
    ws = pkv.new_prefill_workspace(128)
    ws.fill_(0xFF)
    for D in (64, 128):
        for wide in range(4):
            b = Wide([(700, 300), (40, 40), (5000, 64), (300, 2)], 2, 4, D, 16, dtype, seed=wide, k_tokens=(), v_tokens=(),
                     q_sigma=0.5)
            plain = b.run(pkv, ws=ws)
            b.check(plain)
            other = Wide(b.seqs, 2, 4, D, 16, dtype, seed=wide, k_tokens=(17,), v_tokens=(), q_sigma=0.5)
            at = torch.from_numpy(b.bt[wide][1:2]).long().to(DEV)  # the block of token 17
            b.k[at] = other.k[at]
            b.k_rows[wide] = b.k_rows[wide].clone()
            b.k_rows[wide][:, 16:32] = other.k_rows[wide][:, 16:32]
            b.q[b.first[wide]:b.first[wide + 1]] *= 2.0 ** -16
            err = torch.zeros(1, dtype=torch.int32, device=DEV)
            out = b.run(pkv, ws=ws, err=err)
            b.check(out, (D, wide))
            assert err.item() == 0
            assert torch.equal(b.run(pkv, ws=ws), out)


def test_infinite_scales(pkv):
    """A d of infinity gives infinite values: NaN or infinity in outputs of the queries that see the token (as in 64
    bits), and nothing in those that do not."""
    for dtype, D in (("bf16", 128), ("f16", 64)):
        b = Wide([(200, 100)], 1, 2, D, 16, dtype, seed=3, k_tokens=(), v_tokens=())
        for rows, pool in ((b.v_rows, b.v), (b.k_rows, b.k)):
            slot = (int(b.bt[0, 150 // 16]), 0, 150 % 16)
            pool[slot][:D // 16] = torch.tensor([0x00, 0x7C] * (D // 32), dtype=torch.uint8, device=DEV)
            out = b.run(pkv)
            want, tol = b.exact(0, 0, 50)  # positions 100 .. 149
            assert torch.isfinite(out[:50]).all() and ((out[:50].double() - want).abs() <= tol).all()
            assert not torch.isfinite(out[50:]).all(-1).any()


@pytest.mark.parametrize("scale", [0.0, -0.09, 2.0 ** -103])
def test_wide_rows_with_other_scales_and_bad_blocks(pkv, scale):
    """Negative scales, equal weights, bfloat16 queries beyond binary16; a bad block among the wide ones, whose rows
    count as zeros."""
    for dtype, D in (("bf16", 128), ("bf16", 64), ("f16", 128)):
        if dtype == "f16" and scale == 2.0 ** -103:
            continue
        b = Wide([(300, 70), (900, 5), (1, 1)], 2, 3, D, 16, dtype, seed=5, v_tokens=None if dtype == "bf16" else (),
                 q_sigma=2.0 ** (84 if scale == 2.0 ** -103 else -17), scale=scale)
        assert torch.isfinite(b.q).all()
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        b.check(b.run(pkv, err=err), (dtype, D))
        assert err.item() == 0
        b.tables[0, 5] = -2
        b.tables[1, 40] = b.nb
        for s, at in ((0, 5), (1, 40)):
            for rows in (b.k_rows, b.v_rows):
                rows[s] = rows[s].clone()
                rows[s][:, 16 * at:16 * at + 16] = 0
        b.check(b.run(pkv, err=err), (dtype, D, "bad"))
        assert err.item() == pkv.DEV_ERR_BLOCK_ID


def test_wide_rows_in_a_replayed_graph(pkv):
    """A graph whose pool gets wide rows, and loses them, between replays."""
    b = Wide([(700, 300), (3000, 9)], 2, 4, 128, 16, "bf16", seed=6, k_tokens=(), v_tokens=(), q_sigma=2.0 ** -17)
    wide = Wide(b.seqs, 2, 4, 128, 16, "bf16", seed=6, v_tokens=(), q_sigma=2.0 ** -17)
    ws, out, plain = pkv.new_prefill_workspace(128), torch.empty_like(b.q), b.k.clone()
    b.run(pkv, ws=ws, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(pkv, ws=ws, out=out)
    small = b.k_rows
    for pool, rows in ((plain, small), (wide.k, wide.k_rows), (plain, small), (wide.k, wide.k_rows)):
        b.k.copy_(pool)
        b.k_rows = rows
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        b.check(out)

"""The bounded-cache operators without a GPU: refusals of the C entry points
(every call below returns before any device work), of the binding, and the
block manager's side of an eviction."""
import numpy as np
import pytest
import torch

FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_204_gb300 as m
    return m


def caller(fn, **defaults):
    def call(**kw):
        a = dict(defaults)
        assert set(kw) <= set(a), kw
        a.update(kw)
        return fn(*a.values())
    return call





def test_decode_window_refusals(pkv):
    INV, UNS, WS, OK = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_WORKSPACE, pkv.PKV_OK
    rc = caller(pkv.lib.pkv_paged_attention_decode_window, out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE,
                scale=0.1, window=100, sinks=4, H=8, Hkv=2, D=128, bs=16, B=4, MB=8, NB=100, mcl=128, dtype=1,
                ws=None, ws_bytes=0, err=None, stream=None)
    assert rc(B=0) == OK
    for bad in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(B=-1), dict(H=9), dict(Hkv=0), dict(mcl=129),
                dict(mcl=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(q=FAKE + 8),
                dict(k=FAKE + 4), dict(v=None), dict(bt=FAKE + 2), dict(cl=None), dict(err=FAKE + 1), dict(NB=0)):
        assert rc(**bad) == INV, bad
    for bad in (dict(D=96), dict(D=256), dict(bs=64), dict(bs=4, mcl=32), dict(dtype=3), dict(dtype=4), dict(dtype=9),
                dict(B=65536), dict(MB=1 << 27, bs=16, mcl=16)):
        assert rc(**bad) == UNS, bad
    need = pkv.decode_window_workspace_bytes(4, 8, 2, 128)
    assert rc() == WS and rc(ws=FAKE, ws_bytes=need - 1) == WS and rc(ws=FAKE + 4, ws_bytes=need) == INV


def test_decode_scores_refusals(pkv):
    INV, UNS, WS, OK = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_WORKSPACE, pkv.PKV_OK
    rc = caller(pkv.lib.pkv_paged_attention_decode_scores, out=FAKE, so=FAKE << 8, si=FAKE << 8, stride=128, q=FAKE,
                k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, scale=0.1, H=8, Hkv=2, D=128, bs=16, B=4, MB=8, NB=100, mcl=128,
                dtype=1, ws=None, ws_bytes=0, err=None, stream=None)
    assert rc(B=0) == OK
    size = 4 * 2 * 128 * 4  # bytes of the score rows
    for bad in (dict(stride=127), dict(so=None), dict(so=(FAKE << 8) + 2), dict(si=(FAKE << 8) + 4),
                dict(si=(FAKE << 8) - size + 4), dict(si=(FAKE << 8) + size - 4), dict(mcl=129), dict(H=7)):
        assert rc(**bad) == INV, bad
    assert rc(dtype=3) == UNS and rc(D=80) == UNS and rc(Hkv=65536, H=65536) == UNS
    need = pkv.decode_scores_workspace_bytes(4, 8, 2, 128, 128)
    for scores in (FAKE << 8, None, (FAKE << 8) + size, (FAKE << 8) - size):
        assert rc(si=scores) == WS and rc(si=scores, ws=FAKE, ws_bytes=need - 1) == WS
    assert rc(ws=FAKE + 8, ws_bytes=need) == INV


def test_prefill_window_refusals(pkv):
    INV, UNS, OK = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_OK
    rc = caller(pkv.lib.pkv_paged_attention_prefill_window, out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE,
                qs=FAKE, scale=0.1, window=100, sinks=4, H=8, Hkv=8, D=128, bs=16, B=4, MB=8, NB=100, mql=64, dtype=2,
                err=None, stream=None)
    assert rc(B=0) == OK and rc(mql=0) == OK
    for bad in (dict(window=0), dict(sinks=-1), dict(mql=-1), dict(qs=None), dict(qs=FAKE + 2), dict(H=9),
                dict(q=FAKE + 8), dict(scale=float("nan"))):
        assert rc(**bad) == INV, bad
    for bad in (dict(dtype=0), dict(dtype=3), dict(D=96), dict(bs=64), dict(MB=1 << 28)):
        assert rc(**bad) == UNS, bad


def test_evict_refusals(pkv):
    INV, UNS, OK = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_OK
    S = FAKE << 8
    rc = caller(pkv.lib.pkv_evict_tokens, k=FAKE, v=FAKE, si=S, stride=128, so=S, out_stride=128, bt=FAKE, dst=FAKE,
                cl=FAKE, nl=FAKE, kept=FAKE, budget=64, sinks=4, recent=16, Hkv=2, D=128, bs=16, B=4, MB=8, NB=100,
                mcl=128, dtype=1, err=None, stream=None)
    assert rc(B=0) == OK
    size = 4 * 2 * 128 * 4
    used = size - 64 * 4  # the last output row ends with its budget
    for bad in (dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=50, recent=15),
                dict(sinks=(1 << 31) - 1, recent=(1 << 31) - 1), dict(stride=127), dict(out_stride=63), dict(mcl=129),
                dict(B=-1), dict(Hkv=0), dict(k=None), dict(v=FAKE + 8), dict(si=None), dict(so=None), dict(bt=None),
                dict(dst=FAKE + 2), dict(cl=None), dict(nl=None), dict(kept=None), dict(err=FAKE + 2),
                dict(out_stride=64), dict(so=S + 4), dict(so=S + size - 4), dict(so=S - used + 4)):
        assert rc(**bad) == INV, bad
    for bad in (dict(D=96), dict(bs=12, mcl=96), dict(dtype=5), dict(B=65536), dict(Hkv=65536), dict(MB=1 << 27)):
        assert rc(**bad) == UNS, bad


def test_workspace_sizes(pkv):
    a = lambda x: -(-x // 256) * 256
    base = a(4 * 8 * 4) + a(32768 * 8) + 32768 * 128 * 4
    assert pkv.decode_window_workspace_bytes(4, 8, 2, 128) == base
    assert pkv.decode_scores_workspace_bytes(4, 8, 2, 128, 1001) == base + a(4 * 8 * 8) + 4 * 8 * 1008 * 4
    assert pkv.decode_scores_workspace_bytes(65535, 128, 8, 128, 1 << 20) > 1 << 42  # no 32-bit overflow
    for args in ((0, 8, 2, 128), (4, 9, 2, 128), (4, 8, 0, 128), (4, -8, -2, 128), (4, 8, 2, 0)):
        assert pkv.decode_window_workspace_bytes(*args) == 0
        assert pkv.decode_scores_workspace_bytes(*args, 10) == 0
    assert pkv.decode_scores_workspace_bytes(4, 8, 2, 128, -1) == 0


def test_binding_wants_cuda_tensors(pkv):
    pool = torch.zeros(4, 2, 16, 64)
    t, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 2, 64)
    sc = torch.zeros(1, 2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_decode_window(q, q, pool, pool, t, n, 1.0, 4, 0, 32, torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_prefill_window(q, q, pool, pool, t, n, t, 1.0, 4, 0, 1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_decode_scores(q, sc, q, pool, pool, t, n, 1.0, 32, torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA"):
        pkv.evict_tokens(pool, pool, sc, sc, t, t, n, n, torch.zeros(1, 2, 8, dtype=torch.int32), 0, 0, 32)


# ---- the block manager's side of an eviction -------------------------------------


@pytest.fixture
def BM(pkv):
    import paged_kv_cache_204_gb300.block_manager as m
    return m


def test_shrink_exclusive_sequences(BM):
    with BM.BlockManager(40, 16, seed=3) as bm:
        a, b, c = bm.add_seq(), bm.add_seq(), bm.add_seq()
        for s, n in ((a, 100), (b, 33), (c, 16)):
            bm.append(s, n)
        before, after, lens = bm.shrink_batch([a, b, c], [33, 33, 0], 8)
        assert lens.tolist() == [100, 33, 16]
        assert after[0, :3].tolist() == before[0, :3].tolist() and (after[0, 3:] == -1).all()
        assert after[1].tolist() == before[1].tolist() and (after[2] == -1).all()
        assert bm.seq_info(a) == (33, 3) and bm.seq_info(c) == (0, 0)
        st = bm.stats()
        assert st["used_blocks"] == 6 and st["free_blocks"] == 34 and st["filled_slots"] == 66
        slots, cow = bm.append(a, 1)  # goes on where the cut left off
        assert cow is None and slots[0] == after[0, 2] * 16 + 1
        assert bm.append(c, 1)[0][0] % 16 == 0


def test_shrink_shared_blocks(BM):
    with BM.BlockManager(64, 8, seed=5) as bm:
        a = bm.add_seq()
        bm.append(a, 40)
        b = bm.fork(a)
        d = bm.fork(a)
        bm.append(b, 24)
        held = set(bm.export([a, b, d], 8)[0].ravel().tolist()) - {-1}
        before, after, _ = bm.shrink_batch([a, b], [20, 50], 8)
        new = set(after.ravel().tolist()) - {-1}
        # a: three blocks, all shared; b: five shared, then two of its own
        assert not set(after[0, :3]) & held and (after[0, 3:] == -1).all()
        assert not set(after[1, :5]) & held and after[1, 5:7].tolist() == before[1, 5:7].tolist()
        assert len(new) == 3 + 7
        assert bm.export([d], 8)[0][0].tolist() == before[0].tolist()  # the third holder keeps its table
        st = bm.stats()
        assert st["used_blocks"] == 5 + 3 + 7 and st["shared_blocks"] == 0


def test_shrink_no_fresh_block_was_held_before(BM):
    """Two sequences share everything and are cut together: neither may get a
    block whose rows the other still has to read, even though both let go."""
    with BM.BlockManager(12, 8) as bm:
        a = bm.add_seq()
        bm.append(a, 32)
        b = bm.fork(a)
        before, after, _ = bm.shrink_batch([a, b], [31, 31], 4)
        assert not set(after.ravel()) & set(before.ravel()) and len(set(after.ravel())) == 8
        assert bm.stats()["free_blocks"] == 4


def test_shrink_refusals_change_nothing(BM):
    with BM.BlockManager(10, 8) as bm:
        a = bm.add_seq()
        bm.append(a, 48)
        b = bm.fork(a)
        state = lambda: (bm.stats(), bm.export([a, b], 8)[0].tolist())
        was = state()
        with pytest.raises(BM.OutOfBlocks):  # needs 10 fresh blocks, 4 are free
            bm.shrink_batch([a, b], [40, 40], 8)
        for seqs, lens in (([a, a], [8, 8]), ([a, 7], [8, 8]), ([a], [49]), ([a], [-1]), ([-1], [0])):
            s, m = BM._i32(seqs), BM._i32(lens)
            assert BM.lib.pkv_bm_shrink_batch(bm._h, s.ctypes.data, m.ctypes.data, len(seqs)) == 1
        assert BM.lib.pkv_bm_shrink_batch(None, None, None, 0) == 1
        assert BM.lib.pkv_bm_shrink_batch(bm._h, None, None, 1) == 1
        assert BM.lib.pkv_bm_shrink_batch(bm._h, None, None, 0) == 0
        assert state() == was
        bm.shrink_batch([a, b], [8, 8], 8)  # and the manager still works
        assert bm.stats()["used_blocks"] == 2


def test_shrink_random_against_a_label_model(BM):
    """Random appends, forks, cuts and ends: lengths, table sizes and the
    number of distinct live blocks follow from the tables alone."""
    rng = np.random.default_rng(9)
    with BM.BlockManager(400, 8, seed=2) as bm:
        live = [bm.add_seq()]
        length = {live[0]: 0}
        for _ in range(400):
            op = rng.integers(4)
            s = int(rng.choice(live))
            if op == 0:
                n = int(rng.integers(1, 30))
                try:
                    bm.append(s, n)
                    length[s] += n
                except BM.OutOfBlocks:
                    pass
            elif op == 1 and len(live) < 12:
                c = bm.fork(s)
                live.append(c)
                length[c] = length[s]
            elif op == 2:
                some = [int(x) for x in rng.permutation(live)[:rng.integers(1, len(live) + 1)]]
                cut = [int(rng.integers(0, length[x] + 1)) for x in some]
                refs = {}
                tables = bm.export(live, 400)[0]
                for row in tables:
                    for b in row[row >= 0]:
                        refs[b] = refs.get(b, 0) + 1
                try:
                    before, after, lens = bm.shrink_batch(some, cut, 400)
                except BM.OutOfBlocks:
                    continue
                for i, x in enumerate(some):
                    assert lens[i] == length[x]
                    nb = -(-cut[i] // 8)
                    assert (after[i, :nb] >= 0).all() and (after[i, nb:] == -1).all()
                    for j in range(nb):
                        if cut[i] == lens[i] or refs[before[i, j]] == 1:
                            assert after[i, j] == before[i, j]
                        else:
                            assert after[i, j] not in refs
                    length[x] = cut[i]
            elif op == 3 and len(live) > 1:
                bm.free_seq(s)
                live.remove(s)
                del length[s]
            tables = bm.export(live, 400)[0]
            used = set(tables.ravel().tolist()) - {-1}
            st = bm.stats()
            assert st["used_blocks"] == len(used) and st["free_blocks"] == 400 - len(used)
            assert st["logical_tokens"] == sum(length.values())

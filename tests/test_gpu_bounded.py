"""The bounded-cache operators on the GPU against plain 64-bit attention and
plain selection: every type, head layout and block size, lengths and windows
at tile and block borders, poison in every place that must not be read, the
device error word, graphs, streams, and a session that uses them together."""
import numpy as np
import pytest
import torch

from bounded_helpers import DEV, TD, Cache, attend, check, eps_p, eps_prefill, half_step, seen_by

pytestmark = pytest.mark.gpu

LENS = (0, 1, 2, 7, 8, 15, 16, 17, 31, 33, 64, 127, 129, 255, 257, 512, 1000, 2047)
COMBOS = [  # dtype, head_dim, block_size, kv heads, group
    ("f32", 64, 16, 2, 1), ("f32", 128, 8, 2, 2), ("f32", 128, 32, 1, 4), ("f32", 64, 8, 1, 7),
    ("f16", 64, 8, 2, 1), ("f16", 128, 16, 2, 3), ("f16", 64, 32, 1, 8), ("f16", 128, 32, 3, 4),
    ("bf16", 128, 16, 2, 1), ("bf16", 64, 16, 2, 4), ("bf16", 128, 8, 1, 5), ("bf16", 128, 16, 1, 12),
    ("bf16", 64, 8, 3, 6), ("bf16", 128, 32, 1, 19),
]
ids = lambda c: "_".join(map(str, c))


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_204_gb300 as m
    return m


def new_err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def run_window(pkv, c, window, sinks, ws=None, err=None, max_len=None, out=None, stream=None):
    ws = pkv.new_window_workspace(len(c.lens), c.H, c.Hkv, c.D) if ws is None else ws
    out = torch.full_like(c.q, float("nan")) if out is None else out
    pkv.paged_attention_decode_window(out, c.q, c.k, c.v, c.tables, c.context, c.scale, window, sinks,
                                      c.max_len if max_len is None else max_len, ws, dev_err=err, stream=stream)
    return out


def check_window(c, out, window, sinks, what):
    for s, L in enumerate(c.lens):
        if L == 0:
            assert (out[s] == 0).all(), what
            continue
        want, _, bound, _ = attend(c.q[s], c.rows_k[s], c.rows_v[s], seen_by(L, L - 1, window, sinks), c.scale,
                                   eps_p(c.dtype))
        check(out[s], want, bound, f"{what} L={L} window={window} sinks={sinks}")


# ---- decode over sinks and a window ---------------------------------------------------


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (16, 4), (100, 17), (256, 64), (5000, 3), (33, 5000)])
@pytest.mark.parametrize("combo", COMBOS, ids=ids)
def test_decode_window(pkv, combo, window, sinks):
    dtype, D, bs, Hkv, G = combo
    c = Cache(LENS, Hkv, G, D, bs, dtype, seed=window + sinks)
    c.poison_unseen(lambda s: seen_by(c.lens[s], c.lens[s] - 1, window, sinks))
    err = new_err()
    ws = pkv.new_window_workspace(len(c.lens), c.H, c.Hkv, c.D)
    out = run_window(pkv, c, window, sinks, ws, err)
    assert int(err.item()) == 0
    assert (ws[:4 * len(c.lens) * c.H] == 0).all()
    check_window(c, out, window, sinks, ids(combo))


@pytest.mark.parametrize("dtype,G", [("f16", 4), ("bf16", 8), ("f32", 2)])
@pytest.mark.parametrize("lens,window,sinks", [((30011,), 8200, 4), ((30011, 3, 0, 9000, 517), 40000, 0),
                                               ((4097,) * 3, 4000, 100)])
def test_decode_window_split(pkv, dtype, G, lens, window, sinks):
    """Few long segments: each is cut into pieces that are joined; the same
    bits on every call, the counters back at zero."""
    c = Cache(lens, 2, G, 128, 16, dtype, seed=5)
    c.poison_unseen(lambda s: seen_by(c.lens[s], c.lens[s] - 1, window, sinks))
    err = new_err()
    ws = pkv.new_window_workspace(len(lens), c.H, c.Hkv, c.D)
    out = run_window(pkv, c, window, sinks, ws, err)
    check_window(c, out, window, sinks, "split")
    for _ in range(3):
        assert torch.equal(run_window(pkv, c, window, sinks, ws, err), out)
    assert int(err.item()) == 0 and (ws[:4 * len(lens) * c.H] == 0).all()


def test_decode_window_equals_plain_decode_when_all_is_seen(pkv):
    c = Cache((700, 33, 1500), 2, 4, 128, 16, "bf16")
    out = run_window(pkv, c, c.max_len, 0)
    ref = torch.empty_like(out)
    pkv.paged_attention_decode(ref, c.q, c.k, c.v, c.tables, c.context, c.scale, c.max_len,
                               workspace=pkv.new_workspace(3, c.H, c.D, c.max_len))
    assert (out.float() - ref.float()).abs().max() <= 2 * half_step(c.dtype) * ref.float().abs().max()


def test_decode_window_larger_bound_and_big_numbers(pkv):
    """max_context_len may be any bound; windows and sinks up to the int limit."""
    c = Cache((100, 17, 2000), 2, 2, 64, 16, "f16")
    c.bt = np.concatenate([c.bt, np.full((3, 5000), -1, np.int32)], 1)
    c.tables = torch.from_numpy(c.bt).to(DEV)
    for window, sinks in (((1 << 31) - 1, (1 << 31) - 1), (50, (1 << 31) - 1), ((1 << 31) - 1, 0)):
        out = run_window(pkv, c, window, sinks, max_len=60000)
        check_window(c, out, window, sinks, "bound")


def test_decode_window_logits_of_infinity(pkv):
    """Logits of -inf (infinite keys) in whole tiles: weight zero, never a NaN."""
    c = Cache((200, 40), 1, 2, 64, 16, "f16")
    c.q[:, :, 0] = 1.0
    for s in range(2):
        c.rows_k[s][:, : 35, 0] = float("-inf")
        c.put(c.k, s, torch.arange(c.lens[s]), c.rows_k[s])
    out = run_window(pkv, c, 5000, 0)
    for s, L in enumerate(c.lens):
        keep = torch.arange(L) >= 35
        want, _, bound, _ = attend(c.q[s], c.rows_k[s], c.rows_v[s], keep, c.scale, eps_p(c.dtype))
        check(out[s], want, bound, "infinite keys")


def test_decode_window_device_errors(pkv):
    c = Cache((300, 50), 2, 2, 128, 16, "bf16")
    good = run_window(pkv, c, 100, 4)
    err = new_err()
    c.tables[0, 300 // 16] = c.nb          # a visible block: reported, the other sequence's result stands
    out = run_window(pkv, c, 100, 4, err=err)
    assert int(err.item()) == pkv.DEV_ERR_BLOCK_ID and torch.equal(out[1], good[1])
    err.zero_()
    c.tables[0, 5] = -7                    # not visible: not looked at
    c.tables[0, 300 // 16] = int(c.bt[0, 300 // 16])
    assert torch.equal(run_window(pkv, c, 100, 4, err=err), good) and int(err.item()) == 0
    c.context[0] = -3
    out = run_window(pkv, c, 100, 4, err=err)
    assert int(err.item()) == pkv.DEV_ERR_CONTEXT_LEN and (out[0] == 0).all() and torch.equal(out[1], good[1])
    err.zero_()
    c.context[0] = 300
    run_window(pkv, c, 100, 4, err=err, max_len=299)
    assert int(err.item()) == pkv.DEV_ERR_CONTEXT_LEN


# ---- decode with scores ------------------------------------------------------------------


def run_scores(pkv, c, scores, scores_out, ws=None, err=None, max_len=None):
    max_len = c.max_len if max_len is None else max_len
    ws = pkv.new_scores_workspace(len(c.lens), c.H, c.Hkv, c.D, max_len) if ws is None else ws
    out = torch.full_like(c.q, float("nan"))
    pkv.paged_attention_decode_scores(out, scores_out, c.q, c.k, c.v, c.tables, c.context, c.scale, max_len, ws,
                                      scores=scores, dev_err=err)
    return out


def check_scores(c, out, old, new, what):
    """old: the scores before (None: none), new: after; entries behind a
    sequence keep the bits they had (NaN here)."""
    for s, L in enumerate(c.lens):
        assert torch.isnan(new[s, :, L:]).all(), what
        if L == 0:
            assert (out[s] == 0).all(), what
            continue
        want, w, bound, rel = attend(c.q[s], c.rows_k[s], c.rows_v[s], torch.ones(L, dtype=torch.bool), c.scale,
                                     eps_p(c.dtype))
        check(out[s], want, bound, f"{what} L={L}")
        part = w.reshape(c.Hkv, c.G, L)
        total = part.sum(1)
        tol = (part * (rel.reshape(c.Hkv, c.G, 1) + (c.G + 2) * 2.0 ** -23)).sum(1) + 2.0 ** -126
        if old is not None:
            total[:, :L - 1] += old[s, :, :L - 1].double()
        check(new[s, :, :L], total, tol, f"{what} scores L={L}")


@pytest.mark.parametrize("combo", COMBOS, ids=ids)
def test_decode_scores(pkv, combo):
    dtype, D, bs, Hkv, G = combo
    c = Cache(LENS, Hkv, G, D, bs, dtype, seed=1)
    n = c.max_len + 5
    err = new_err()
    nan = lambda: torch.full((len(LENS), Hkv, n), float("nan"), device=DEV)
    new = nan()
    out = run_scores(pkv, c, None, new, err=err)
    check_scores(c, out, None, new, "first")
    old = nan()
    for s, L in enumerate(LENS):
        if L:
            old[s, :, :L - 1] = torch.rand(Hkv, L - 1, device=DEV)  # the newest token's place holds NaN
    new = nan()
    out2 = run_scores(pkv, c, old, new, err=err)
    check_scores(c, out2, old, new, "apart")
    assert torch.equal(out, out2)
    both = old.clone()
    run_scores(pkv, c, both, both, err=err)
    assert torch.equal(torch.nan_to_num(both, -1.0), torch.nan_to_num(new, -1.0))
    assert int(err.item()) == 0


@pytest.mark.parametrize("n,off", [(1104, 0), (1104, 1), (1101, 0), (1101, 2)])
@pytest.mark.parametrize("how", ["apart", "in_place"])
def test_decode_scores_alignment(pkv, n, off, how):
    """Score rows on and off 16 bytes, lengths that end anywhere in 4 tokens."""
    c = Cache((1101, 1100, 1099, 1098, 1, 2, 0, 5), 2, 3, 64, 8, "bf16", seed=n)
    rows = lambda: torch.full((8 * 2 * n + off,), float("nan"), device=DEV)[off:].view(8, 2, n)
    old, new = rows(), rows()
    for s, L in enumerate(c.lens):
        old[s, :, :max(L - 1, 0)] = torch.rand(2, max(L - 1, 0), device=DEV)
    before = old.clone()
    if how == "in_place":
        new = old
    out = run_scores(pkv, c, old, new)
    check_scores(c, out, before, new, how)


@pytest.mark.parametrize("dtype,G", [("f16", 4), ("bf16", 7), ("f32", 1)])
def test_decode_scores_long(pkv, dtype, G):
    c = Cache((20011, 0, 5000), 2, G, 128, 16, dtype, seed=8)
    new = torch.full((3, 2, 20020), float("nan"), device=DEV)
    ws = pkv.new_scores_workspace(3, c.H, c.Hkv, c.D, 20020)
    out = run_scores(pkv, c, None, new, ws, max_len=20020)
    check_scores(c, out, None, new, "long")
    again = torch.full_like(new, float("nan"))
    assert torch.equal(run_scores(pkv, c, None, again, ws, max_len=20020), out)
    assert torch.equal(torch.nan_to_num(again, -1.0), torch.nan_to_num(new, -1.0))
    total = torch.nan_to_num(new, 0.0).double().sum(2)
    assert ((total[[0, 2]] - G).abs() <= 1e-3).all()  # each head's weights sum to 1


# ---- eviction ---------------------------------------------------------------------------


def kept_of(row, L, budget, sinks, recent):
    if L <= budget:
        return list(range(L))
    key = [(-np.inf, 0) if np.isnan(x) else (x, 1) for x in row[:L]]  # NaN below every number
    middle = sorted(range(sinks, L - recent), key=lambda t: (-key[t][0], -key[t][1], t))
    return list(range(sinks)) + sorted(middle[:budget - sinks - recent]) + list(range(L - recent, L))


def special_scores(rng, shape):
    """Random scores with many ties, zeros of both signs, infinities and NaN."""
    x = rng.choice(np.array([0.0, -0.0, 1.0, 1.0000001, 2.5, -3.0, np.inf, -np.inf, np.nan, 1e-42, -1e-42], np.float32),
                   shape)
    pick = rng.random(shape) < 0.5
    return np.where(pick, rng.standard_normal(shape).astype(np.float32), x).astype(np.float32)


POOLS = {"f32": (torch.float32, 1, 1), "f16": (torch.float16, 1, 1), "bf16": (torch.bfloat16, 1, 1),
         "fp8": (torch.uint8, 1, 1), "q4": (torch.uint8, 9, 16)}


@pytest.mark.parametrize("how", ["in_place", "fresh", "mixed"])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (64, 4, 16), (100, 0, 100), (333, 50, 33),
                                                 (700, 0, 0), (3000, 5, 7)])
@pytest.mark.parametrize("pool,D,bs,Hkv", [("f32", 64, 8, 2), ("f16", 128, 16, 3), ("bf16", 64, 32, 1),
                                           ("fp8", 64, 16, 2), ("fp8", 128, 8, 2), ("q4", 64, 16, 2),
                                           ("q4", 128, 32, 2)])
def test_evict(pkv, pool, D, bs, Hkv, budget, sinks, recent, how):
    rng = np.random.default_rng([D, bs, budget, len(how)])
    lens = [0, 1, 63, 64, 65, 100, 101, 334, 699, 1500, 2311]
    B, width = len(lens), 2311 // bs + 2
    counts = [-(-L // bs) for L in lens]
    nb = 2 * sum(counts) + 2
    perm = rng.permutation(nb).astype(np.int32)
    src = np.full((B, width), -1, np.int32)
    dst = np.full((B, width), -1, np.int32)
    at = 0
    for s, c in enumerate(counts):
        src[s, :c] = perm[at:at + c]
        at += c
    for s, L in enumerate(lens):
        n = -(-min(L, budget) // bs)
        for j in range(n):
            if how == "in_place" or (how == "mixed" and rng.random() < 0.5):
                dst[s, j] = src[s, j]
            else:
                dst[s, j] = perm[at]
                at += 1
    dtype, num, den = POOLS[pool]
    row = D * num // den
    gen = torch.Generator(device=DEV).manual_seed(int(budget))
    raw = torch.empty(nb, Hkv, bs, row, dtype=dtype).element_size()
    k0 = torch.randint(0, 256, (nb, Hkv, bs, row * raw), device=DEV, generator=gen, dtype=torch.uint8)
    v0 = torch.randint(0, 256, (nb, Hkv, bs, row * raw), device=DEV, generator=gen, dtype=torch.uint8)
    k, v = k0.clone(), v0.clone()
    scores0 = special_scores(rng, (B, Hkv, 2315))
    scores = torch.from_numpy(scores0).to(DEV)
    inplace_scores = how != "fresh"
    out = scores if inplace_scores else torch.full((B, Hkv, budget + 3), 77.0, device=DEV)
    kept = torch.full((B, Hkv, budget), -9, dtype=torch.int32, device=DEV)
    context = torch.tensor(lens, dtype=torch.int32, device=DEV)
    new = context if how == "mixed" else torch.full((B,), -1, dtype=torch.int32, device=DEV)
    tables = torch.from_numpy(src).to(DEV)
    err = new_err()
    pkv.evict_tokens(k.view(dtype), v.view(dtype), scores, out, tables,
                     tables if how == "in_place" else torch.from_numpy(dst).to(DEV), context, new, kept, sinks, recent,
                     2311, head_dim=D, dev_err=err)
    assert int(err.item()) == 0
    assert new.tolist() == [min(L, budget) for L in lens]
    want_k, want_v = k0.cpu().numpy().copy(), v0.cpu().numpy().copy()
    k0n, v0n = k0.cpu().numpy(), v0.cpu().numpy()
    want_s = scores0.copy() if inplace_scores else np.full((B, Hkv, budget + 3), 77.0, np.float32)
    want_kept = np.full((B, Hkv, budget), -9, np.int32)
    for s, L in enumerate(lens):
        for h in range(Hkv):
            keep = np.array(kept_of(scores0[s, h], L, budget, sinks, recent), np.int64)
            n = len(keep)
            assert n == min(L, budget)
            i = np.arange(n)
            a, b = src[s][keep // bs], dst[s][i // bs]
            want_k[b, h, i % bs] = k0n[a, h, keep % bs]
            want_v[b, h, i % bs] = v0n[a, h, keep % bs]
            want_s[s, h, :n] = scores0[s, h, keep]
            want_kept[s, h, :n] = keep
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(out.cpu().numpy().view(np.int32), want_s.view(np.int32))
    assert np.array_equal(k.cpu().numpy(), want_k) and np.array_equal(v.cpu().numpy(), want_v)


@pytest.mark.parametrize("values", ["equal", "rising", "falling", "near", "skewed"])
def test_evict_long_rows(pkv, values):
    """Long rows: all ties, sorted rows, keys that differ in their last bits only."""
    L, budget, bs, Hkv = 40009, 9001, 16, 2
    nb = -(-L // bs)
    rng = np.random.default_rng(3)
    base = {"equal": np.full(L, 0.25), "rising": np.arange(L) * 1e-3, "falling": -np.arange(L) * 1e-3,
            "near": 1.0 + rng.integers(0, 3, L) * 2.0 ** -23, "skewed": rng.pareto(0.7, L)}[values]
    sc = np.stack([base, base[::-1]]).astype(np.float32)[None]
    k = torch.randn(nb, Hkv, bs, 64, device=DEV).half()
    v = torch.randn(nb, Hkv, bs, 64, device=DEV).half()
    k0 = k.clone()
    tables = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    scores = torch.from_numpy(sc).to(DEV)
    kept = torch.zeros(1, Hkv, budget, dtype=torch.int32, device=DEV)
    context = torch.tensor([L], dtype=torch.int32, device=DEV)
    pkv.evict_tokens(k, v, scores, scores, tables, tables, context, context, kept, 4, 1000, L)
    assert context.tolist() == [budget]
    for h in range(Hkv):
        keep = kept_of(sc[0, h], L, budget, 4, 1000)
        assert kept[0, h].tolist() == keep
        flat = lambda p: p[:, h].reshape(-1, 64)
        assert torch.equal(flat(k)[:budget], flat(k0)[torch.tensor(keep, device=DEV)])


@pytest.mark.parametrize("L", [8191, 8192, 8193, 32767, 32768, 32769])
@pytest.mark.parametrize("recent", [0, 200])
def test_evict_row_sizes(pkv, L, recent):
    """Rows at the bounds of the selection's variants, at every alignment; with `recent`
    the budget is spent, and no score decides."""
    budget, Hkv = 204, 4
    nb = -(-L // 32)
    sc = torch.randn(1, Hkv, L + 1, device=DEV)              # a row begins 4 or more bytes off 16
    want = [kept_of(sc[0, h].cpu().numpy(), L, budget, 4, recent) for h in range(Hkv)]
    k = torch.randn(nb, Hkv, 32, 64, device=DEV).half()
    v, k0 = k.clone(), k.clone()
    tables = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    kept = torch.zeros(1, Hkv, budget, dtype=torch.int32, device=DEV)
    out = torch.zeros(1, Hkv, budget, device=DEV)
    new = torch.zeros(1, dtype=torch.int32, device=DEV)
    pkv.evict_tokens(k, v, sc, out, tables, tables, torch.tensor([L], dtype=torch.int32, device=DEV), new, kept, 4,
                     recent, L)
    for h in range(Hkv):
        assert kept[0, h].tolist() == want[h]
        at = torch.tensor(want[h], device=DEV)
        assert torch.equal(out[0, h], sc[0, h, at])
        assert torch.equal(k[:, h].reshape(-1, 64)[:budget], k0[:, h].reshape(-1, 64)[at])


def test_evict_device_errors(pkv):
    c = Cache((300, 50), 2, 1, 64, 16, "f16")
    scores = torch.rand(2, 2, 300, device=DEV)
    call = lambda err, tables, context: pkv.evict_tokens(
        c.k, c.v, scores, torch.zeros(2, 2, 100, device=DEV), tables, c.tables, context, torch.zeros_like(context),
        torch.zeros(2, 2, 100, dtype=torch.int32, device=DEV), 4, 20, 300, dev_err=err)
    err = new_err()
    bad = c.tables.clone()
    bad[0, 0] = c.nb                                    # the sinks' block: its rows are not moved
    before = c.k[c.bt[0, 0]].clone()
    call(err, bad, c.context)
    assert int(err.item()) == pkv.DEV_ERR_BLOCK_ID
    assert torch.equal(c.k[c.bt[0, 0]][:, :4], before[:, :4])
    err.zero_()
    call(err, c.tables, torch.tensor([301, -1], dtype=torch.int32, device=DEV))
    assert int(err.item()) == pkv.DEV_ERR_CONTEXT_LEN


# ---- prefill over sinks and a window --------------------------------------------------------


def run_prefill(pkv, c, new, window, sinks, q, err=None, stream=None):
    start = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    out = torch.full_like(q, float("nan"))
    pkv.paged_attention_prefill_window(out, q, c.k, c.v, c.tables, c.context, start, c.scale, window, sinks,
                                       max(new), dev_err=err, stream=stream)
    return out


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 4), (63, 1), (64, 0), (100, 70), (300, 64), (129, 200),
                                          (5000, 0), (40, 1 << 30)])
@pytest.mark.parametrize("combo", [("f16", 64, 8, 2, 1), ("bf16", 128, 16, 1, 4), ("f16", 128, 32, 1, 3),
                                   ("bf16", 64, 16, 2, 2)], ids=ids)
def test_prefill_window(pkv, combo, window, sinks):
    dtype, D, bs, Hkv, G = combo
    lens = [5, 700, 128, 300, 1, 0, 513]
    new = [5, 130, 128, 1, 1, 0, 300]
    c = Cache(lens, Hkv, G, D, bs, dtype, seed=window)
    q = torch.randn(sum(new), c.H, D, device=DEV).to(c.dtype)

    def seen(s):  # by any query of the call
        any_ = torch.zeros(lens[s], dtype=torch.bool)
        for P in range(lens[s] - new[s], lens[s]):
            any_ |= seen_by(lens[s], P, window, sinks)
        return any_
    c.poison_unseen(seen)
    err = new_err()
    out = run_prefill(pkv, c, new, window, sinks, q, err)
    assert int(err.item()) == 0
    at = 0
    for s, L in enumerate(lens):
        for i in range(new[s]):
            if i % 7 in (0, 3) or i in (127, 128, new[s] - 1):
                want, _, bound, _ = attend(q[at + i], c.rows_k[s], c.rows_v[s],
                                           seen_by(L, L - new[s] + i, window, sinks), c.scale,
                                           eps_prefill(c.dtype))
                check(out[at + i], want, bound, f"L={L} n={new[s]} i={i}")
        at += new[s]


@pytest.mark.parametrize("scale", [-0.11, 0.0, 3.0])
def test_scales_of_either_sign(pkv, scale):
    """A negative scale turns the order of the scores, zero makes them equal."""
    c = Cache((300, 40), 1, 2, 64, 16, "f16", seed=9)
    c.scale = scale
    new = [140, 40]
    q = torch.randn(sum(new), c.H, 64, device=DEV).half()
    out = run_prefill(pkv, c, new, 130, 4, q)
    dec = run_window(pkv, c, 130, 4)
    for s, L in enumerate(c.lens):
        for i in (0, 1, new[s] - 1):
            want, _, bound, _ = attend(q[140 * s + i], c.rows_k[s], c.rows_v[s],
                                       seen_by(L, L - new[s] + i, 130, 4), scale, eps_prefill(c.dtype))
            check(out[140 * s + i], want, bound, f"prefill {s} {i}")
    check_window(c, dec, 130, 4, "decode")


@pytest.mark.parametrize("D,Hkv", [(64, 1), (128, 160)])  # a cluster shares a pair of query tiles, or none does
def test_prefill_window_logits_of_infinity(pkv, D, Hkv):
    """Logits of -inf have weight zero; where a query sees nothing else, 0 / 0."""
    c = Cache((200,), Hkv, 1, D, 16, "f16")
    c.rows_k[0][:, :35, 0] = float("-inf")
    c.put(c.k, 0, torch.arange(200), c.rows_k[0])
    q = torch.randn(200, c.H, D, device=DEV).half()
    q[:, :, 0] = 1.0
    out = run_prefill(pkv, c, [200], 20, 0, q)
    assert torch.isnan(out[:35]).all()
    for i in range(35, 200, 7):
        seen = seen_by(200, i, 20, 0) & (torch.arange(200) >= 35)
        want, _, bound, _ = attend(q[i], c.rows_k[0], c.rows_v[0], seen, c.scale, eps_prefill(c.dtype))
        check(out[i], want, bound, f"query {i}")
    c.q, c.lens[0], c.context[0] = q[29:30], 30, 30
    assert torch.isnan(run_window(pkv, c, 20, 0)).all()


@pytest.mark.parametrize("at", [0, 29, 59])
def test_prefill_window_one_long_among_short(pkv, at):
    """A grid for the longest sequence, in which most work items have no rows; one
    sequence's lengths are wrong, a bound far above every length changes nothing."""
    lens = [5 + (7 * s) % 40 for s in range(60)]
    lens[at] = 1400
    c = Cache(lens, 4, 4, 64, 16, "bf16", seed=at)
    new = [1 + s % 3 for s in range(60)]
    new[at] = 1400
    wrong = 30
    c.context[wrong] = -1
    q = torch.randn(sum(new), c.H, 64, device=DEV).to(c.dtype)
    start = [sum(new[:s]) for s in range(61)]
    outs = []
    for bound in (1400, 1 << 30):
        err = new_err()
        out = torch.full_like(q, 7.0)
        pkv.paged_attention_prefill_window(out, q, c.k, c.v, c.tables, c.context,
                                           torch.tensor(start, dtype=torch.int32, device=DEV), c.scale, 100, 4,
                                           bound, err)
        assert err.item() == pkv.DEV_ERR_CONTEXT_LEN
        outs.append(out)
    assert torch.equal(*outs)
    for s, L in enumerate(lens):
        got = outs[0][start[s]:start[s + 1]]
        if s == wrong:
            assert (got == 7.0).all()
            continue
        for i in sorted({0, new[s] // 2, new[s] - 1}):
            want, _, bound, _ = attend(q[start[s] + i], c.rows_k[s], c.rows_v[s],
                                       seen_by(L, L - new[s] + i, 100, 4), c.scale, eps_prefill(c.dtype))
            check(got[i], want, bound, f"{s} {i}")


def test_prefill_window_last_query_sees_what_decode_shows(pkv):
    c = Cache((900, 77), 2, 4, 128, 16, "bf16")
    new = [300, 77]
    q = torch.randn(sum(new), c.H, 128, device=DEV).to(c.dtype)
    out = run_prefill(pkv, c, new, 128, 4, q)
    c.q = torch.stack([q[299], q[376]])
    ref = run_window(pkv, c, 128, 4)
    got = torch.stack([out[299], out[376]])
    # the prefill's weights are off by eps_prefill each (a sum of them, relative to the values'
    # size, by no more), both outputs by their own rounding
    size = torch.cat([v.abs().amax(1) for v in c.rows_v]).max().item()
    assert (got.float() - ref.float()).abs().max() <= 2 * half_step(c.dtype) * ref.float().abs().max() \
        + eps_prefill(c.dtype) * size


def test_prefill_window_agrees_with_prefill_when_all_is_seen(pkv):
    """Both are within their bound of the same exact value: the window's
    probabilities have one 16-bit part, the prefill's two."""
    c = Cache((900, 77), 2, 4, 128, 16, "bf16")
    new = [300, 77]
    q = torch.randn(sum(new), c.H, 128, device=DEV).to(c.dtype)
    out = run_prefill(pkv, c, new, 1000, 0, q)
    ref = torch.empty_like(out)
    start = torch.tensor([0, 300, 377], dtype=torch.int32, device=DEV)
    pkv.paged_attention_prefill(ref, q, c.k, c.v, c.tables, c.context, start, c.scale, 300)
    for row, s, P in ((0, 0, 600), (150, 0, 750), (299, 0, 899), (300, 1, 0), (376, 1, 76)):
        want, _, bound, _ = attend(q[row], c.rows_k[s], c.rows_v[s], seen_by(c.lens[s], P, 1000, 0), c.scale,
                                   eps_prefill(c.dtype))
        check(out[row], want, bound, f"window {row}")
        check(ref[row], want, bound, f"prefill {row}")


def test_prefill_window_gives_up_on_a_wait(pkv):
    """With a limit of 0 any wait not over at its first test gives up: the call
    reports it and the next one works."""
    c = Cache((900, 77), 2, 4, 128, 16, "bf16")
    new = [300, 77]
    q = torch.randn(sum(new), c.H, 128, device=DEV).to(c.dtype)
    good = run_prefill(pkv, c, new, 100, 4, q)
    old, err = pkv.get_wait_timeout_ns(), new_err()
    try:
        pkv.set_wait_timeout_ns(0)
        run_prefill(pkv, c, new, 100, 4, q, err)
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_timeout_ns(old)
    assert int(err.item()) == pkv.DEV_ERR_TIMEOUT
    err.zero_()
    assert torch.equal(run_prefill(pkv, c, new, 100, 4, q, err), good) and int(err.item()) == 0


@pytest.mark.parametrize("dtype,D,bs,Hkv,G,lens,new", [
    ("bf16", 128, 16, 8, 4, (2777,), (100,)),            # one chunk: clusters share its tiles
    ("f16", 64, 8, 1, 1, (9000,), (130,)),
    ("f16", 128, 32, 2, 7, (1500, 3, 4000), (5, 3, 17)),
    ("bf16", 64, 16, 2, 3, (4000,) * 3, (1, 1, 1)),       # single queries
    ("bf16", 128, 16, 20, 1, (600,) * 8, (600,) * 8),     # many tiles, none shared
])
@pytest.mark.parametrize("window,sinks", [(1024, 4), (100, 300), (1 << 30, 0)])
def test_prefill_window_shapes(pkv, dtype, D, bs, Hkv, G, lens, new, window, sinks):
    c = Cache(lens, Hkv, G, D, bs, dtype, seed=3)
    q = torch.randn(sum(new), c.H, D, device=DEV).to(c.dtype)
    err = new_err()
    out = run_prefill(pkv, c, list(new), window, sinks, q, err)
    assert int(err.item()) == 0
    assert torch.equal(run_prefill(pkv, c, list(new), window, sinks, q, err), out)
    at = 0
    for s, L in enumerate(lens):
        for i in sorted({0, 1, new[s] // 2, new[s] - 2, new[s] - 1} & set(range(new[s]))):
            want, _, bound, _ = attend(q[at + i], c.rows_k[s], c.rows_v[s], seen_by(L, L - new[s] + i, window, sinks),
                                       c.scale, eps_prefill(c.dtype))
            check(out[at + i], want, bound, f"L={L} i={i}")
        at += new[s]
    assert torch.isfinite(out).all()


def test_prefill_window_device_errors(pkv):
    c = Cache((400, 50), 1, 2, 64, 16, "f16")
    new = [100, 50]
    q = torch.randn(150, 2, 64, device=DEV).half()
    good = run_prefill(pkv, c, new, 60, 4, q)
    err = new_err()
    c.tables[0, 10] = 1 << 20          # no query sees it
    assert torch.equal(run_prefill(pkv, c, new, 60, 4, q, err), good) and int(err.item()) == 0
    c.tables[0, 390 // 16] = -1
    run_prefill(pkv, c, new, 60, 4, q, err)
    assert int(err.item()) == pkv.DEV_ERR_BLOCK_ID
    err.zero_()
    c.context[1] = 49                  # more queries than tokens
    run_prefill(pkv, c, new, 60, 4, q, err)
    assert int(err.item()) & pkv.DEV_ERR_CONTEXT_LEN


# ---- streams, graphs, the binding ---------------------------------------------------------------


def test_other_stream_and_captured_graph(pkv):
    """The calls on a side stream, captured together and replayed on new values."""
    c = Cache((3000, 500, 1), 2, 4, 128, 16, "f16", seed=2)
    B = 3
    ws, ws2 = pkv.new_window_workspace(B, c.H, 2, 128), pkv.new_scores_workspace(B, c.H, 2, 128, 3000)
    out, out2 = torch.zeros_like(c.q), torch.zeros_like(c.q)
    sc = torch.zeros(B, 2, 3000, device=DEV)
    so, kept = torch.zeros(B, 2, 200, device=DEV), torch.zeros(B, 2, 200, dtype=torch.int32, device=DEV)
    nl = torch.zeros(B, dtype=torch.int32, device=DEV)
    spare = torch.arange(c.nb, c.nb + 39, dtype=torch.int32).reshape(3, 13)
    k = torch.cat([c.k, torch.zeros_like(c.k[:39])])
    v = torch.cat([c.v, torch.zeros_like(c.v[:39])])
    dst = torch.full_like(c.tables, -1)
    dst[:, :13] = spare.to(DEV)

    def step():
        pkv.paged_attention_decode_window(out, c.q, k, v, c.tables, c.context, c.scale, 400, 4, 3000, ws)
        pkv.paged_attention_decode_scores(out2, sc, c.q, k, v, c.tables, c.context, c.scale, 3000, ws2)
        pkv.evict_tokens(k, v, sc, so, c.tables, dst, c.context, nl, kept, 4, 20, 3000)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    eager = [t.clone() for t in (out, out2, sc, so, kept, nl, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, out2, sc, so):
        t.fill_(0.0)
    kept.fill_(0)
    k[c.nb:] = 0
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((out, out2, sc, so, kept, nl, k, v), eager):
        assert torch.equal(torch.nan_to_num(a.float(), -1.0), torch.nan_to_num(b.float(), -1.0))
    c.q.copy_(torch.randn_like(c.q))
    graph.replay()
    check_window(c, out, 400, 4, "replayed")
    # an explicit stream
    third = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run_window(pkv, c, 400, 4, stream=third)
    third.synchronize()
    assert torch.equal(got, out)


def test_binding_refusals(pkv):
    c = Cache((100, 20), 2, 2, 64, 16, "f16")
    ws = pkv.new_window_workspace(2, c.H, 2, 64)
    good = dict(out=torch.empty_like(c.q), q=c.q, k_cache=c.k, v_cache=c.v, block_tables=c.tables,
                context_lens=c.context, scale=1.0, window=5, num_sinks=0, max_context_len=100, workspace=ws)
    pkv.paged_attention_decode_window(**good)
    for name, value in (("q", c.q.float()), ("q", c.q[:1]), ("out", c.q.cpu()), ("v_cache", c.v[:-1]),
                        ("block_tables", c.tables.long()), ("context_lens", c.context[:1]), ("q", c.q[0]),
                        ("k_cache", c.k.transpose(2, 3)), ("block_tables", c.tables.t()), ("workspace", ws.cpu())):
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_window(**{**good, name: value})
    for name, value in (("window", 0), ("num_sinks", -1), ("max_context_len", 10 ** 6), ("workspace", ws[:64])):
        with pytest.raises(pkv.PkvError):
            pkv.paged_attention_decode_window(**{**good, name: value})
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_window(**good, dev_err=torch.zeros(1, device=DEV))
    sc = torch.zeros(2, 2, 100, device=DEV)
    wss = pkv.new_scores_workspace(2, c.H, 2, 64, 100)
    for bad in (sc.double(), sc[:, :1], sc[0], sc.cpu()):
        with pytest.raises(ValueError):
            pkv.paged_attention_decode_scores(good["out"], bad, c.q, c.k, c.v, c.tables, c.context, 1.0, 100, wss)
    with pytest.raises(pkv.PkvError):
        pkv.paged_attention_decode_scores(good["out"], sc[:, :, :50].contiguous(), c.q, c.k, c.v, c.tables, c.context,
                                          1.0, 100, wss)
    kept = torch.zeros(2, 2, 10, dtype=torch.int32, device=DEV)
    n = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(pkv.PkvError):
        pkv.evict_tokens(c.k, c.v, sc, sc, c.tables, c.tables, c.context, n, kept, 8, 8, 100)  # more than the budget
    with pytest.raises(ValueError):
        pkv.evict_tokens(c.k, c.v, sc, sc, c.tables, c.tables, c.context, n, kept, 0, 0, 100, head_dim=128)


# ---- together ---------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_session(pkv, dtype):
    """Two users fork a shared system prompt, prefill their own, decode with
    scores, and are cut to a budget twice; a plain model of the kept rows in 64
    bits follows along. The system prompt's blocks survive the users' cuts."""
    import paged_kv_cache_204_gb300.block_manager as bmod
    D, Hkv, G, bs, MB = 64, 2, 4, 16, 64
    H, td = Hkv * G, TD[dtype]
    gen = torch.Generator(device=DEV).manual_seed(4)
    norm = lambda *sh: torch.randn(*sh, device=DEV, generator=gen).to(td)
    nb = 160
    k, v = (torch.full((nb, Hkv, bs, D), float("nan"), device=DEV, dtype=td) for _ in range(2))
    bm = bmod.BlockManager(nb, bs, seed=6)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    err = new_err()

    def write(slots, kk, vv):
        pkv.reshape_and_cache(kk, vv, k, v, up(slots), dev_err=err)

    root = bm.add_seq()
    sys_k, sys_v = norm(70, Hkv, D), norm(70, Hkv, D)
    write(bm.append(root, 70)[0], sys_k, sys_v)
    users, model = [], []
    for n in (200, 90):
        u = bm.fork(root)
        slots, cow = bm.append(u, n)
        if cow is not None:
            pkv.copy_blocks(k, v, up(np.array([cow], np.int64)), dev_err=err)
        kk, vv = norm(n, Hkv, D), norm(n, Hkv, D)
        write(slots, kk, vv)
        users.append(u)
        model.append([torch.cat([sys_k, kk]).transpose(0, 1).contiguous(),
                      torch.cat([sys_v, vv]).transpose(0, 1).contiguous()])
    scale, eps = 1.0 / 8.0, eps_prefill(td)
    # the prompts, seen through a window
    bt, cl = bm.export(users, MB)
    q, start = norm(290, H, D), up(np.array([0, 200, 290], np.int32))
    out = torch.empty_like(q)
    pkv.paged_attention_prefill_window(out, q, k, v, up(bt), up(cl), start, scale, 100, 4, 200, dev_err=err)
    for row, s, P in ((0, 0, 70), (199, 0, 269), (200, 1, 70), (289, 1, 159)):
        want, _, bound, _ = attend(q[row], *model[s], seen_by(int(cl[s]), P, 100, 4), scale, eps)
        check(out[row], want, bound, f"prefill row {row}")
    scores = torch.zeros(2, Hkv, MB * bs, device=DEV)
    total = [torch.zeros(Hkv, int(n), dtype=torch.float64, device=DEV) for n in cl]
    slack = [torch.zeros_like(t) for t in total]
    ws = pkv.new_scores_workspace(2, H, Hkv, D, MB * bs)
    for step in range(24):
        slots, pairs = bm.append_batch(users, [1, 1])
        if len(pairs):
            pkv.copy_blocks(k, v, up(pairs), dev_err=err)
        kk, vv = norm(2, Hkv, D), norm(2, Hkv, D)
        write(slots, kk, vv)
        bt, cl = bm.export(users, MB)
        q = norm(2, H, D)
        out = torch.empty_like(q)
        pkv.paged_attention_decode_scores(out, scores, q, k, v, up(bt), up(cl), scale, MB * bs, ws, scores=scores,
                                          dev_err=err)
        for s in range(2):
            model[s] = [torch.cat([m, r[s][:, None]], 1) for m, r in zip(model[s], (kk, vv))]
            L = int(cl[s])
            want, w, bound, rel = attend(q[s], *model[s], torch.ones(L, dtype=torch.bool), scale, eps_p(td))
            check(out[s], want, bound, f"step {step}")
            part = w.reshape(Hkv, G, L)
            grow = lambda t: torch.cat([t, torch.zeros(Hkv, 1, dtype=torch.float64, device=DEV)], 1)
            total[s] = grow(total[s]) + part.sum(1)
            slack[s] = grow(slack[s]) + (part * (rel.reshape(Hkv, G, 1) + (G + 2) * 2.0 ** -23)).sum(1) \
                + total[s] * 2.0 ** -23
            check(scores[s, :, :L], total[s], slack[s], f"step {step} scores")
        if step in (9, 19):
            budget = 120 if step == 9 else 61
            new = [min(int(n), budget) for n in cl]
            before, after, _ = bm.shrink_batch(users, new, MB)
            kept = torch.full((2, Hkv, budget), -1, dtype=torch.int32, device=DEV)
            lens = up(cl)
            by = scores.cpu().numpy().copy()
            pkv.evict_tokens(k, v, scores, scores, up(before), up(after), lens, lens, kept, 4, 30, MB * bs,
                             dev_err=err)
            assert lens.tolist() == new
            for s in range(2):
                keep = torch.tensor([kept_of(by[s, h], int(cl[s]), budget, 4, 30) for h in range(Hkv)], device=DEV)
                assert torch.equal(kept[s, :, :new[s]].long(), keep)
                pick = lambda t: torch.stack([t[h][keep[h]] for h in range(Hkv)])
                model[s] = [pick(m) for m in model[s]]
                total[s], slack[s] = pick(total[s]), pick(slack[s])
    # what the system prompt's own sequence holds was not touched
    bt, cl = bm.export([root], MB)
    c = norm(1, H, D)
    out = torch.empty_like(c)
    pkv.paged_attention_decode_window(out, c, k, v, up(bt), up(cl), scale, 50, 4, 70,
                                      pkv.new_window_workspace(1, H, Hkv, D), dev_err=err)
    want, _, bound, _ = attend(c[0], sys_k.transpose(0, 1), sys_v.transpose(0, 1), seen_by(70, 69, 50, 4), scale,
                               eps_p(td))
    check(out[0], want, bound, "system prompt")
    assert int(err.item()) == 0
    bm.close()


# ---- far blocks, calls at once ------------------------------------------------------------------


def test_blocks_beyond_32_bit_offsets(pkv):
    """Pools of more than 2^31 elements: the same rows in the last blocks give
    what they give in a small pool, bit for bit."""
    c = Cache((1000, 333), 8, 4, 128, 32, "bf16", seed=4)
    far = 65536 + 200 - c.nb                              # 65736 blocks x 8 x 32 x 128 elements
    k = torch.empty((far + c.nb, 8, 32, 128), dtype=c.dtype, device=DEV)
    v = torch.empty_like(k)
    assert k.numel() > 1 << 31
    k[far:], v[far:] = c.k, c.v
    near, tables = c.tables, torch.where(c.tables >= 0, c.tables + far, c.tables)
    q = torch.randn(333 + 50, c.H, 128, device=DEV).to(c.dtype)
    sc = [torch.zeros(2, 8, 1000, device=DEV) for _ in range(2)]
    results, results_pools = [], [(c.k, c.v)]
    for pools, table, score in (((c.k, c.v), near, sc[0]), ((k, v), tables, sc[1])):
        c.k, c.v = pools
        c.tables = table
        res = [run_window(pkv, c, 300, 4), run_prefill(pkv, c, [333, 50], 300, 4, q)]
        res.append(run_scores(pkv, c, None, score))
        kept = torch.zeros(2, 8, 200, dtype=torch.int32, device=DEV)
        new = torch.zeros(2, dtype=torch.int32, device=DEV)
        pkv.evict_tokens(c.k, c.v, score, score, table, table, c.context, new, kept, 4, 50, 1000)
        results.append(res + [score, kept, new])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    for small, large in ((results_pools[0][0], k), (results_pools[0][1], v)):
        assert torch.equal(small.view(torch.int16), large[far:].view(torch.int16))


def test_two_calls_at_once(pkv):
    """Two streams, a workspace each: what each call gives by itself."""
    c = [Cache((9000, 40, 2500), 2, 4, 128, 16, "f16", seed=s) for s in (5, 6)]
    alone = [(run_window(pkv, x, 3000, 4), run_scores(pkv, x, None, torch.zeros(3, 2, 9000, device=DEV))) for x in c]
    ws = [(pkv.new_window_workspace(3, x.H, 2, 128), pkv.new_scores_workspace(3, x.H, 2, 128, 9000)) for x in c]
    sc = [torch.zeros(3, 2, 9000, device=DEV) for _ in c]
    out = [(torch.zeros_like(x.q), torch.zeros_like(x.q)) for x in c]
    streams = [torch.cuda.Stream() for _ in c]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, w, s, o, st in zip(c, ws, sc, out, streams):
            pkv.paged_attention_decode_window(o[0], x.q, x.k, x.v, x.tables, x.context, x.scale, 3000, 4, 9000, w[0],
                                              stream=st)
            pkv.paged_attention_decode_scores(o[1], s, x.q, x.k, x.v, x.tables, x.context, x.scale, 9000, w[1],
                                              stream=st)
    torch.cuda.synchronize()
    for o, a in zip(out, alone):
        assert torch.equal(o[0], a[0]) and torch.equal(o[1], a[1])

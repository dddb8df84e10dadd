"""The rotating cache writes on the GPU: the bytes of the rule worked out in
binary32 on the host, for every type of cache, pairing, number of axes and row
layout; idle tokens, slots that store nothing, bad slots and positions; in
place, strided, on another stream, in a replayed graph; and with the calls
that belong beside them."""
import numpy as np
import pytest
import torch

from rope_helpers import F, e4m3_rows, q4_rows, turned

pytestmark = pytest.mark.gpu

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"
K_SCALE, V_SCALE = 0.017, 0.023


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_204_gb300 as m
    return m


class Step:
    """A step of T tokens into scattered slots. Rows lie in one packed projection, or apart."""

    def __init__(self, pkv, T, H, G, D, bs, dtype, cache="same", rot=None, axes=1, interleaved=False, packed=True, seed=0,
                 max_position=5000):
        self.pkv, self.T, self.H, self.G, self.D, self.bs = pkv, T, H, G, D, bs
        self.dtype, self.cache, self.interleaved = TD[dtype], cache, interleaved
        self.rot = D if rot is None else rot
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        if packed:
            rows = torch.randn(T, H + 2 * G, D, device=DEV, generator=gen, dtype=torch.float32).to(self.dtype)
            self.q, self.k, self.v = rows[:, :H], rows[:, H:H + G], rows[:, H + G:]
        else:
            self.q, self.k, self.v = (torch.randn(T, n, D, device=DEV, generator=gen).to(self.dtype) for n in (H, G, G))
        self.table = pkv.rope_table(max_position, self.rot)
        self.positions = rng.integers(0, max_position, (axes, T)).astype(np.int32)
        self.positions[:, -1] = max_position - 1
        self.axis = rng.integers(0, axes, self.rot // 2)
        self.nb = -(-T // bs) + 3
        self.slots = rng.permutation(self.nb * bs)[:T].astype(np.int64)
        width = {"same": D, "fp8": D, "q4": D // 16 * 9}[cache]
        pool = lambda: torch.from_numpy(rng.integers(0, 256, (self.nb, G, bs, width * (self.dtype.itemsize if cache == "same" else 1)),
                                                     dtype=np.uint8)).to(DEV)
        self.k_bytes, self.v_bytes = pool(), pool()
        view = (lambda p: p.view(self.dtype)) if cache == "same" else (lambda p: p)
        self.k_cache, self.v_cache = view(self.k_bytes), view(self.v_bytes)
        self.q_out = torch.full((T, H, D), float("nan"), device=DEV, dtype=self.dtype)

    def expected(self):
        """(q_out, K pool bytes, V pool bytes) after the call."""
        tab = self.table.cpu().numpy()
        live = self.positions[0] >= 0
        q_out, k_bytes, v_bytes = self.q_out.clone().cpu(), self.k_bytes.cpu().numpy().copy(), self.v_bytes.cpu().numpy().copy()
        f = lambda t: t[torch.from_numpy(live).to(DEV)].float().cpu().numpy()
        pos = self.positions[:, live]
        q_out[torch.from_numpy(live)] = torch.from_numpy(turned(f(self.q), tab, pos, self.axis, self.interleaved)).to(self.dtype)
        k, v = turned(f(self.k), tab, pos, self.axis, self.interleaved), f(self.v)
        slots = self.slots[live]
        for pool, x, scale in ((k_bytes, k, K_SCALE), (v_bytes, v, V_SCALE)):
            if self.cache == "fp8":
                rows = e4m3_rows(x, scale)
            elif self.cache == "q4":
                rows = q4_rows(x)
            else:
                rows = torch.from_numpy(x).to(self.dtype).view(torch.uint8).numpy()
            some = slots >= 0
            pool[slots[some] // self.bs, :, slots[some] % self.bs] = rows[some]
        return q_out, k_bytes, v_bytes

    def run(self, q_out=None, stream=None, err=None):
        pos = torch.from_numpy(self.positions).to(DEV)
        pos = pos[0] if len(pos) == 1 else pos
        axis = None if len(self.positions) == 1 else bytes(self.axis.tolist())
        args = [self.q_out if q_out is None else q_out, self.q, self.k, self.v, self.k_cache, self.v_cache,
                torch.from_numpy(self.slots).to(DEV), pos, self.table]
        more = dict(pair_axis=axis, interleaved=self.interleaved, dev_err=err, stream=stream)
        call = {"same": lambda: self.pkv.rope_and_cache(*args, **more),
                "fp8": lambda: self.pkv.rope_and_cache_fp8(*args, K_SCALE, V_SCALE, **more),
                "q4": lambda: self.pkv.rope_and_cache_q4_0(*args, **more)}[self.cache]
        call()
        return call

    def check(self, want, q_out=None):
        torch.cuda.synchronize()
        q = self.q_out if q_out is None else q_out
        same = lambda a, b: torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        assert same(q.cpu(), want[0]), "q_out"
        assert np.array_equal(self.k_bytes.cpu().numpy(), want[1]), "K"
        assert np.array_equal(self.v_bytes.cpu().numpy(), want[2]), "V"


SHAPES = [  # T, q heads, kv heads, head_dim, block_size
    (1, 32, 8, 128, 16), (3, 1, 1, 64, 8), (33, 7, 1, 128, 32), (100, 12, 4, 64, 16), (517, 40, 40, 128, 8),
    (2000, 32, 8, 64, 32)]
KINDS = [("f32", "same"), ("f16", "same"), ("bf16", "same"), ("f16", "fp8"), ("bf16", "fp8"), ("f16", "q4"), ("bf16", "q4")]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,cache", KINDS)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bytes(pkv, shape, dtype, cache, interleaved):
    T, H, G, D, bs = shape
    for i, rot in enumerate([D, D // 2, D // 4, 16]):
        s = Step(pkv, T, H, G, D, bs, dtype, cache, rot, 1, interleaved, packed=i % 2 == 0, seed=T + i)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        want = s.expected()
        s.run(err=err)
        s.check(want)
        assert err.item() == 0


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("dtype,cache", KINDS)
def test_axes(pkv, dtype, cache, axes):
    for i, (T, H, G, D, bs) in enumerate(SHAPES):
        s = Step(pkv, T, H, G, D, bs, dtype, cache, [D, D // 2][i % 2], axes, bool(i & 2), seed=axes)
        want = s.expected()
        s.run()
        s.check(want)


def test_sections_are_runs_of_one_axis(pkv):
    """Sections of three axes whose positions agree give the bytes of one axis."""
    s = Step(pkv, 50, 8, 2, 128, 16, "bf16", axes=3)
    s.axis = np.frombuffer(pkv.rope_sections(16, 24, 24), np.uint8)
    assert s.axis.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    s.positions[1:] = s.positions[0]
    want = s.expected()
    s.run()
    s.check(want)
    one = Step(pkv, 50, 8, 2, 128, 16, "bf16", axes=3)
    one.positions = s.positions[:1]
    one.run()
    torch.cuda.synchronize()
    assert torch.equal(one.q_out, s.q_out) and torch.equal(one.k_bytes, s.k_bytes)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_against_64_bits(pkv, dtype):
    """q_out against the formula in 64 bits: three roundings to binary32 (two products, a sum of at most
    |a| + |b|, all of 2^-24 relative at most) and one to the type."""
    s = Step(pkv, 300, 8, 2, 128, 16, dtype)
    s.run()
    c = s.table[torch.from_numpy(s.positions[0]).long().to(DEV)].double()
    x = s.q.double()
    a, b, c, sn = x[..., :64], x[..., 64:], c[:, None, :64], c[:, None, 64:]
    want = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    tol = 2 * 2.0 ** -24 * size * (1 + 2.0 ** -20) + torch.finfo(s.dtype).eps / 2 * (want.abs() + 2.0 ** -22 * size)
    tol += torch.finfo(s.dtype).smallest_normal * torch.finfo(s.dtype).eps
    assert ((s.q_out.double() - want).abs() <= tol).all()


def test_table_of_far_positions(pkv):
    """Angles of far positions come from 64 bits: the table's sines and cosines are the formula's to a half step."""
    t = pkv.rope_table(1 << 17, 64, base=10000.0).double().cpu().numpy()
    P = np.arange(1 << 17)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    # an angle up to 2^17 in 64 bits is off by 2^-36 or so, far below binary32's half step of 2^-25
    assert np.abs(t - np.concatenate([np.cos(P), np.sin(P)], 1)).max() <= 2.0 ** -25 + 2.0 ** -34


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_idle_tokens_and_unstored_slots(pkv, dtype, cache):
    s = Step(pkv, 40, 8, 4, 128, 16, dtype, cache, axes=2)
    s.positions[0, [3, 17, 39]] = [-1, -7, -(1 << 31)]  # idle: their slots and other positions hold anything
    s.positions[1, [3, 17]] = [1 << 30, -5]
    s.slots[3] = 1 << 60
    s.slots[[5, 20]] = [-1, -(1 << 40)]                 # turned, not stored
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = s.expected()
    s.run(err=err)
    s.check(want)
    assert err.item() == 0
    assert torch.isnan(s.q_out[[3, 17, 39]].float()).all() and torch.isfinite(s.q_out[[5, 20]].float()).all()


@pytest.mark.parametrize("dtype,cache", KINDS)
def test_bad_slots_and_positions(pkv, dtype, cache):
    s = Step(pkv, 12, 8, 4, 64, 8, dtype, cache, axes=2)
    s.slots[4] = s.nb * s.bs
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ok = s.slots.copy()
    s.slots[4] = -1  # as if it stored nothing
    want = s.expected()
    s.slots = ok
    s.run(err=err)
    s.check(want)
    assert err.item() == pkv.DEV_ERR_SLOT
    for axis, bad in ((0, 5000), (1, 5000), (1, -1), (1, (1 << 31) - 1)):
        s = Step(pkv, 12, 8, 4, 64, 8, dtype, cache, axes=2)
        s.axis[:] = 0  # the second axis is checked although no pair turns by it
        keep = s.positions.copy()
        s.positions[0, 6] = -1  # as if it were idle
        want = s.expected()
        s.positions = keep
        s.positions[axis, 6] = bad
        err.zero_()
        s.run(err=err)
        s.check(want)
        assert err.item() == pkv.DEV_ERR_POSITION
    s.run()  # without an error word


@pytest.mark.parametrize("packed", [False, True])
def test_in_place(pkv, packed):
    for T in (5, 700):
        s = Step(pkv, T, 32, 8, 128, 16, "bf16", packed=packed)
        want = s.expected()
        v = s.v.clone()
        s.run(q_out=s.q)
        s.check(want, s.q)
        assert torch.equal(v, s.v)


def test_strided_output(pkv):
    s = Step(pkv, 21, 8, 2, 64, 16, "f16")
    wide = torch.full((21, 11, 64), 7.0, device=DEV, dtype=torch.float16)
    want = s.expected()
    s.run(q_out=wide[:, 2:10])
    s.check(want, wide[:, 2:10])
    assert (wide[:, :2] == 7).all() and (wide[:, 10:] == 7).all()


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "fp8"), ("bf16", "q4")])
def test_stream_and_graph(pkv, dtype, cache):
    s = Step(pkv, 64, 32, 8, 128, 16, dtype, cache)
    want = s.expected()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        s.run(stream=other)
    other.synchronize()
    s.check(want)
    # a graph replayed over new rows and positions in the same places
    pos, slots = torch.from_numpy(s.positions[0]).to(DEV), torch.from_numpy(s.slots).to(DEV)
    args = [s.q_out, s.q, s.k, s.v, s.k_cache, s.v_cache, slots, pos, s.table]
    fn = {"same": pkv.rope_and_cache, "fp8": lambda *a: pkv.rope_and_cache_fp8(*a, K_SCALE, V_SCALE),
          "q4": pkv.rope_and_cache_q4_0}[cache]
    fn(*args)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn(*args)
    s.positions = (s.positions + 1234) % 5000
    pos.copy_(torch.from_numpy(s.positions[0]))
    s.k.mul_(-1.5)
    s.q.add_(0.25)
    want = s.expected()
    g.replay()
    s.check(want)


def test_positions_of_zero_store_what_reshape_and_cache_stores(pkv):
    """At position 0 nothing turns: the pools get the bytes of the plain writes."""
    for dtype, cache in KINDS:
        s = Step(pkv, 60, 8, 4, 128, 16, dtype, cache, packed=False)
        s.positions[:] = 0
        k, v = s.k_cache.clone(), s.v_cache.clone()
        slots = torch.from_numpy(s.slots).to(DEV)
        if cache == "same":
            pkv.reshape_and_cache(s.k, s.v, k, v, slots)
        elif cache == "fp8":
            pkv.reshape_and_cache_fp8(s.k, s.v, k, v, slots, K_SCALE, V_SCALE)
        else:
            pkv.reshape_and_cache_q4_0(s.k, s.v, k, v, slots)
        s.run()
        torch.cuda.synchronize()
        # (x c - y 0 is x, but for the sign of a zero)
        got, want = (s.k_cache, k) if cache != "same" else (s.k_cache + 0, k + 0)
        if cache == "same":
            got, want = got.view(torch.uint8), want.view(torch.uint8)
        assert torch.equal(got, want) and torch.equal(s.v_bytes, v.view(torch.uint8))
        assert torch.equal(s.q_out, s.q)


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "q4"), ("bf16", "fp8")])
def test_slots_past_four_gigabytes(pkv, dtype, cache):
    """Slots at the far end of pools of more than 2^32 bytes: the same bytes as at the near end."""
    s = Step(pkv, 50, 8, 4, 128, 16, dtype, cache)
    want = s.expected()
    width = s.k_cache.shape[3] * s.k_cache.element_size()
    nb = (1 << 32) // (4 * 16 * width) + 500
    pools = [torch.empty(nb, 4, 16, s.k_cache.shape[3], dtype=s.k_cache.dtype, device=DEV) for _ in range(2)]
    far = nb - s.nb
    for pool, near in zip(pools, (s.k_cache, s.v_cache)):
        pool[far:] = near
    s.k_cache, s.v_cache = pools
    s.slots = s.slots + far * 16
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    s.run(err=err)
    assert err.item() == 0
    for pool, bytes_ in zip(pools, want[1:]):
        assert np.array_equal(pool[far:].contiguous().view(torch.uint8).cpu().numpy().reshape(bytes_.shape), bytes_)
    assert torch.equal(s.q_out.cpu().view(torch.uint8), want[0].view(torch.uint8))


def test_binding_refusals(pkv):
    s = Step(pkv, 10, 8, 2, 128, 16, "bf16", axes=2)
    pos, slots = torch.from_numpy(s.positions).to(DEV), torch.from_numpy(s.slots).to(DEV)
    axis = bytes(s.axis.tolist())
    good = dict(q_out=s.q_out, q=s.q, k=s.k, v=s.v, k_cache=s.k_cache, v_cache=s.v_cache, slot_mapping=slots, positions=pos,
                cos_sin=s.table, pair_axis=axis)
    for name, bad in (("q", s.q.float()), ("q", s.q[:, :, ::2]), ("q", s.q.transpose(0, 1)), ("q", s.q.cpu()), ("k", s.k[:5]),
                      ("k", s.k[:, :1]), ("v", s.v.half()), ("q_out", s.q_out[:, :4]), ("k_cache", s.k_cache.float()),
                      ("v_cache", s.v_cache[:2]), ("slot_mapping", slots.int()), ("slot_mapping", slots[:3]),
                      ("positions", pos.long()), ("positions", pos[:, :4]), ("positions", pos[None]), ("cos_sin", s.table.double()),
                      ("cos_sin", s.table[0]), ("cos_sin", s.table.t()), ("pair_axis", axis[:-1]), ("pair_axis", list(axis)),
                      ("dev_err", slots)):
        with pytest.raises((ValueError, TypeError)):
            pkv.rope_and_cache(**{**good, name: bad})
    for bad in (dict(pair_axis=None), dict(pair_axis=bytes([2] * 64)), dict(q_out=s.q[1:], q=s.q[:-1], k=s.k[1:], v=s.v[1:],
                                                                           slot_mapping=slots[1:], positions=pos[:, 1:].contiguous())):
        with pytest.raises(pkv.PkvError) as e:
            pkv.rope_and_cache(**{**good, **bad})
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    for cache in (pkv.rope_and_cache_q4_0, lambda **a: pkv.rope_and_cache_fp8(**a, k_scale=1.0, v_scale=1.0)):
        with pytest.raises(ValueError):
            cache(**good)


@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "fp8"), ("bf16", "q4"), ("f32", "same")])
def test_rows_of_one_buffer(pkv, dtype, cache):
    """Outputs, keys and values anywhere in one buffer, with strides of their own: refused where a byte of an output
    would lie on a key's or a value's, and else as from tensors of their own."""
    T, H, G, D = 7, 3, 1, 64
    rng = np.random.default_rng(8)
    done = {True: 0, False: 0}
    chunk = 16 // TD[dtype].itemsize
    for i in range(100):
        s = Step(pkv, T, H, G, D, 8, dtype, cache, packed=False, seed=i)
        want = s.expected()
        k, v = s.k.clone(), s.v.clone()
        buf = torch.zeros(40 * T * D, device=DEV, dtype=s.dtype)
        used, views = [], []
        same = int(rng.integers(H + 2 * G, H + 2 * G + 4)) * D
        for heads in (H, G, G):  # one stride for all, whole heads apart or any chunks, or strides of their own
            stride = same if i % 2 else heads * D + int(rng.integers(0, 20)) * chunk
            if i % 4 == 1:
                at = int(rng.integers(0, 2 * same // D)) * D
            else:
                at = int(rng.integers(0, (2 * same if i % 4 == 3 else 30 * T * D) // chunk)) * chunk
            views.append(buf.as_strided((T, heads, D), (stride, D, 1), at))
            used.append({at + t * stride + e for t in range(T) for e in range(heads * D)})
        views[1].copy_(k)
        views[2].copy_(v)
        if used[1] & used[2] and not (used[0] & (used[1] | used[2])):
            continue  # (keys and values may share memory, but these have not both their values then)
        s.k, s.v = views[1], views[2]
        meet = bool(used[0] & (used[1] | used[2]))
        done[meet] += 1
        if meet:
            with pytest.raises(pkv.PkvError) as e:
                s.run(q_out=views[0])
            assert e.value.status == pkv.PKV_ERR_INVALID_ARG
        else:
            views[0].fill_(float("nan"))
            s.run(q_out=views[0])
            s.check(want, views[0])
    assert min(done.values()) >= 10, done

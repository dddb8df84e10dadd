"""The rotating cache writes without a GPU: refusals of the C entry points
(every call below returns before any device work) and of the binding."""
import pytest
import torch

FAKE = 0x100000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_204_gb300 as m
    return m


def calls(pkv):
    """(call, result with q_out as it is) of each entry point; a call takes changed arguments by name."""
    base = dict(out=FAKE, so=8 * 128, q=FAKE << 4, sq=8 * 128, k=FAKE, sk=2 * 128, v=FAKE, sv=2 * 128, kc=FAKE, vc=FAKE,
                slots=FAKE, pos=FAKE, table=FAKE, most=100, R=128, axis=None, axes=1, inter=0, T=4, H=8, G=2, D=128, bs=16,
                nb=10, dtype=1)
    tail = dict(err=None, stream=None)
    scales = dict(ks=0.5, vs=0.5)
    for fn, a in ((pkv.lib.pkv_rope_and_cache, {**base, **tail}), (pkv.lib.pkv_rope_and_cache_fp8, {**base, **scales, **tail}),
                  (pkv.lib.pkv_rope_and_cache_q4_0, {**base, **tail})):
        def call(fn=fn, a=a, **kw):
            return fn(*{**a, **{k: v for k, v in kw.items() if k in a}}.values())
        yield call


def test_refusals(pkv):
    INV, UNS, OK = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_OK
    for call in calls(pkv):
        assert call(T=0) == OK and call(T=0, out=None) == OK
        row = 8 * 128 * 2
        for bad in (dict(T=-1), dict(H=0), dict(G=0), dict(H=9), dict(D=0), dict(bs=0), dict(nb=0), dict(most=0), dict(R=0),
                    dict(R=-16), dict(axes=0), dict(axes=2), dict(out=None), dict(q=None), dict(k=None), dict(v=None),
                    dict(kc=None), dict(vc=None), dict(slots=None), dict(pos=None), dict(table=None), dict(out=FAKE + 8),
                    dict(q=FAKE + 2), dict(k=FAKE + 8), dict(v=FAKE + 4), dict(kc=FAKE + 8), dict(vc=FAKE + 8),
                    dict(slots=FAKE + 4), dict(pos=FAKE + 2), dict(table=FAKE + 4), dict(err=FAKE + 1), dict(so=8 * 128 - 8),
                    dict(sq=8 * 128 + 4), dict(sk=2 * 128 - 8), dict(sv=2 * 128 + 1), dict(sv=-2 * 128), dict(sq=1 << 62),
                    dict(axis=bytes([0] * 63 + [1])), dict(axes=3, axis=bytes([3] + [0] * 63)),
                    # q_out meets q: another stride, or rows that overlap
                    dict(q=FAKE, sq=8 * 128 + 8), dict(q=FAKE + row), dict(q=FAKE - 4 * row + 16)):
            assert call(**bad) == INV, bad
        for bad in (dict(D=96, R=96), dict(D=256), dict(bs=64), dict(dtype=3), dict(dtype=4), dict(dtype=9), dict(R=72),
                    dict(R=8), dict(R=144), dict(D=64, R=128), dict(axes=5, axis=bytes(64)), dict(H=65536, G=1),
                    dict(H=65536, G=65536)):
            assert call(**bad) == UNS, bad
    _, fp8, q4 = calls(pkv)
    assert fp8(dtype=0) == UNS and q4(dtype=0) == UNS
    for bad in (dict(ks=0.0), dict(vs=-1.0), dict(ks=float("nan")), dict(vs=float("inf"))):
        assert fp8(**bad) == INV, bad


def test_binding_refusals(pkv):
    cpu = torch.zeros(4, 2, 16, 128)
    x, p = torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int32)
    for fn, more in ((pkv.rope_and_cache, ()), (pkv.rope_and_cache_fp8, (1.0, 1.0)), (pkv.rope_and_cache_q4_0, ())):
        with pytest.raises(ValueError, match="CUDA"):
            fn(x, x, x, x, cpu, cpu, p.long(), p, torch.zeros(8, 128), *more)
        with pytest.raises(ValueError, match="tensor"):
            fn(x, x, x, x, None, cpu, p.long(), p, torch.zeros(8, 128), *more)


def test_sections(pkv):
    assert pkv.rope_sections(2, 0, 3) == bytes([0, 0, 2, 2, 2]) and pkv.rope_sections() == b""


def test_rule_of_the_tests(pkv):
    """The helpers' rows against the oracle's, where both have them: rows of 16-bit values."""
    import numpy as np
    import oracle
    from rope_helpers import e4m3_rows, q4_rows, q4_values
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((40, 128)) * np.exp(rng.uniform(-8, 4, (40, 1)))).astype(np.float16)
    x[3] = 0
    x[4, 5:9] = [2, -2, 2, -2]
    got = q4_rows(x.astype(np.float32))
    for i in range(40):
        want = oracle.q4_0_quantize_row(x[i].view(np.uint16), "f16")
        assert np.array_equal(got[i], want)
        assert np.array_equal(q4_values(got[i]), oracle.q4_0_values(want, 128))
    y = (x[:8].astype(np.float32) / np.float32(0.03)).astype(np.float64)
    assert np.array_equal(e4m3_rows(x[:8].astype(np.float32), 0.03), oracle.encode_e4m3(np.clip(y, -448, 448)))

"""Query outputs of the rotating cache writes that would lie on keys, values or caches are refused (every call below
returns before any device work)."""
import pytest

from test_rope_host import calls

MB = 1 << 20


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_204_gb300 as m
    return m


def apart(**kw):
    """4 tokens of 8 query and 2 kv heads of 128 values of 16 bits, pools of 10 blocks of 16 tokens: everything apart."""
    return dict(dict(out=1 * MB, q=2 * MB, k=3 * MB, v=4 * MB, kc=5 * MB, vc=6 * MB, slots=7 * MB, pos=8 * MB, table=9 * MB), **kw)


def test_output_on_keys_or_values(pkv):
    q_row, kv_row = 8 * 128 * 2, 2 * 128 * 2
    for call in calls(pkv):
        for name, stride in (("k", "sk"), ("v", "sv")):
            # rows that lie side by side: from the last byte of the first output to the first of the last
            for at in (1 * MB, 1 * MB - kv_row + 16, 1 * MB + q_row - 16, 1 * MB + 4 * q_row - 16, 1 * MB - 4 * kv_row + 16):
                assert call(**apart(**{name: at})) == pkv.PKV_ERR_INVALID_ARG, (name, at)
            # parts of one projection of 12 heads: outputs where the keys or the values are, or a chunk into them
            for at in (8 * 256, 0, 16, 10 * 256, -1 * 256, -2 * 256 + 16, 8 * 256 - 16, 2 * 12 * 256, -12 * 256 - 256):
                place = dict(so=12 * 128, sq=12 * 128, sk=12 * 128, sv=12 * 128, q=20 * MB)
                place[name] = 1 * MB + at
                hit = any(-kv_row < at + d * 12 * 256 < q_row for d in range(-3, 4))
                if hit:
                    assert call(**apart(**place)) == pkv.PKV_ERR_INVALID_ARG, (name, at)
            # other strides: only the last rows meet
            last = 1 * MB + 3 * 2 * q_row
            assert call(**apart(so=2 * 8 * 128, **{name: last - 3 * (kv_row + 16), stride: 2 * 128 + 8})) == pkv.PKV_ERR_INVALID_ARG
        assert call(**apart(T=1, k=1 * MB + q_row - 16)) == pkv.PKV_ERR_INVALID_ARG


def test_output_on_caches(pkv):
    for call, row in zip(calls(pkv), (256, 128, 72)):
        for name in ("kc", "vc"):
            size = 10 * 2 * 16 * row
            for at in (1 * MB, 1 * MB + 4 * 2048 - 16, 1 * MB - size + 16):
                assert call(**apart(**{name: at})) == pkv.PKV_ERR_INVALID_ARG, (name, at)


def test_refusals_with_everything_apart(pkv):
    """The refusals of single arguments, from a call in which nothing else stands against it."""
    INV, UNS = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED
    for call in calls(pkv):
        for bad in (dict(T=-1), dict(H=0), dict(G=0), dict(H=9), dict(bs=0), dict(nb=0), dict(most=0), dict(R=0), dict(axes=2),
                    dict(out=1 * MB + 8), dict(q=2 * MB + 2), dict(k=3 * MB + 8), dict(v=4 * MB + 4), dict(kc=5 * MB + 8),
                    dict(vc=6 * MB + 8), dict(slots=7 * MB + 4), dict(pos=8 * MB + 2), dict(table=9 * MB + 4), dict(err=MB + 1),
                    dict(so=8 * 128 - 8), dict(sq=8 * 128 + 4), dict(sk=2 * 128 - 8), dict(sv=2 * 128 + 1), dict(sq=1 << 62),
                    dict(axis=bytes([0] * 63 + [1])), dict(axes=3, axis=bytes([3] + [0] * 63)), dict(q=1 * MB, sq=8 * 128 + 8),
                    dict(q=1 * MB + 2048), dict(q=1 * MB - 4 * 2048 + 16),
                    *({name: None} for name in ("out", "q", "k", "v", "kc", "vc", "slots", "pos", "table"))):
            assert call(**apart(**bad)) == INV, bad
        for bad in (dict(D=96, R=96), dict(bs=64), dict(dtype=3), dict(R=72), dict(R=144), dict(axes=5, axis=bytes(64))):
            assert call(**apart(**bad)) == UNS, bad

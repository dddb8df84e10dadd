"""Prefill over quantised caches without a GPU: refusals of the C entry points
(every call below returns before any device work) and of the binding."""
import pytest
import torch

FAKE = 0x10000  # aligned, never dereferenced


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_cache_204_gb300 as m
    return m


def calls(pkv):
    head = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, qs=FAKE, scale=0.1)
    scales = dict(ks=0.5, vs=0.5)
    tail = dict(H=8, Hkv=2, D=128, bs=16, B=4, MB=8, NB=100, mql=64, dtype=2, ws=None, ws_bytes=0, err=None, stream=None)
    for fn, a in ((pkv.lib.pkv_paged_attention_prefill_fp8, {**head, **scales, **tail}),
                  (pkv.lib.pkv_paged_attention_prefill_q4_0, {**head, **tail})):
        def call(fn=fn, a=a, **kw):
            assert set(kw) <= set(a), kw
            return fn(*{**a, **kw}.values())
        yield call


def test_refusals(pkv):
    INV, UNS, WS, OK = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED, pkv.PKV_ERR_WORKSPACE, pkv.PKV_OK
    fp8, q4 = calls(pkv)
    for rc in (fp8, q4):
        assert rc(B=0) == OK and rc(mql=0) == OK and rc(B=0, q=None) == OK
        for bad in (dict(B=-1), dict(mql=-1), dict(H=9), dict(H=0), dict(Hkv=0), dict(D=0), dict(bs=0), dict(MB=0),
                    dict(NB=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(q=FAKE + 8),
                    dict(k=FAKE + 4), dict(v=None), dict(bt=FAKE + 2), dict(cl=None), dict(qs=None), dict(qs=FAKE + 2),
                    dict(err=FAKE + 1), dict(out=FAKE + 2)):
            assert rc(**bad) == INV, bad
        for bad in (dict(dtype=0), dict(dtype=3), dict(dtype=4), dict(D=96), dict(D=256), dict(bs=64), dict(bs=4),
                    dict(B=65536), dict(MB=1 << 28)):
            assert rc(**bad) == UNS, bad
        need = pkv.prefill_workspace_bytes(128)
        assert rc() == WS and rc(ws=FAKE, ws_bytes=need - 1) == WS and rc(ws=FAKE + 8, ws_bytes=need) == INV
        # queries are read by CTAs that come after others' outputs: no run in place
        assert rc(ws=FAKE, ws_bytes=need, out=FAKE) == INV
    for bad in (dict(ks=0.0), dict(ks=-1.0), dict(vs=float("nan")), dict(vs=float("inf")), dict(scale=1e30, ks=1e30)):
        assert fp8(**bad) == INV, bad


def test_workspace_sizes(pkv):
    assert pkv.prefill_workspace_bytes(128) >= pkv.prefill_workspace_bytes(64) > 0
    for D in (0, -64, 96, 256):
        assert pkv.prefill_workspace_bytes(D) == 0


def test_binding_wants_cuda_tensors(pkv):
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    t, n, q = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 64).half()
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_prefill_fp8(q, q, pool, pool, t, n, t, 1.0, 1.0, 1.0, 1, pool)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_attention_prefill_q4_0(q, q, pool, pool, t, n, t, 1.0, 1, pool)


def test_workspace_holds_what_is_used(pkv):
    """Of 152 CTAs: what each tells the join (32 bytes), and two places for 256 rows' maxima, sums and outputs in 32
    bits. Nothing beside that."""
    for D in (64, 128):
        assert pkv.prefill_workspace_bytes(D) == 152 * (32 + 2 * 256 * (8 + 4 * D))

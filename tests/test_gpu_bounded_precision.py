"""How precise the bounded-cache operators' outputs are where a bound of the largest possible error
says little: the size of the error over many outputs, weights far below the largest one, values of
infinity."""
import pytest
import torch

from bounded_helpers import DEV, Cache, attend, check, eps_p, seen_by
from test_gpu_bounded import check_scores, check_window, pkv, run_prefill, run_scores, run_window  # noqa: F401

pytestmark = pytest.mark.gpu


def rms(x):
    return x.double().pow(2).mean().sqrt().item()


def exact_rows(c, s, q, positions, window, sinks):
    """64-bit outputs [len(positions), H, D] of the queries q at the positions of sequence s."""
    L = c.lens[s]
    k, v = (r.double().repeat_interleave(c.G, 0) for r in (c.rows_k[s], c.rows_v[s]))
    seen = torch.stack([seen_by(L, P, window, sinks) for P in positions]).to(DEV)
    x = torch.einsum("nhd,hld->hnl", q.double(), k) * c.scale
    p = torch.softmax(x.masked_fill(~seen[None], float("-inf")), 2)
    return torch.einsum("hnl,hld->nhd", p, v)


@pytest.mark.parametrize("dtype,D,bs,Hkv,G,L,n,window,sinks", [
    ("bf16", 128, 16, 8, 4, 2777, 100, 1024, 4),      # a chunk: clusters share its tiles
    ("bf16", 128, 16, 20, 2, 1500, 1500, 700, 4),
    ("f16", 128, 16, 8, 4, 1501, 333, 1024, 0),
    ("bf16", 64, 8, 40, 1, 1500, 900, 500, 1),
    ("f16", 64, 8, 40, 1, 1500, 900, 500, 1),
])
def test_prefill_window_is_as_precise_as_its_type(pkv, dtype, D, bs, Hkv, G, L, n, window, sinks):
    """With w the relative error of a weight (independent from weight to weight) the output has an error of
    w times its own size before it is rounded, rms: out^2 is on average sum p^2 v^2 for values of either sign.
    Fp32 logits of this size are off by some 2^-18 and a weight in two 16-bit parts by 2^-16 at most, so w is
    below 2^-14; the rounding alone is 0.38 (rms, of the outputs' rms) of a half step of 2^-8 or 2^-11, 2^-12.4
    for binary16. Together: sqrt(1 + 2^-3.2) = 1.05 times the rounding, and no more than a per cent of
    chance over the 10^5 outputs. Weights in one part give 1.3 to 1.4."""
    c = Cache((L,), Hkv, G, D, bs, dtype, seed=L)
    q = torch.randn(n, c.H, D, device=DEV).to(c.dtype)
    out = run_prefill(pkv, c, [n], window, sinks, q)
    want = torch.cat([exact_rows(c, 0, q[a:a + 100], range(L - n + a, min(L, L - n + a + 100)), window, sinks)
                      for a in range(0, n, 100)])
    assert rms(out - want) <= 1.1 * rms(want.to(c.dtype) - want)


# ---- one large weight, many far below it ---------------------------------------------------------


def one_large(dtype, D, Hkv, G, L, bits):
    """Token 0 has a logit above all others by `bits` (base 2), and values of 0 in the even head dims: what
    an even dim of the output holds comes from the many small weights alone."""
    c = Cache((L, 700), Hkv, G, D, 16, dtype, seed=int(10 * bits))
    for s, n in enumerate(c.lens):
        c.rows_k[s].zero_()
        c.rows_k[s][:, 0, 0] = bits * 0.6931472 * D ** 0.5 / 16.0
        c.rows_v[s].abs_()
        c.rows_v[s][:, 0, ::2] = 0.0
        c.put(c.k, s, torch.arange(n), c.rows_k[s])
        c.put(c.v, s, torch.arange(n), c.rows_v[s])
    c.q.zero_()
    c.q[:, :, 0] = 16.0
    return c


@pytest.mark.parametrize("bits", [16.0, 23.0, 25.5, 27.0])
@pytest.mark.parametrize("dtype,D,Hkv,G", [("f16", 64, 2, 1), ("f16", 128, 1, 8), ("bf16", 128, 2, 4)])
def test_decode_keeps_small_weights(pkv, dtype, D, Hkv, G, bits):
    c = one_large(dtype, D, Hkv, G, 20011, bits)
    check_window(c, run_window(pkv, c, 15000, 1), 15000, 1, f"{bits} bits")
    new = torch.full((2, Hkv, c.max_len), float("nan"), device=DEV)
    out = run_scores(pkv, c, None, new)
    check_scores(c, out, None, new, f"{bits} bits")


@pytest.mark.parametrize("bits", [16.0, 23.0, 25.5, 27.0])
@pytest.mark.parametrize("dtype,D,Hkv,G", [("f16", 64, 2, 1), ("f16", 128, 1, 8), ("bf16", 128, 2, 4)])
def test_prefill_window_keeps_small_weights(pkv, dtype, D, Hkv, G, bits):
    """Few queries (clusters share a walk) and many (they do not)."""
    c = one_large(dtype, D, Hkv, G, 3000, bits)
    for n in (3, 700):
        q = c.q[:1].expand(2 * n, -1, -1).contiguous()
        out = run_prefill(pkv, c, [n, n], 2500, 1, q)
        for s, L in enumerate(c.lens):
            for i in sorted({0, 2, n // 2, n - 1}):
                P = L - n + i
                want, _, bound, _ = attend(q[0], c.rows_k[s], c.rows_v[s], seen_by(L, P, 2500, 1), c.scale,
                                           eps_p(c.dtype))
                check(out[s * n + i], want, bound, f"{bits} bits L={L} P={P}")


# ---- infinities among the values ----------------------------------------------------------------


@pytest.mark.parametrize("dtype,D,bs,Hkv,G", [("f16", 64, 8, 2, 1), ("f16", 128, 16, 1, 8), ("bf16", 128, 16, 2, 4),
                                             ("bf16", 64, 32, 2, 12), ("f32", 128, 16, 1, 2)])
@pytest.mark.parametrize("L,window", [(9, 5), (500, 300), (12011, 12000)])
def test_decode_infinity_in_a_value(pkv, dtype, D, bs, Hkv, G, L, window):
    """A visible value of infinity makes its head dim of the output infinite, two of either sign or a NaN
    make it a NaN; all other dims, and the scores, are what they are without. Weights lie within 2^-40 of
    each other, so that none is 0 in fp32."""
    c = Cache((L, L - 2), Hkv, G, D, bs, dtype, seed=L)
    c.q *= 0.5
    inf = float("inf")
    clean = [v.clone() for v in c.rows_v]
    for s, n in enumerate(c.lens):
        c.rows_v[s][:, n - 2, 5] = inf
        c.rows_v[s][:, n - 1, 11] = -inf
        c.rows_v[s][:, n - 3, 40] = inf
        c.rows_v[s][:, n - 4, 40] = -inf
        c.rows_v[s][:, n - 1, 50] = float("nan")
        c.put(c.v, s, torch.arange(n), c.rows_v[s])
    plain = torch.ones(D, dtype=torch.bool, device=DEV)
    plain[[5, 11, 40, 50]] = False
    new = torch.full((2, Hkv, L), float("nan"), device=DEV)
    for what, out, w in (("window", run_window(pkv, c, window, 1), window), ("scores", run_scores(pkv, c, None, new), L)):
        assert (out[..., 5] == inf).all() and (out[..., 11] == -inf).all(), what
        assert torch.isnan(out[..., 40]).all() and torch.isnan(out[..., 50]).all(), what
        for s, n in enumerate(c.lens):
            want, _, bound, _ = attend(c.q[s], c.rows_k[s], clean[s], seen_by(n, n - 1, w, 1), c.scale, eps_p(c.dtype))
            check(out[s][:, plain], want[:, plain], bound[:, plain], f"{what} L={n}")
    again = torch.full_like(new, float("nan"))
    c.rows_v = clean
    for s, n in enumerate(c.lens):
        c.put(c.v, s, torch.arange(n), clean[s])
    run_scores(pkv, c, None, again)
    assert torch.equal(torch.nan_to_num(new, -1.0), torch.nan_to_num(again, -1.0))


# ---- a scale of zero ----------------------------------------------------------------------------


@pytest.mark.parametrize("D,n", [(64, 3), (128, 400)])
def test_scale_of_zero_with_large_scores(pkv, D, n):
    """All logits are 0 however large q . k is (up to 10^37 here): every visible token has the same weight."""
    c = Cache((400,), 20, 1, D, 16, "bf16", seed=D)
    c.scale = 0.0
    c.k *= 3e17
    c.rows_k = [r * 3e17 for r in c.rows_k]
    q = (torch.randn(n, c.H, D, device=DEV) * 3e17).to(c.dtype)
    size = torch.einsum("nhd,hld->nhl", q.float().abs(), c.rows_k[0].float().abs())
    assert size.max() < 1e38 and (torch.einsum("nhd,hld->nhl", q.float(), c.rows_k[0].float()).abs() > 1e36).any()
    out = run_prefill(pkv, c, [n], 150, 4, q)
    c.q = q[-1:]
    dec = run_window(pkv, c, 150, 4)
    for i in sorted({0, n // 2, n - 1}):
        seen = seen_by(400, 400 - n + i, 150, 4).to(DEV)
        v = c.rows_v[0][:, seen].double()
        bound = (seen.sum() + 8) * 2.0 ** -23 * v.abs().mean(1) + (eps_p(c.dtype) + 2.0 ** -20) * v.abs().mean(1)
        check(out[i], v.mean(1), bound, f"query {i}")
        if i == n - 1:
            check(dec[0], v.mean(1), bound, "decode")


# ---- logits far from zero -----------------------------------------------------------------------


@pytest.mark.parametrize("D,Hkv,L,n", [(64, 2, 300, 3), (128, 20, 600, 500), (64, 1, 2000, 700)])
@pytest.mark.parametrize("dtype,log2", [("f16", 9), ("f16", 10), ("f16", 11), ("f16", 12), ("bf16", 10), ("bf16", 11),
                                        ("bf16", 12)])
def test_logits_far_from_zero(pkv, dtype, log2, D, Hkv, L, n):
    """Elements of +-2^log2: q . k is a whole multiple of 2^(2 log2 + 1), so that one logit is above all others or
    exactly as large as some, and the output is the mean of those tokens' values. (Weights of 1/c are off by 2^-24, their
    sum by c 2^-24.)"""
    c = Cache((L,), Hkv, 1, D, 16, dtype, seed=log2)
    sign = lambda x: torch.where(x < 0, -1.0, 1.0).to(c.dtype) * 2.0 ** log2
    c.rows_k[0] = sign(c.rows_k[0])
    c.put(c.k, 0, torch.arange(L), c.rows_k[0])
    q = sign(torch.randn(n, c.H, D, device=DEV))
    out = run_prefill(pkv, c, [n], 250, 4, q)
    c.q = q[-1:]
    dec = run_window(pkv, c, 250, 4)
    x = torch.einsum("nhd,hld->hnl", q.double(), c.rows_k[0].double())
    seen = torch.stack([seen_by(L, L - n + i, 250, 4) for i in range(n)]).to(DEV)
    assert x.abs().max() * c.scale < 2.0 ** 27
    x = x.masked_fill(~seen, float("-inf"))
    p = (x == x.amax(2, keepdim=True)).double()
    count = p.sum(2).T[..., None]
    want = torch.einsum("hnl,hld->nhd", p, c.rows_v[0].double()) / count
    size = torch.einsum("hnl,hld->nhd", p, c.rows_v[0].double().abs()) / count
    bound = (eps_p(c.dtype) + (2 * count + 8) * 2.0 ** -23) * size
    check(out, want, bound, "prefill")
    check(dec, want[-1:], bound[-1:], "decode")

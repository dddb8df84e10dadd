"""How precise the bounded-cache operators' outputs are where a bound of the largest possible error
says little: the size of the error over many outputs, weights far below the largest one, values of
infinity."""
import pytest
import torch

from bounded_helpers import DEV, Cache, seen_by
from test_gpu_bounded import pkv, run_prefill  # noqa: F401  (pkv: the module's fixture)

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

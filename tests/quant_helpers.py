"""Quantised pools, their 64-bit values and bounds of the prefill over them."""
from __future__ import annotations

import math

import numpy as np
import torch

from rope_helpers import q4_values

TD = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


class Batch:
    """Sequences of (context length, new tokens) over scattered blocks of quantised pools. Bytes that hold no token
    are 0xFF: NaN as an e4m3 code, a NaN scale and the largest codes as a q4_0 row."""

    def __init__(self, seqs, Hkv, G, D, bs, dtype, kind, seed=0, sigma=1.0, q_sigma=1.0, scale=None):
        self.seqs, self.Hkv, self.G, self.H, self.D, self.bs, self.kind = list(seqs), Hkv, G, Hkv * G, D, bs, kind
        self.dtype = TD[dtype]
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.k_scale, self.v_scale = (0.037, 0.021) if kind == "fp8" else (1.0, 1.0)
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.lens = [L for L, _ in self.seqs]
        self.new = [n for _, n in self.seqs]
        counts = [-(-L // bs) for L in self.lens]
        self.nb = sum(counts) + 3
        perm = rng.permutation(self.nb).astype(np.int32)
        self.bt = np.full((len(self.seqs), max(counts + [1]) + 1), -1, np.int32)
        at = 0
        for s, c in enumerate(counts):
            self.bt[s, :c] = perm[at:at + c]
            at += c
        width = D if kind == "fp8" else D // 16 * 9
        self.k, self.v = (torch.full((self.nb, Hkv, bs, width), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.k_rows, self.v_rows = [], []  # float64 values [Hkv, L, D]
        for s, L in enumerate(self.lens):
            for pool, rows, unit in ((self.k, self.k_rows, self.k_scale), (self.v, self.v_rows, self.v_scale)):
                raw = self.random_rows(gen, L, sigma / unit)
                self.put(pool, s, raw)
                rows.append(self.values(raw, unit))
        starts = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.q = (torch.randn(int(starts[-1]), self.H, D, device=DEV, generator=gen) * q_sigma).to(self.dtype)
        self.starts = torch.from_numpy(starts).to(DEV)
        self.context = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.tables = torch.from_numpy(self.bt).to(DEV)
        self.first = starts

    def random_rows(self, gen, L, sigma):
        x = torch.randn(self.Hkv, L, self.D, device=DEV, generator=gen) * sigma
        if self.kind == "fp8":
            return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes = torch.randint(0, 256, (self.Hkv, L, self.D // 2), device=DEV, generator=gen, dtype=torch.uint8)
        d = (torch.randn(self.Hkv, L, self.D // 32, device=DEV, generator=gen) * sigma / 4.6).half()
        return torch.cat([d.view(torch.uint8), codes], -1)

    def values(self, raw, unit):
        if self.kind == "fp8":
            return raw.view(torch.float8_e4m3fn).double() * float(np.float32(unit))
        return torch.from_numpy(q4_values(raw.cpu().numpy())).to(DEV)

    def put(self, pool, s, raw):
        pos = np.arange(raw.shape[1])
        if len(pos):
            pool[torch.from_numpy(self.bt[s][pos // self.bs]).long().to(DEV), :,
                 torch.from_numpy(pos % self.bs).to(DEV)] = raw.transpose(0, 1)

    def run(self, pkv, ws=None, err=None, out=None, max_new=None, stream=None):
        ws = pkv.new_prefill_workspace(self.D) if ws is None else ws
        out = torch.full_like(self.q, float("nan")) if out is None else out
        args = [out, self.q, self.k, self.v, self.tables, self.context, self.starts, self.scale]
        most = max(self.new) if max_new is None else max_new
        if self.kind == "fp8":
            pkv.paged_attention_prefill_fp8(*args, self.k_scale, self.v_scale, most, ws, dev_err=err, stream=stream)
        else:
            pkv.paged_attention_prefill_q4_0(*args, most, ws, dev_err=err, stream=stream)
        return out

    def check(self, out, what="", seqs=None):
        for s in range(len(self.seqs)) if seqs is None else seqs:
            L, n = self.seqs[s]
            if n == 0:
                continue
            got = out[self.first[s]:self.first[s] + n]
            for a in range(0, n, 256):
                b = min(n, a + 256)
                want, tol = self.exact(s, a, b)
                assert torch.isfinite(got[a:b]).all(), f"{what} seq {s} (L={L}, n={n}): not finite"
                off = (got[a:b].double() - want).abs() - tol
                assert (off <= 0).all(), (f"{what} seq {s} (L={L}, n={n}): {int((off > 0).sum())} values off, worst "
                                          f"{off.max().item():.3e} beyond {tol.max().item():.3e}")

    def exact(self, s, a, b):
        """Queries a .. b - 1 of sequence s in 64 bits, [b - a, H, D], and how far off the kernel may be.

        A logit: q and K enter as binary16 (q4_0's values d (q - 8) rounded, 2^-11 relative or, subnormal, 2^-25;
        e4m3 codes exact; bfloat16 queries a power of two of the row's own, values below 2^-28 of the largest
        rounded to 2^-39 of it), a sum of D products in fp32 (2^-23 of the sum of absolute products a step,
        whatever the order), scaled and shifted (3 more). A weight: an exponential of it, off by the logit's
        error and 2^-21, rounded to binary16 (2^-11 relative; once subnormal 2^-25, that is 2^-32 of the row's largest,
        which stands for 2^7 at least), over
        a sum of L of them in fp32. An output: a sum of L products, V rounded as K is; then its own rounding."""
        L, n = self.seqs[s]
        q = self.q[self.first[s] + a:self.first[s] + b].double().transpose(0, 1)   # [H, b - a, D]
        k, v = (r[s].repeat_interleave(self.G, 0) for r in (self.k_rows, self.v_rows))
        see = torch.arange(L, device=DEV)[None] <= torch.arange(L - n + a, L - n + b, device=DEV)[:, None]
        x = (q @ k.transpose(1, 2) * self.scale).masked_fill(~see, -math.inf)
        p = x.softmax(-1)
        u, in16 = 2.0 ** -23, 2.0 ** -11 if self.kind == "q4" else 0.0
        tiny = 2.0 ** -25 if self.kind == "q4" else 0.0
        size = (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~see, 0).amax(-1, keepdim=True)
        E = abs(self.scale) * (size * (in16 + (self.D + 6) * u) + tiny * q.abs().sum(-1, keepdim=True)
                               + 2.0 ** -39 * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax(-1)[:, None, None])
        rel = torch.expm1(2 * E) + 2 ** -20 + L * u + 2.0 ** -11
        out, mag = p @ v, p @ v.abs()
        far = 2.0 ** -32 * p.amax(-1, keepdim=True) * v.abs().sum(1, keepdim=True)
        bound = (rel + in16 + L * u) * mag + tiny + far
        half = torch.finfo(self.dtype).eps / 2
        tol = bound + half * (out.abs() + bound) + torch.finfo(self.dtype).smallest_normal * 2 * half
        return out.transpose(0, 1), tol.transpose(0, 1)

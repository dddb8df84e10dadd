"""Layouts and 64-bit references of the bounded-cache operators' GPU tests."""
from __future__ import annotations

import math

import numpy as np
import torch

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


class Cache:
    """Sequences of the given lengths over scattered blocks of two pools. Bytes
    that hold no token are 0xFF (NaN in every type)."""

    def __init__(self, lens, Hkv, G, D, bs, dtype, seed=0, extra_blocks=3, value_scale=1.0):
        self.lens, self.Hkv, self.G, self.D, self.bs, self.H = list(lens), Hkv, G, D, bs, Hkv * G
        self.dtype = TD[dtype]
        self.scale = 1.0 / math.sqrt(D)
        B = len(self.lens)
        self.max_len = max(self.lens)
        MB = max(1, -(-self.max_len // bs)) + 1
        counts = [-(-L // bs) for L in self.lens]
        self.nb = sum(counts) + extra_blocks
        rng = np.random.default_rng(seed)
        perm = rng.permutation(self.nb).astype(np.int32)
        bt = np.full((B, MB), -1, np.int32)
        at = 0
        for s, c in enumerate(counts):
            bt[s, :c] = perm[at:at + c]
            at += c
        self.spare = perm[at:].tolist()
        gen = torch.Generator(device=DEV).manual_seed(seed)
        norm = lambda *sh: (torch.randn(*sh, device=DEV, generator=gen) * value_scale).to(self.dtype)
        self.rows_k = [norm(Hkv, L, D) for L in self.lens]
        self.rows_v = [norm(Hkv, L, D) for L in self.lens]
        self.q = norm(B, self.H, D)
        self.k = self.poisoned()
        self.v = self.poisoned()
        self.bt = bt
        self.tables = torch.from_numpy(bt).to(DEV)
        self.context = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        for s, L in enumerate(self.lens):
            self.put(self.k, s, torch.arange(L), self.rows_k[s])
            self.put(self.v, s, torch.arange(L), self.rows_v[s])

    def poisoned(self):
        n = torch.empty((self.nb, self.Hkv, self.bs, self.D), dtype=self.dtype, device=DEV)
        n.view(torch.uint8).fill_(0xFF)
        return n

    def put(self, pool, s, pos, rows):
        """rows [Hkv, n, D] to the positions pos of sequence s."""
        if len(pos):
            b = torch.from_numpy(self.bt[s][(pos // self.bs).numpy()]).to(DEV).long()
            pool[b, :, (pos % self.bs).to(DEV)] = rows.transpose(0, 1)

    def poison_unseen(self, seen):
        """Overwrite the rows of tokens outside seen(s) (a bool vector) with
        0xFF and forget the blocks that hold no seen token."""
        for s, L in enumerate(self.lens):
            keep = seen(s)
            out = torch.nonzero(~keep).flatten()
            bad = torch.empty((self.Hkv, len(out), self.D), dtype=self.dtype, device=DEV)
            bad.view(torch.uint8).fill_(0xFF)
            self.put(self.k, s, out, bad)
            self.put(self.v, s, out, bad)
            for j in range(-(-L // self.bs)):
                if not keep[j * self.bs:(j + 1) * self.bs].any():
                    self.bt[s, j] = -1 if j % 2 else 1 << 30
        self.tables = torch.from_numpy(self.bt).to(DEV)


def seen_by(L, P, window, sinks):
    """Tokens t < L that a query at position P sees."""
    t = torch.arange(L)
    return (t <= P) & ((t < sinks) | (t > P - window))


def attend(q, k, v, seen, scale, eps_p):
    """64-bit attention of one query row per head: q [H, D], k, v [Hkv, L, D],
    seen [L]. Returns out [H, D], weights [H, L] and a bound of what fp32
    arithmetic may add to each output and, relatively, to each weight.

    A logit is a sum of D products in fp32 (each step off by 2^-23 of the sum of
    absolute products at most, whatever the order), scaled and shifted by the
    maximum (two more roundings of numbers of the logits' size): E bounds its
    error. A weight is an exponential of it (relative error E plus a few 2^-23)
    over a sum of n of them (n roundings); an output is a weighted sum of n
    values, its weights rounded to eps_p relatively when they enter it."""
    H = q.shape[0]
    Hkv, L, D = k.shape
    q, k, v = q.double(), k.double(), v.double()
    k, v = k.repeat_interleave(H // Hkv, 0), v.repeat_interleave(H // Hkv, 0)
    seen = seen.to(q.device)
    k, v = k[:, seen], v[:, seen]
    x = torch.einsum("hd,hld->hl", q, k) * scale
    size = torch.einsum("hd,hld->hl", q.abs(), k.abs()).amax(1, keepdim=True) * abs(scale)
    p = torch.softmax(x, 1)
    n = int(seen.sum())
    u = 2.0 ** -23
    E = (D + 4) * u * size
    rel = 2 * E + (n + 8) * u                       # [H, 1]
    out = torch.einsum("hl,hld->hd", p, v)
    mag = torch.einsum("hl,hld->hd", p, v.abs())
    bound = (rel + eps_p + (n + 8) * u) * mag
    w = torch.zeros(H, L, dtype=torch.float64, device=q.device)
    w[:, seen] = p
    return out, w, bound, rel


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def eps_p(dtype, parts=2):
    """Rounding of a probability on its way into the output's product: none in
    fp32; `parts` 16-bit parts else."""
    return 0.0 if dtype == torch.float32 else half_step(dtype) ** parts


def eps_prefill(dtype):
    """The windowed prefill's probabilities have one 16-bit part."""
    return eps_p(dtype, 1)


def check(got, want, bound, what):
    """|got - want| within the bound plus the rounding to got's type (and its
    subnormals' half step)."""
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    tol = bound + half_step(got.dtype) * (want.abs() + bound) + tiny
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert (err <= tol).all(), f"{what}: off by {(err - tol).max().item():.3e} more than {tol.max().item():.3e}"

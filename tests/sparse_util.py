"""Inputs and tolerances of the tests of rotary positions and block-sparse attention."""
from __future__ import annotations

import numpy as np
import torch

BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def angle_table(rows, rot, base=10000.0):
    """cos_sin float32 [rows, rot]."""
    freq = base ** (-np.arange(rot // 2) / (rot // 2))
    a = np.arange(rows)[:, None] * freq
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32))


def rotary_bound(ref, mag, dtype):
    """x' = fma(x, c, -(y s)): the product is off by half a step of itself (2^-24), the
    fma by half a step of the result, both within 2^-23 of the magnitudes; then one
    rounding to the type.  Results below the least normal number: its step."""
    e = 2.0 ** -23 * mag
    return e + half_step(dtype) * (np.abs(ref) + e) + 2.0 ** -133


def make_cache(seed, lens, hkv, d, bs, dtype, width=None, spare=3, gain=1.0):
    """A paged cache whose requests hold lens tokens: dict of k, v (NaN wherever no
    token is), table, lens, bounds (over the tokens that are there)."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    held = [-(-max(n, 0) // bs) for n in lens]
    nb = sum(held) + spare
    perm = rng.permutation(nb)
    table = np.full((len(lens), width or max(1, max(held, default=1))), -1, dtype=np.int32)
    k = torch.full((nb, bs, hkv, d), float("nan"), dtype=dtype)
    v = torch.full((nb, bs, hkv, d), float("nan"), dtype=dtype)
    bounds = torch.full((nb, hkv, 2, d), float("nan"), dtype=dtype)
    at = 0
    for r, n in enumerate(lens):
        for j in range(held[r]):
            p = int(perm[at])
            at += 1
            table[r, j] = p
            rows = min(bs, n - j * bs)
            k[p, :rows] = (torch.randn(rows, hkv, d, generator=g) * gain).to(dtype)
            v[p, :rows] = torch.randn(rows, hkv, d, generator=g).to(dtype)
            bounds[p, :, 0], bounds[p, :, 1] = k[p, :rows].amin(0), k[p, :rows].amax(0)
    return dict(k=k, v=v, table=torch.from_numpy(table), bounds=bounds, lens=torch.tensor(lens, dtype=torch.int32))


def attend_bound(ref, info, d, dtype):
    """Largest error of pa_sparse, per element of ref [Tq, Hq, D].

    A score is a sum of d exact products in fp32, taken as d / 16 matrix steps and 2 joins
    (bf16) or 4 fmas and 4 or 5 joins (fp32), each off by at most 2^-23 of
    Z = scale sum |q||k| (2^-24 for a rounding), and is scaled once: 16 * 2^-23 Z covers both.
    Its exponent is off by 2^-22 (ex2) and 2^-24 of the argument, at most 3 Z: together
    e = (16 + 2) 2^-23 Z + 2^-22.  Every weight moves by a factor within exp(+-e), the output
    by 2 e A with A = max |v|.  bf16 weights are two bf16 numbers: off by 2^-16.
    Sums over n positions: 2^-23 for each 16 and for each unit's rescaling, and the
    joins of partials, at most 64 one after another (of a warp's two sides, of 4 warps, of 16 CTAs:
    two weights of 2^-22 and three roundings each, A bounds all): (n / 4 + 64 * 6) 2^-23 A.  The result is rounded once."""
    tq, hq, _ = ref.shape
    hkv = info.shape[1]
    z, a, n = (np.repeat(info[:, :, i], hq // hkv, axis=1)[:, :, None] for i in range(3))
    e = (16 + 2) * 2.0 ** -23 * z + 2.0 ** -22
    err = a * (2 * e + (2.0 ** -16 if dtype == BF16 else 0) + (n / 4 + 384) * 2.0 ** -23)
    half = half_step(dtype)
    return err * (1 + half) + half * np.abs(ref) + 2.0 ** -133

"""Inputs and tolerances of the 4-bit pool's tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import q4


def make(seed, lens, hq, hkv, d, bs, dtype, spare=3, k_gain=1.0, v_gain=1.0, shared_blocks=0):
    """A decode case on the CPU: dict of q, pool (uint8 numpy; unowned scales
    NaN), table, lens, k_new, v_new.  The first `shared_blocks` blocks of every
    sequence are the same physical blocks."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    b = len(lens)
    held = [n // bs + 1 for n in lens]
    nb = sum(held) + spare
    perm = rng.permutation(nb)
    table = np.full((b, max(held) + 1), -1, dtype=np.int32)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = perm[at:at + h]
        at += h
        m = min(shared_blocks, lens[i] // bs)
        table[i, :m] = table[0, :m]
    pool = rng.integers(0, 256, (nb, hkv, q4.record_bytes(d, bs)), dtype=np.uint8)
    pool[:, :, bs * d:] = 255  # NaN scales wherever nothing is stored
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    # stored rows: random codes and the scales of normal data
    for i, n in enumerate(lens):
        for j in range(held[i]):
            rows = min(bs, n - j * bs)
            if rows <= 0:
                continue
            x = np.stack([k_gain * (rand(hkv, rows).numpy() * 0.02 + 0.3), k_gain * (rand(hkv, rows).numpy() * 0.2 - 2.2),
                          v_gain * (rand(hkv, rows).numpy() * 0.02 + 0.3), v_gain * (rand(hkv, rows).numpy() * 0.4 - 2.2)],
                         -1).astype(np.float32)
            bits = (np.ascontiguousarray(x).view(np.uint32) >> 16).astype("<u2")
            pool[table[i, j], :, bs * d:bs * d + 8 * rows] = bits.reshape(hkv, -1).view(np.uint8)
    return dict(q=rand(b, hq, d).to(dtype), pool=pool, table=table, lens=np.array(lens, dtype=np.int32),
                k_new=(rand(b, hkv, d) * k_gain).to(dtype), v_new=(rand(b, hkv, d) * v_gain).to(dtype), bs=bs)


def decode_bound(q, seen, ref, dtype, scale):
    """Largest error the kernel's arithmetic allows, per element of ref [B, Hq, D].

    out = sum_j p_j (b_j + s_j n_j) with p the softmax of the scores x_j, and
    x_j = scale (s_j q.n_j + b_j sum q).
      * scores: the operands are exact (the codes, and q as one or two f16
        numbers up to 2^-22 of its largest element); q.n is D / 16 matrix
        steps, sum q is 5 shuffles and the lane's own sum, and 8 further
        operations follow, each off by at most 2^-23 of
        Z = max_j scale (|b_j| + 15 s_j) sum |q_i|: (D / 8 + 16) 2^-23 Z in all.
        ex2 is off by 2^-22 and its argument, |x| log2(e) <= 1.5 Z large, by
        2^-24 of itself: together e.  Each p_j moves by a factor within
        exp(+-2 e), so the output by 2 e A, A = max_j (|b_j| + 15 s_j) of V.
      * weights p s go to the tensor cores as f16 (half a step is 2^-11) or as
        a sum of two (2^-21), and are multiplied by n <= 15: that much of A.
      * sums over T tokens in fp32: a cut of 2^-23 for each 16 tokens, at most
        one rounding for each 16 more and 64 for the joins, each of at most A.
      * the result is rounded once, half a step: 2^-8 or 2^-24 of it.
    """
    b, hq, d = ref.shape
    bound = np.zeros_like(ref)
    qa = np.abs(q.double().numpy())
    bf16 = dtype == torch.bfloat16
    for i, (k, v, km, vm) in enumerate(seen):
        t, hkv, _ = k.shape
        z = scale * qa[i].sum(-1).reshape(hkv, -1) * km.max(0)[:, None]
        e = (d / 8 + 16) * 2.0 ** -23 * z + 2.0 ** -22 + 1.5 * z * 2.0 ** -24
        a = vm.max(0)[:, None]
        err = a * (2 * e + (2.0 ** -11 if bf16 else 2.0 ** -21) + (t / 8 + 64) * 2.0 ** -23)
        bound[i] = np.broadcast_to(err.reshape(-1)[:, None], (hq, d))
    half = 2.0 ** -8 if bf16 else 2.0 ** -24
    return bound * (1 + half) + half * np.abs(ref)


def check(got, ref, bound, what="", norm=None):
    """Every element within its bound; and, where `norm` is given, the 2-norm
    of the difference within that part of the result's (the bound is for the
    worst case, roundings that do not line up stay far below it)."""
    g = got.detach().double().cpu().numpy()
    assert np.isfinite(g).all(), f"{what}: not finite"
    off = np.abs(g - ref) - bound
    if (off > 0).any():
        at = np.unravel_index(off.argmax(), off.shape)
        raise AssertionError(f"{what}: {int((off > 0).sum())} of {off.size} outside; at {at} got {g[at]} for "
                             f"{ref[at]}, allowed {bound[at]}")
    # an output of zeros must not pass
    assert (np.abs(ref) > bound).any(), f"{what}: the bound is too wide to tell anything"
    if norm is not None:
        rel = np.linalg.norm(g - ref) / np.linalg.norm(ref)
        assert rel <= norm, f"{what}: 2-norm of the difference {rel:.3g}, allowed {norm:.3g}"


# 2-norms: a bf16 result is off by its own rounding, at most half a step (2^-8)
# of every element; for fp32 the library's own tolerance.
NORM = {torch.bfloat16: 2.0 ** -8, torch.float32: 1e-5}


def write_rows(pool, slots, k, v, bs):
    """oracle.q4.write for many tokens at once: rows k, v [T, Hkv, D] into the
    slots (in place; negative ones are skipped)."""
    t = np.flatnonzero(slots >= 0)
    blk, off = (slots[t] // bs)[:, None, None], slots[t] % bs
    h, d = np.arange(k.shape[1])[None, :, None], k.shape[2]
    for kv, x in enumerate((k, v)):
        n, s, b = q4.quantise(x[t])
        if kv == 0:
            pool[blk, h, (off[:, None] * (d // 2) + np.arange(d // 2))[:, None]] = n[..., 0::2] | n[..., 1::2] << 4
        else:
            at = bs * d // 2 + 2 * q4.v_unit(off[:, None], np.arange(d // 4)[None], d)[:, None]
            pool[blk, h, at] = n[..., 0::4] | n[..., 1::4] << 4
            pool[blk, h, at + 1] = n[..., 2::4] | n[..., 3::4] << 4
        scale = np.stack([s & 255, s >> 8, b & 255, b >> 8], -1).astype(np.uint8)
        pool[blk, h, (bs * d + 8 * off[:, None] + 4 * kv + np.arange(4))[:, None]] = scale


def edge_rows(dtype):
    """Finite rows with their largest element at the end of the numbers, and
    their smallest from the same to its opposite."""
    top = torch.finfo(dtype).max
    if dtype == torch.float32:
        tops = [top, 3.3895e38, 3.3896e38, 3.396e38, 3.4e38, 3.3e38, 3.35e38, 3.38e38]
    else:
        tops = [top, 3.3e38, 3.34e38, 3.36e38, 3.38e38]
    g = torch.Generator().manual_seed(1)
    rows = []
    for hi in tops:
        for low in (1.0, 0.999, 0.99, 17 / 32, 0.9, 0.5, 0.3, 0.05, 0.01, 0.0, -0.05, -0.7, -0.99):
            x = hi * (low + (1 - low) * torch.rand(64, generator=g, dtype=torch.float64))
            x[:2] = torch.tensor([hi * low, hi], dtype=torch.float64)
            rows.append(x.clamp(-3.385e38, top).to(dtype))
    return torch.stack(rows)

"""Plain reference of the 4-bit paged pool and of the step's block tables
(test infrastructure; shares no code with the library).

The format is the one include/pa.h states under "The 4-bit pool".  Which code
a value takes is defined by fp32 steps, so those are taken in float32 here
too; everything after it (values, attention) is float64.
"""
from __future__ import annotations

import numpy as np


BF16_MAX = (2 - 2.0 ** -7) * 2.0 ** 127


def bf16_bits_to_f64(bits):
    return (np.asarray(bits, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _step_bits(x):
    """bits of float32 x with the low 16 bits rounded away from zero."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u.astype(np.uint64) + 0xFFFF) & 0xFFFF0000).astype(np.uint32)


def quantise(x):
    """x float32 [..., D] -> codes uint8 [..., D], step bits, low bits (uint16 [...])."""
    x = np.asarray(x, dtype=np.float32)
    f = np.float32
    finite = np.isfinite(x).all(-1)
    safe = np.where(finite[..., None], x, f(0))
    hi, lo = safe.max(-1), safe.min(-1)
    lo_bits = np.ascontiguousarray(lo).view(np.uint32)
    low_bits = np.where(lo < 0, _step_bits(lo), lo_bits & np.uint32(0xFFFF0000)).astype(np.uint32)
    low = low_bits.view(f)
    finite &= np.isfinite(low)
    with np.errstate(over="ignore", invalid="ignore"):
        r = (hi * f(0.0625) - low * f(0.0625)) * f(16.0 / 15.0)
        step_bits = np.where(r < f(2.0 ** -100), np.uint32(0), _step_bits(r)).astype(np.uint32)
        for _ in range(2):  # a top value that would read back as an infinity
            top = (15 * step_bits.view(f).astype(np.float64) + low).astype(f)
            step_bits = np.where(finite & (top > f(BF16_MAX)), step_bits - np.uint32(0x10000), step_bits)
        step = step_bits.view(f)
        some = finite & (step > 0)
        inv = f(16) / np.where(some, step, f(1))
        n = np.rint((safe * f(0.0625) - (low * f(0.0625))[..., None]) * inv[..., None])
    n = np.where(some[..., None], np.clip(n, 0, 15), 0).astype(np.uint8)
    nan = np.uint16(0x7FC0)
    return (n, np.where(finite, (step_bits >> 16).astype(np.uint16), nan),
            np.where(finite, (low_bits >> 16).astype(np.uint16), nan))


def values(n, step_bits, low_bits):
    """What codes stand for, float64."""
    return bf16_bits_to_f64(low_bits)[..., None] + n * bf16_bits_to_f64(step_bits)[..., None]


def record_bytes(d, bs):
    return bs * (d + 8)


def v_unit(t, x, d):
    """Number of the 16-bit unit of V's dims 4x..4x+3 of token t."""
    p = t // 2
    u = (x // 8) ^ (p % 4 if d == 128 else p // 2 % 2)
    return 2 * (p * (d // 4) + 8 * u + x % 8) + t % 2


def write(pool, slot, k, v, bs):
    """Quantise one token's K and V rows [Hkv, D] into the slot (in place)."""
    hkv, d = k.shape
    rec = pool[slot // bs]
    t = slot % bs
    for kv, x in enumerate((k, v)):
        n, s, b = quantise(x)
        for h in range(hkv):
            if kv == 0:
                rec[h, t * d // 2:(t + 1) * d // 2] = n[h, 0::2] | (n[h, 1::2] << 4)
            else:
                for u in range(d // 4):
                    c = n[h, 4 * u:4 * u + 4].astype(np.int64)
                    w = int(c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12)
                    at = bs * d // 2 + 2 * v_unit(t, u, d)
                    rec[h, at], rec[h, at + 1] = w & 255, w >> 8
            at = bs * d + 8 * t + 4 * kv
            rec[h, at:at + 4] = np.array([s[h], b[h]], dtype="<u2").view(np.uint8)


def read(pool, table_row, n, d, bs):
    """K and V float64 [n, Hkv, D] of positions 0..n-1 of one request, and the
    largest magnitudes |low| + 15 step of their rows, [n, Hkv] each."""
    hkv = pool.shape[1]
    t, i = np.arange(bs)[:, None], np.arange(d)[None, :]
    unit = v_unit(t, i // 4, d)
    ks, vs, km, vm = [], [], [], []
    for j in range(-(-n // bs)):
        rec = pool[table_row[j]]
        kn = (rec[:, t * (d // 2) + i // 2] >> (4 * (i % 2))) & 15
        vn = (rec[:, bs * d // 2 + 2 * unit + i % 4 // 2] >> (4 * (i % 2))) & 15
        sc = np.ascontiguousarray(rec[:, bs * d:]).view("<u2").reshape(hkv, bs, 4)
        with np.errstate(invalid="ignore"):
            ks.append(values(kn, sc[..., 0], sc[..., 1]))
            vs.append(values(vn, sc[..., 2], sc[..., 3]))
        sc = np.abs(bf16_bits_to_f64(sc))
        km.append(sc[..., 1] + 15 * sc[..., 0])
        vm.append(sc[..., 3] + 15 * sc[..., 2])
    if not ks:
        return (np.zeros((0, hkv, d)),) * 2 + (np.zeros((0, hkv)),) * 2
    join = lambda x: np.concatenate(x, 1).swapaxes(0, 1)[:n]  # noqa: E731
    return join(ks), join(vs), join(km), join(vm)


def decode(q, pool, table, lens, k_new, v_new, bs, scale=None):
    """One decode step: appends in place, returns (out float64, seen) with
    seen the read() of every sequence.  q, k_new, v_new float32."""
    b, hq, d = q.shape
    hkv = k_new.shape[1]
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((b, hq, d))
    seen = []
    for i in range(b):
        n = int(lens[i])
        write(pool, int(table[i, n // bs]) * bs + n % bs, k_new[i], v_new[i], bs)
    for i in range(b):
        seen.append(read(pool, table[i], int(lens[i]) + 1, d, bs))
        k, v = seen[-1][:2]
        qq = q[i].astype(np.float64).reshape(hkv, hq // hkv, d)
        w = np.einsum("hgd,thd->hgt", qq, k) * scale
        p = np.exp(w - w.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[i] = np.einsum("hgt,thd->hgd", p, v).reshape(hq, d)
    return out, seen


def block_tables(lens, new, table, free, num_free, total_slots, bs):
    """The step that include/pa.h states for pa_block_tables, request by
    request.  Returns (table, free, num_free, slot_map, cu_q, cu_k, lens) as
    copies, or None where the step is refused."""
    table, free = table.copy(), free.copy()
    nb, mb = len(free), table.shape[1]
    stack = [int(x) for x in free[:num_free]]
    held = [-(-int(n) // bs) for n in lens]
    for n, m in zip(lens, new):
        if n < 0 or m < -1 or n + max(m, 0) > mb * bs:
            return None
    for b, m in enumerate(new):
        if m < 0:
            stack += [int(x) if 0 <= x < nb else -1 for x in table[b, :held[b]]]
    if len(stack) > nb:
        return None
    free[:len(stack)] = stack
    slots, cu_q, cu_k, after = [], [0], [0], []
    for b, (n, m) in enumerate(zip(lens, new)):
        n, m = int(n), int(m)
        for j in range(held[b], -(-(n + m) // bs) if m >= 0 else 0):
            if not stack:
                return None
            p = stack.pop()
            table[b, j] = p if 0 <= p < nb else -1
        for pos in range(n, n + max(m, 0)):
            p = int(table[b, pos // bs])
            slots.append(p * bs + pos % bs if 0 <= p < nb else -1)
        after.append(0 if m < 0 else n + m)
        cu_q.append(cu_q[-1] + max(m, 0))
        cu_k.append(cu_k[-1] + after[-1])
    if len(slots) > total_slots:
        return None
    slots += [-1] * (total_slots - len(slots))
    i32 = lambda x: np.array(x, dtype=np.int32)  # noqa: E731
    return table, free, len(stack), i32(slots), i32(cu_q), i32(cu_k), i32(after)

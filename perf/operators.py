"""Timed cases of the 4-bit paged cache and of the GPU-built block tables.

Four operators, reached through the package's public calls:

* ``tables``  pa_block_tables: one serving step's block tables, slot map and
  cumulative lengths from the requests' lengths;
* ``store``   pa_cache_update_q4 followed by pa_cache_gather_q4: a prefill
  chunk is quantised into the pool and every request's whole key sequence is
  read back for the varlen attention;
* ``gather``  pa_cache_gather_q4 alone: cached sequences read back;
* ``decode``  pa_decode_q4: one token per sequence appended and attended.

The 4-bit pool is uint8 [num_blocks, num_kv_heads, block_size * (D + 8)]; one
record (one head of one block) holds

    K codes   [block_size][D / 2]            dim 2i in the low nibble of byte i
    V codes   block_size * D / 2 bytes       16-bit units of 4 dims, two tokens
                                             interleaved (see _v_map)
    scales    [block_size][4] bf16           K step, K low, V step, V low

and a value is low + code * step.
"""
import torch

own = False

_GOLD = 0.6180339887498949


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a busy server: every request adds one token
        dict(name="tables_decode_256", op="tables", batch=256, lo=64, hi=8192, new_lo=1, new_hi=1, end_every=0, bs=16),
        # a single chat: the smallest call there is
        dict(name="tables_single", op="tables", batch=1, lo=1000, hi=1000, new_lo=1, new_hi=1, end_every=0, bs=32),
        # a full queue: prompts, decode steps and finished requests in one step
        dict(name="tables_mixed_4096", op="tables", batch=4096, lo=0, hi=2048, new_lo=0, new_hi=250, end_every=7, bs=16),
        # prefill chunks after cached prefixes, read back for the varlen attention
        dict(name="store_prefill_bf16", op="store", batch=32, lo=0, hi=1024, new_lo=1, new_hi=2048, hkv=8, d=128, bs=16, dtype="bf16"),
        # a few short prompts of a small fp32 model
        dict(name="store_small_f32", op="store", batch=3, lo=0, hi=70, new_lo=5, new_hi=37, hkv=2, d=64, bs=32, dtype="f32"),
        # long cached prefixes pulled out of the 4-bit pool
        dict(name="gather_long_bf16", op="gather", batch=16, lo=2000, hi=16000, hkv=8, d=128, bs=16, dtype="bf16"),
        # many small-head sequences, odd lengths, fp32
        dict(name="gather_f32", op="gather", batch=61, lo=1, hi=777, hkv=6, d=64, bs=32, dtype="f32"),
        # the block-table example of the documentation: three short sequences
        dict(name="decode_tiny_f32", op="decode", batch=3, lo=30, hi=70, hq=4, hkv=2, d=64, bs=32, dtype="f32"),
        # one conversation: latency of a single token
        dict(name="decode_single_bf16", op="decode", batch=1, lo=5000, hi=5000, hq=32, hkv=8, d=128, bs=16, dtype="bf16"),
        # the repository's decode workload: 64 sequences, grouped heads
        dict(name="decode_gqa_bf16", op="decode", batch=64, lo=512, hi=4096, hq=32, hkv=8, d=128, bs=16, dtype="bf16"),
        # many short sequences, one query head per kv head
        dict(name="decode_mha64_bf16", op="decode", batch=1024, lo=257, hi=768, hq=32, hkv=32, d=64, bs=32, dtype="bf16"),
        # long contexts with 8 query heads to a kv head
        dict(name="decode_long_bf16", op="decode", batch=96, lo=4096, hi=16384, hq=64, hkv=8, d=128, bs=16, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["tables", "store", "gather", "decode", "decode"])
    bs = rng.choice([16, 32])
    if op == "tables":
        batch = _log_int(rng, 1, 4096)
        hi = _log_int(rng, 1, 8192)
        room = max(1, min(2048, 500000 // batch))
        new_hi = rng.choice([1, _log_int(rng, 1, room)])
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, new_lo=rng.randint(0, 1), new_hi=new_hi,
                    end_every=rng.choice([0, 0, 5, 9]), bs=bs)
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = {"decode": 1000e6, "gather": 110e6, "store": 40e6}[op]  # elements of K
    budget = _log_int(rng, 2000, int(most) // (d * hkv))  # tokens
    batch = min(_log_int(rng, 1, 512), budget)
    hi = min(16384, max(1, budget // batch))
    c = dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, hkv=hkv, d=d, bs=bs, dtype=dtype)
    if op == "store":
        c["new_lo"], c["new_hi"] = 1, _log_int(rng, 1, min(4096, hi + 1))
    if op == "decode":
        c["hq"] = hkv * rng.choice([1, 2, 3, 4, 7, 8])
    return c


def _spread(n, lo, hi, shift=0.0):
    """n whole numbers spread evenly over lo..hi, the same for every seed."""
    return [lo + int((hi - lo + 1) * (((i + 1) * _GOLD + shift) % 1.0)) for i in range(n)]


def _lens(case):
    cached = _spread(case["batch"], case["lo"], case["hi"])
    new = _spread(case["batch"], case["new_lo"], case["new_hi"], 0.37) if "new_lo" in case else [1] * case["batch"]
    every = case.get("end_every", 0)
    if every:
        new = [-1 if i % every == every - 1 else n for i, n in enumerate(new)]
    return cached, new


def _blocks(n, bs):
    return -(-n // bs)


def work(case):
    cached, new = _lens(case)
    bs = case["bs"]
    if case["op"] == "tables":
        tokens = sum(max(n, 0) for n in new)
        fresh = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in zip(cached, new) if n > 0)
        back = sum(_blocks(c, bs) for c, n in zip(cached, new) if n < 0)
        return {"bytes": 4.0 * (5 * case["batch"] + tokens + 2 * fresh + 2 * back), "flops": 0}
    d, hkv = case["d"], case["hkv"]
    e = 2 if case["dtype"] == "bf16" else 4
    row4, row = hkv * (d + 8), hkv * d * e
    if case["op"] == "decode":
        pos = sum(c + 1 for c in cached)
        entries = sum(_blocks(c + 1, bs) for c in cached)
        hq = case["hq"]
        return {"bytes": float(pos * row4 + 4 * entries + case["batch"] * (2 * hq * d * e + 4 * row + 8)),
                "flops": 4.0 * pos * hq * d}
    chunk = sum(new) if case["op"] == "store" else 0
    total = sum(cached) + chunk
    entries = sum(_blocks(c + (n if case["op"] == "store" else 0), bs) for c, n in zip(cached, new))
    # the chunk is read and stored once, then every row is read back and written out
    return {"bytes": float(2 * chunk * row + chunk * (row4 + 4) + total * row4 + 2 * total * row + 4 * entries), "flops": 0}


# ------------------------------------------------------------------ plain forms
def _up(x):
    """fp32 -> bf16, away from zero."""
    return ((x.view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32).to(torch.bfloat16)


def _down(x):
    """fp32 -> bf16, towards minus infinity."""
    cut = (x.view(torch.int32) & -0x10000).view(torch.float32).to(torch.bfloat16)
    return torch.where(x < 0, _up(x), cut)


def _quantise(x):
    """codes uint8 [.., D], step and low bf16 [..] of fp32 rows."""
    hi, lo = x.amax(-1), x.amin(-1)
    low = _down(lo)
    good = torch.isfinite(hi) & torch.isfinite(low.float())
    r = (hi * 0.0625 - low.float() * 0.0625) * (16.0 / 15.0)
    step = torch.where(r < 2.0 ** -100, torch.zeros_like(r).to(torch.bfloat16), _up(r))
    some = (step > 0) & good
    inv = 16.0 * (1.0 / torch.where(some, step.float(), torch.ones_like(r)))
    n = ((x * 0.0625 - (low.float() * 0.0625).unsqueeze(-1)) * inv.unsqueeze(-1)).round().clamp(0, 15)
    n = torch.where(some.unsqueeze(-1), n, torch.zeros_like(n)).to(torch.uint8)
    bad = torch.full_like(step, float("nan"))
    return n, torch.where(good, step, bad), torch.where(good, low, bad)


def _v_map(bs, d, device):
    """Place of the 16-bit unit (token t, dims 4x..4x+3) inside a record's V
    codes: tokens 2p and 2p + 1 share a 32-bit word, and the 32-byte parts of
    a pair's row are permuted by the pair's number."""
    t = torch.arange(bs, device=device).unsqueeze(1)
    x = torch.arange(d // 4, device=device).unsqueeze(0)
    p = t // 2
    part = (x // 8) ^ ((p if d == 128 else p // 2) % (d // 32))
    return 2 * (p * (d // 4) + part * 8 + x % 8) + t % 2


def _put(pool, bs, slots, k, v):
    """Quantise rows k, v [T, Hkv, D] into the slots [T] of the pool."""
    d, hkv = k.shape[2], k.shape[1]
    kc, ks, kl = _quantise(k.float())
    vc, vs, vl = _quantise(v.float())
    block, off = (slots // bs).long().view(-1, 1, 1), (slots % bs).long()
    head = torch.arange(hkv, device=pool.device).view(1, -1, 1)
    row = torch.arange(d // 2, device=pool.device).view(1, 1, -1)
    pool[block, head, off.view(-1, 1, 1) * (d // 2) + row] = kc[..., 0::2] | (kc[..., 1::2] << 4)
    v4 = vc.view(*vc.shape[:2], d // 4, 4).to(torch.int32)
    v4 = v4[..., 0] | (v4[..., 1] << 4) | (v4[..., 2] << 8) | (v4[..., 3] << 12)
    half = pool.view(torch.int16)
    half[block, head, bs * d // 4 + _v_map(bs, d, pool.device)[off].unsqueeze(1)] = v4.to(torch.int16)
    par = torch.stack([ks, kl, vs, vl], -1).view(torch.int16)
    half[block, head, bs * d // 2 + off.view(-1, 1, 1) * 4 + torch.arange(4, device=pool.device)] = par


def _values(rec, bs, d):
    """fp32 K and V [.., bs, D] of records [.., bs * (D + 8)]."""
    lead = rec.shape[:-1]
    par = rec[..., bs * d:].contiguous().view(torch.bfloat16).view(*lead, bs, 4).float()
    kb = rec[..., : bs * d // 2].reshape(*lead, bs, d // 2)
    k = torch.stack([kb & 15, kb >> 4], -1).view(*lead, bs, d).float()
    k = k.mul_(par[..., 0:1]).add_(par[..., 1:2])
    vb = rec[..., bs * d // 2 : bs * d].contiguous().view(torch.int16)[..., _v_map(bs, d, rec.device)].to(torch.int32)
    v = torch.stack([vb & 15, (vb >> 4) & 15, (vb >> 8) & 15, (vb >> 12) & 15], -1).view(*lead, bs, d).float()
    return k, v.mul_(par[..., 2:3]).add_(par[..., 3:4])


def _rows(lens, total):
    """(request, position in it) of each of `total` packed rows."""
    start = torch.cumsum(lens, 0) - lens
    req = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens, output_size=total)
    return req, torch.arange(total, device=lens.device) - start[req]


def _plain_tables(s):
    bs = s["bs"]
    old, new = s["cached"].long(), s["new"].long()
    ended = new < 0
    held = (old + bs - 1) // bs
    tok = new.clamp(min=0)
    back = torch.where(ended, held, 0)
    take = torch.where(ended, 0, (old + tok + bs - 1) // bs - held)
    after = torch.where(ended, 0, old + tok)
    zero = torch.zeros(1, dtype=torch.int64, device=old.device)
    cu_q = torch.cat([zero, tok.cumsum(0)]).int()
    cu_k = torch.cat([zero, after.cumsum(0)]).int()
    free, table = s["free"], s["table"]
    req, j = _rows(back, s["n_back"])
    free[s["count"] + torch.arange(s["n_back"], device=old.device)] = table[req, j]
    top = s["count"].long() + s["n_back"]
    req, j = _rows(take, s["n_take"])
    table[req, held[req] + j] = free[top - 1 - torch.arange(s["n_take"], device=old.device)]
    req, j = _rows(tok, s["n_tok"])
    pos = old[req] + j
    s["slots"].fill_(-1)
    s["slots"][: s["n_tok"]] = table[req, pos // bs] * bs + (pos % bs).int()
    return dict(table=table, free=free, count=(top - s["n_take"]).int(), slots=s["slots"], cu_q=cu_q, cu_k=cu_k,
                lens=after.int())


def _plain_gather(s):
    bs, d, pool = s["bs"], s["d"], s["pool"]
    req, pos = _rows(s["cu_k"][1:].long() - s["cu_k"][:-1].long(), s["total"])
    block, off = s["table"][req, pos // bs].long().view(-1, 1, 1), (pos % bs).view(-1, 1, 1)
    head = torch.arange(pool.shape[1], device=pool.device).view(1, -1, 1)
    half = pool.view(torch.int16)
    lane = torch.arange(d // 2, device=pool.device)
    kb = pool[block, head, off * (d // 2) + lane]
    vb = half[block, head, bs * d // 4 + _v_map(bs, d, pool.device)[off.view(-1)].unsqueeze(1)].to(torch.int32)
    par = half[block, head, bs * d // 2 + off * 4 + lane[:4]].view(torch.bfloat16).float()
    k = torch.stack([kb & 15, kb >> 4], -1).view(*kb.shape[:2], d).float()
    v = torch.stack([vb & 15, (vb >> 4) & 15, (vb >> 8) & 15, (vb >> 12) & 15], -1).view(*kb.shape[:2], d).float()
    k = k.mul_(par[..., 0:1]).add_(par[..., 1:2]).to(s["dtype"])
    return dict(k=k, v=v.mul_(par[..., 2:3]).add_(par[..., 3:4]).to(s["dtype"]))


def _plain_decode(s):
    bs, d, pool, table = s["bs"], s["d"], s["pool"], s["table"]
    b, hq, hkv = s["q"].shape[0], s["q"].shape[1], pool.shape[1]
    old = s["cached"].long()
    mine = torch.arange(b, device=pool.device)
    slot = table[mine, old // bs].long() * bs + old % bs
    _put(pool, bs, slot, s["k_new"], s["v_new"])
    k, v = _values(pool[table.clamp(min=0).long()], bs, d)  # [B, blocks, Hkv, bs, D]
    k, v = (x.transpose(1, 2).reshape(b, hkv, -1, d) for x in (k, v))
    seen = (torch.arange(k.shape[2], device=pool.device) <= old.unsqueeze(1)).view(b, 1, 1, -1)
    v = torch.where(seen.view(b, 1, -1, 1), v, 0.0)
    score = (s["q"].float().view(b, hkv, hq // hkv, d) @ k.transpose(2, 3)) * (d ** -0.5)
    score = torch.where(seen, score, -float("inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = (p @ v) / p.sum(-1, keepdim=True)
    at = old.view(b, 1, 1, 1).expand(b, hkv, 1, d)
    return dict(out=out.view(b, hq, d).to(s["dtype"]), k_stored=k.gather(2, at)[:, :, 0].to(s["dtype"]),
                v_stored=v.gather(2, at)[:, :, 0].to(s["dtype"]))


# ------------------------------------------------------------------ inputs
def _filled_pool(g, dev, lens, room, case, extra):
    """A pool whose requests hold `lens` cached tokens and own blocks for
    `room` tokens each; unused scales are NaN, as uninitialised memory may be.
    Returns (pool, table)."""
    bs, d, hkv = case["bs"], case["d"], case["hkv"]
    held = [_blocks(n, bs) for n in room]
    nb = sum(held) + extra
    perm = torch.randperm(nb, generator=g, device=dev)
    table = torch.full((len(lens), max(1, max(held))), -1, dtype=torch.int32, device=dev)
    counts = torch.tensor(held, device=dev)
    req, j = _rows(counts, sum(held))
    table[req, j] = perm[: sum(held)].int()
    pool = torch.full((nb, hkv, bs * (d + 8)), 255, dtype=torch.uint8, device=dev)
    cached = torch.tensor(lens, device=dev)
    req, pos = _rows(cached, sum(lens))
    slots = table[req, pos // bs].long() * bs + pos % bs
    gain = torch.exp(0.4 * torch.randn(hkv, d, generator=g, device=dev))  # keys have strong and weak channels
    k, v = (torch.randn(len(slots), hkv, d, generator=g, device=dev) for _ in range(2))
    _put(pool, bs, slots, k.mul_(gain), v)
    return pool, table


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    cached, new = _lens(case)
    bs, b = case["bs"], case["batch"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] == "tables":
        held = [_blocks(c, bs) for c in cached]
        take = [_blocks(c + n, bs) - h if n >= 0 else 0 for c, n, h in zip(cached, new, held)]
        back = sum(h for h, n in zip(held, new) if n < 0)
        wide = max(h + t for h, t in zip(held, take)) + 1
        spare = sum(take) + 64 + b // 8
        nb = sum(held) + spare
        perm = torch.randperm(nb, generator=g, device=dev).int()
        table = torch.full((b, wide), -1, dtype=torch.int32, device=dev)
        req, j = _rows(torch.tensor(held, device=dev), sum(held))
        table[req, j] = perm[: sum(held)]
        free = torch.full((nb,), -1, dtype=torch.int32, device=dev)
        free[:spare] = perm[sum(held):]
        tok = sum(max(n, 0) for n in new)
        slots = torch.empty(tok + 3, dtype=torch.int32, device=dev)
        outs = dict(cu_q=i32([0] * (b + 1)), cu_k=i32([0] * (b + 1)), lens=i32([0] * b), left=i32([0]))
        return dict(op="tables", cached=i32(cached), new=i32(new), table=table, free=free, count=i32([spare]),
                    slots=slots, bs=bs, n_back=back, n_take=sum(take), n_tok=tok, **outs)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    d, hkv = case["d"], case["hkv"]
    more = [1] * b if case["op"] == "decode" else new if case["op"] == "store" else [0] * b
    pool, table = _filled_pool(g, dev, cached, [c + n for c, n in zip(cached, more)], case, 1 + b // 4)
    rand = lambda *sh: torch.randn(*sh, generator=g, device=dev).to(dtype)  # noqa: E731
    s = dict(op=case["op"], pool=pool, table=table, bs=bs, d=d, dtype=dtype, cached=i32(cached))
    if case["op"] == "decode":
        s.update(q=rand(b, case["hq"], d), k_new=rand(b, hkv, d), v_new=rand(b, hkv, d))
        s.update(out=torch.empty_like(s["q"]), k_stored=torch.empty_like(s["k_new"]), v_stored=torch.empty_like(s["k_new"]))
        return s
    total = sum(cached) + sum(more)
    ends = torch.tensor([c + n for c, n in zip(cached, more)], device=dev).cumsum(0)
    s.update(total=total, cu_k=torch.cat([torch.zeros_like(ends[:1]), ends]).int())
    s.update(k_full=torch.empty(total, hkv, d, dtype=dtype, device=dev), v_full=torch.empty(total, hkv, d, dtype=dtype, device=dev))
    if case["op"] == "store":
        req, j = _rows(torch.tensor(new, device=dev), sum(new))
        pos = s["cached"][req] + j
        s.update(slots=(table[req, pos // bs] * bs + pos % bs).int(), k=rand(sum(new), hkv, d), v=rand(sum(new), hkv, d))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import paged_kv_cache_300_gb300 as pa

        if s["op"] == "tables":
            pa.pa_block_tables(s["cached"], s["new"], s["table"], s["free"], s["count"], s["slots"], s["bs"],
                               cu_seq_lens_q=s["cu_q"], cu_seq_lens_k=s["cu_k"], seqlens_k=s["lens"],
                               num_free_out=s["left"])
            return dict(table=s["table"], free=s["free"], count=s["left"], slots=s["slots"], cu_q=s["cu_q"],
                        cu_k=s["cu_k"], lens=s["lens"])
        if s["op"] == "decode":
            pa.pa_decode_q4(s["q"], s["pool"], s["table"], s["cached"], s["k_new"], s["v_new"], s["out"],
                            k_stored=s["k_stored"], v_stored=s["v_stored"])
            return dict(out=s["out"], k_stored=s["k_stored"], v_stored=s["v_stored"])
        if s["op"] == "store":
            pa.pa_cache_update_q4(s["k"], s["v"], s["slots"], s["pool"])
        pa.pa_cache_gather_q4(s["pool"], s["table"], s["cu_k"], s["k_full"], s["v_full"])
        return dict(k=s["k_full"], v=s["v_full"])
    if s["op"] == "tables":
        return _plain_tables(s)
    if s["op"] == "decode":
        return _plain_decode(s)
    if s["op"] == "store":
        _put(s["pool"], s["bs"], s["slots"], s["k"], s["v"])
    return _plain_gather(s)


# ------------------------------------------------------------------ in 64 bits
def _bf16_ulp(x):
    """The distance of bf16 numbers at |x|, a power of two in 64 bits (put
    together from its exponent: pow() is not exact on the GPU)."""
    return ((torch.frexp(x).exponent.long() - 8 + 1023) << 52).view(torch.float64)


def _exact_row(x):
    """The stored values of rows, in 64 bits.  Which code a value takes is
    part of the format and defined in fp32 steps; the rest is exact."""
    x = x.float()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    low = lo.bfloat16().double()
    ulp = _bf16_ulp(lo)
    low = torch.where(low > lo.double(), low - ulp, low)
    f = torch.float32
    r = ((hi / 16 - low.to(f) / 16) * torch.tensor(16.0 / 15.0, dtype=f)).double()
    up = _bf16_ulp(r)
    step = torch.where(r < 2.0 ** -100, 0.0, torch.ceil(r / up) * up)
    inv = (16.0 / torch.where(step > 0, step, 1.0)).to(f)
    n = torch.round((x / 16 - low.to(f) / 16) * inv).double().clamp(0, 15)
    return low + torch.where(step > 0, n, 0.0) * step


def _exact_read(pool, table, b, n, bs, d):
    """K and V [n, Hkv, D] of positions 0..n-1 of request b, in 64 bits."""
    rec = pool[table[b, : _blocks(n, bs)].long()].long()
    hkv = rec.shape[1]
    t, i = torch.arange(bs, device=pool.device).view(-1, 1), torch.arange(d, device=pool.device).view(1, -1)
    k = (rec[:, :, t * (d // 2) + i // 2] >> (4 * (i % 2))) & 15
    # byte of V's dim i of token t: word of the token pair, low or high half, byte of the half
    pair = t // 2
    part = (i // 32) ^ (pair % 4 if d == 128 else pair // 2 % 2)
    byte = bs * d // 2 + pair * d + part * 32 + (i % 32) // 4 * 4 + (t % 2) * 2 + (i % 4) // 2
    v = (rec[:, :, byte] >> (4 * (i % 2))) & 15

    def par(c):
        at = bs * d + t[:, 0] * 8 + 2 * c
        bits = (rec[:, :, at] << 16) | (rec[:, :, at + 1] << 24)
        bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
        return bits.view(torch.float32).double().unsqueeze(-1)

    k, v = k.double() * par(0) + par(1), v.double() * par(2) + par(3)
    return tuple(x.transpose(1, 2).reshape(-1, hkv, d)[:n] for x in (k, v))


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    cached, new = _lens(case)
    bs, d = case["bs"], case["d"]
    if case["op"] == "decode":
        kn, vn = _exact_row(s["k_new"]), _exact_row(s["v_new"])
        q = s["q"].double().view(case["batch"], case["hkv"], -1, d)
        out = torch.empty_like(q)
        for b, n in enumerate(cached):
            k, v = _exact_read(s["pool"], s["table"], b, n, bs, d)
            k, v = torch.cat([k, kn[b : b + 1]]), torch.cat([v, vn[b : b + 1]])
            w = torch.einsum("hgd,thd->hgt", q[b], k) / d ** 0.5
            out[b] = torch.einsum("hgt,thd->hgd", torch.softmax(w, -1), v)
        return dict(out=out.view(case["batch"], -1, d), k_stored=kn, v_stored=vn)
    ks, vs, at = [], [], 0
    if case["op"] == "store":
        kn, vn = _exact_row(s["k"]), _exact_row(s["v"])
    for b, n in enumerate(cached):
        k, v = _exact_read(s["pool"], s["table"], b, n, bs, d)
        ks.append(k), vs.append(v)
        if case["op"] == "store":
            ks.append(kn[at : at + new[b]]), vs.append(vn[at : at + new[b]])
            at += new[b]
    return dict(k=torch.cat(ks), v=torch.cat(vs))

"""Timed cases of rotary positions, the rotated append and block-sparse attention.

Four operators, reached through the package's public calls:

* ``rotary``  pa_rotary: queries and keys turned by their positions, one axis or
  several (time, height, width);
* ``append``  pa_cache_append_rotary: a step's queries and keys turned, keys and
  values put into the paged cache, the bounds of the keys of each block kept;
* ``select``  pa_select_blocks: the blocks whose bounds promise the largest
  scores, for each query and kv head;
* ``sparse``  pa_sparse: attention over the selected blocks of the paged cache.

The cache is [num_blocks, block_size, num_kv_heads, head_dim], its bounds
[num_blocks, num_kv_heads, 2, head_dim]: the least and the largest value of each
channel over the keys of the block.
"""
import torch

own = False

_GOLD = 0.6180339887498949


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a chat, q and k only: the smallest call there is
        dict(name="rotary_single", op="rotary", tokens=1, lo=4321, hq=32, hkv=8, d=128, rot=128, style="half", axes=1, fused=False, dtype="bf16"),
        # a video prompt: time, height and width in sections, heads cut out of one projection
        dict(name="rotary_video", op="rotary", tokens=32761, lo=57, hq=32, hkv=8, d=128, rot=128, style="half", axes=3, fused=True, dtype="bf16"),
        # a decode step of the repository's 64-sequence workload
        dict(name="append_decode_64", op="append", batch=64, lo=512, hi=4096, new_lo=1, new_hi=1, hq=32, hkv=8, d=128, bs=16, rot=128,
             style="half", axes=1, fused=True, bounds=True, dtype="bf16"),
        # its prefill workload: 32 chunks after cached prefixes
        dict(name="append_prefill", op="append", batch=32, lo=0, hi=1024, new_lo=1, new_hi=2048, hq=32, hkv=8, d=128, bs=16, rot=128,
             style="half", axes=1, fused=True, bounds=True, dtype="bf16"),
        # one conversation: the latency of choosing 64 blocks of 313
        dict(name="select_single", op="select", batch=1, lo=5000, hi=5000, hq=32, hkv=8, d=128, bs=16, top=64, dtype="bf16"),
        # many long contexts, 8 query heads to a kv head
        dict(name="select_long", op="select", batch=96, lo=4096, hi=32768, hq=64, hkv=8, d=128, bs=16, top=128, dtype="bf16"),
        # chunks of prompts, every token with its own choice
        dict(name="select_chunk", op="select", batch=5, lo=3000, hi=12000, new_lo=33, new_hi=161, hq=32, hkv=8, d=128, bs=16, top=64, dtype="bf16"),
        # a small fp32 model, odd lengths
        dict(name="select_f32", op="select", batch=13, lo=777, hi=9000, hq=12, hkv=3, d=64, bs=32, top=17, dtype="f32"),
        # one conversation: 64 blocks for a single token
        dict(name="sparse_single", op="sparse", batch=1, lo=5000, hi=5000, hq=32, hkv=8, d=128, bs=16, top=64, dtype="bf16"),
        # many long contexts, 2048 keys of each
        dict(name="sparse_long", op="sparse", batch=96, lo=4096, hi=32768, hq=64, hkv=8, d=128, bs=16, top=128, dtype="bf16"),
        # chunks of prompts, every token with its own blocks
        dict(name="sparse_chunk", op="sparse", batch=5, lo=3000, hi=12000, new_lo=33, new_hi=161, hq=32, hkv=8, d=128, bs=16, top=64, dtype="bf16"),
        # a small fp32 model, odd lengths, some shorter than the selection
        dict(name="sparse_f32", op="sparse", batch=13, lo=300, hi=9000, hq=12, hkv=3, d=64, bs=32, top=17, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["rotary", "append", "append", "select", "select", "sparse", "sparse"])
    d, bs = rng.choice([64, 128]), rng.choice([16, 32])
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    turn = dict(rot=rng.choice([d, d, d // 2]), style=rng.choice(["half", "pairs"]), axes=rng.choice([1, 1, 2, 3]),
                fused=rng.random() < 0.5)
    if op == "rotary":
        tokens = _log_int(rng, 1, min(65536, 100_000_000 // ((hq + hkv) * d)))
        return dict(op=op, tokens=tokens, lo=rng.randint(0, 65536), hq=hq, hkv=hkv, d=d, dtype=dtype, **turn)
    if op == "append":
        budget = _log_int(rng, 1, 70_000_000 // ((hq + 2 * hkv) * d))  # new tokens
        batch = min(_log_int(rng, 1, 1024), budget)
        room = max(1, (2 if batch > 4 else 1) * (budget // batch))
        return dict(op=op, batch=batch, lo=0, hi=_log_int(rng, 1, 4096), new_lo=rng.choice([0, 1]) if room > 1 else 1, new_hi=room,
                    hq=hq, hkv=hkv, d=d, bs=bs, bounds=rng.random() < 0.8, dtype=dtype, **turn)
    top = _log_int(rng, 3, 256)
    chunk = rng.random() < 0.4
    if op == "select":
        blocks = _log_int(rng, 8, 100_000_000 // (2 * hkv * d))  # of all requests
        batch = min(_log_int(rng, 1, 256), max(1, blocks // 8))
        hi = min(131072, max(8, blocks // batch) * bs)
        top = min(top, hi // bs // 2)  # some of the requests have more blocks than that
        most = max(1, 8_000_000 // (hq * (hi // bs + 1)))  # queries
    else:
        most = 130_000_000 // (hkv * d * bs * top)
        batch = min(_log_int(rng, 1, 256), most)
        hi = min(131072, max(1, _log_int(rng, bs, 50_000_000 // (hkv * d * batch))))
    c = dict(op=op, batch=min(batch, most), lo=rng.randint(0, hi), hi=hi, hq=hq, hkv=hkv, d=d, bs=bs, top=top, dtype=dtype)
    if chunk and most >= 2 * batch:
        c["new_lo"], c["new_hi"] = rng.choice([0, 1]), _log_int(rng, 1, min(256, most // batch))
    return c


def _spread(n, lo, hi, shift=0.0):
    """n whole numbers spread evenly over lo..hi, the same for every seed."""
    return [lo + int((hi - lo + 1) * (((i + 1) * _GOLD + shift) % 1.0)) for i in range(n)]


def _lens(case):
    """Tokens cached before the step and new ones, of each request."""
    cached = _spread(case["batch"], case["lo"], case["hi"])
    new = _spread(case["batch"], case["new_lo"], case["new_hi"], 0.37) if "new_lo" in case else [1] * case["batch"]
    new[0] = max(1, new[0])
    return cached, new


def _blocks(n, bs):
    return -(-n // bs)


def _bytes(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    op, d, hq, hkv, e = case["op"], case["d"], case["hq"], case["hkv"], _bytes(case)
    if op == "rotary":
        t = case["tokens"]
        return {"bytes": float(t * (2 * (hq + hkv) * d * e + 4 * case["axes"] + 4 * case["rot"])), "flops": 3.0 * t * (hq + hkv) * case["rot"]}
    cached, new = _lens(case)
    bs, t = case["bs"], sum(new)
    if op == "append":
        fresh = sum(_blocks(c + n, bs) - _blocks(c, bs) for c, n in zip(cached, new))
        begun = sum(1 for c, n in zip(cached, new) if n and c % bs)
        bound = (fresh + 2 * begun) * hkv * 2 * d * e if case["bounds"] else 0
        return {"bytes": float(t * (2 * (hq + 2 * hkv) * d * e + 4 * case["axes"] + 4 + 4 * case["rot"]) + bound),
                "flops": 3.0 * t * (hq + hkv) * case["rot"]}
    top = case["top"]
    nbytes = flops = 0.0
    for c, n in zip(cached, new):
        if n == 0:
            continue
        have = _blocks(c + n, bs)
        seen = [_blocks(c + i + 1, bs) for i in range(n)]
        nbytes += n * (hq * d * e + hkv * top * 4)
        if op == "select":  # where the blocks are more than the selection, all but the first and the last are scored
            if have > top:
                nbytes += (have - 2) * (hkv * 2 * d * e + 4)
            flops += sum(4.0 * (s - 2) * hq * d for s in seen if s > top)
        else:  # the blocks that any of the queries chose, as often as chance has it
            mean = sum(min(s, top) for s in seen) / n
            union = have * (1.0 - (1.0 - mean / have) ** n)
            nbytes += union * (hkv * bs * 2 * d * e + 4) + n * hq * d * e
            flops += 4.0 * sum(min(s, top) for s in seen) * bs * hq * d
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ plain forms
def _rows(lens, total):
    """(request, position in it) of each of `total` packed rows."""
    start = torch.cumsum(lens, 0) - lens
    req = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens, output_size=total)
    return req, torch.arange(total, device=lens.device) - start[req]


def _turn(x, s, kind):
    """Rows x [T, H, D] turned by the tokens' positions, in `kind`."""
    half = s["cos_sin"].shape[1] // 2
    axis = torch.tensor(s["pair_axis"] or [0] * half, device=x.device)
    pos = s["positions"].view(-1, x.shape[0])[axis].t().long()  # [T, pairs]
    pair = torch.arange(half, device=x.device)
    cos, sin = (s["cos_sin"][pos, pair + k * half].to(kind).unsqueeze(1) for k in (0, 1))
    y = x.to(kind)
    if s["style"] == "half":
        a, b = y[..., :half], y[..., half: 2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0: 2 * half: 2], y[..., 1: 2 * half: 2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _plain_append(s):
    dtype, bs = s["dtype"], s["bs"]
    q_out, k = _turn(s["q"], s, torch.float32).to(dtype), _turn(s["k"], s, torch.float32).to(dtype)
    slot = s["slots"].long()
    block, off = slot // bs, slot % bs
    s["k_cache"][block, off] = k
    s["v_cache"][block, off] = s["v"]
    out = dict(q=q_out, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["bounds"] is not None:
        _widen(s["bounds"], block, off, k)
        out["bounds"] = s["bounds"]
    return out


def _widen(bounds, block, off, k):
    """Bounds [NB, Hkv, 2, D] with the keys k [T, Hkv, D] of `block` taken in:
    a block whose first key is among them starts anew."""
    fresh = block[off == 0]
    bounds[fresh, :, 0], bounds[fresh, :, 1] = float("inf"), -float("inf")
    at = block.view(-1, 1, 1).expand(k.shape)
    bounds[:, :, 0] = bounds[:, :, 0].scatter_reduce(0, at, k, "amin")
    bounds[:, :, 1] = bounds[:, :, 1].scatter_reduce(0, at, k, "amax")


def _positions(s):
    """(request, last visible position) of each query."""
    if s["cu_q"] is None:
        return torch.arange(s["q"].shape[0], device=s["q"].device), s["lens"].long() - 1
    count = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    req, i = _rows(count, s["q"].shape[0])
    return req, s["lens"].long()[req] - count[req] + i


def _plain_select(s):
    q, bounds, top, bs = s["q"].double(), s["bounds"], s["top"], s["bs"]
    hkv, d = bounds.shape[1], bounds.shape[3]
    req, last = _positions(s)
    width = s["table"].shape[1]
    got = []
    for r in range(len(s["counts"])):
        n = s["counts"][r]
        if n == 0:
            continue
        mine = req == r
        lo, hi = bounds[s["table"][r].clamp(min=0).long()].double().permute(2, 1, 3, 0)  # [Hkv, D, blocks]
        x = q[mine].view(n, hkv, -1, d).transpose(0, 1)  # [Hkv, n, G, D]
        x = x.reshape(hkv, -1, d)
        score = (x.clamp(min=0) @ hi + x.clamp(max=0) @ lo).view(hkv, n, -1, width).amax(2).transpose(0, 1)
        seen = (last[mine] // bs + 1).view(-1, 1, 1)
        j = torch.arange(width, device=q.device)
        forced = (j < s["first"]) | (j >= seen - s["final"])
        score = torch.where(forced, float("inf"), score).masked_fill(j >= seen, -float("inf"))
        pick = score.sort(dim=-1, descending=True, stable=True).indices
        rank = torch.arange(min(top, width), device=q.device)
        pick = pick[..., :top].masked_fill(rank >= seen, width).sort(-1).values
        pick = pick.masked_fill(pick == width, -1).int()
        got.append(torch.nn.functional.pad(pick, (0, top - pick.shape[-1]), value=-1))
    return dict(selected=torch.cat(got))


def _plain_sparse(s):
    q, bs, top = s["q"].float(), s["bs"], s["selected"].shape[2]
    t, hq, d = q.shape
    hkv = s["k_cache"].shape[2]
    req, last = _positions(s)
    sel = s["selected"].long()
    phys = s["table"].long()[req.view(-1, 1, 1), sel.clamp(min=0)].clamp(min=0)  # [T, Hkv, top]
    head = torch.arange(hkv, device=q.device).view(1, -1, 1, 1)
    off = torch.arange(bs, device=q.device)
    seen = (sel.unsqueeze(-1) >= 0) & (sel.unsqueeze(-1) * bs + off <= last.view(-1, 1, 1, 1))
    seen = seen.view(t, hkv, 1, top * bs)
    k, v = (s[x][phys.unsqueeze(-1), off, head].float().view(t, hkv, top * bs, d) for x in ("k_cache", "v_cache"))
    v = v * seen.view(t, hkv, -1, 1)
    score = (q.view(t, hkv, hq // hkv, d) @ k.transpose(2, 3)) * d ** -0.5
    score = score.masked_fill(~seen, -float("inf"))
    most = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(most == -float("inf"), 0.0, most))
    total = p.sum(-1, keepdim=True)
    return dict(out=((p @ v) / torch.where(total == 0, 1.0, total)).view(t, hq, d).to(s["dtype"]))


# ------------------------------------------------------------------ inputs
def _turning(case, dev, first, new):
    """What the rotation takes: positions [axes, T] of tokens that follow `first`
    cached ones, the table of cos and sin, the axis of each pair."""
    axes, rot = case["axes"], case["rot"]
    req, i = _rows(torch.tensor(new, device=dev), sum(new))
    start = torch.tensor(first, device=dev)[req]
    if axes == 1:
        pos = start + i
    else:  # frames of 28 x 44 patches, or pictures of 44 columns
        grid = [i // 1232, i // 44 % 28, i % 44] if axes == 3 else [i // 44, i % 44]
        pos = torch.stack([start + x for x in grid])
    most = int(pos.max()) + 1 if pos.numel() else 1
    pairs = rot // 2
    freq = 10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)
    angle = torch.arange(most, device=dev, dtype=torch.float64).unsqueeze(1) * freq
    axis = None
    if axes == 2:
        axis = [0] * (pairs // 2) + [1] * (pairs - pairs // 2)
    if axes == 3:
        t = pairs // 4
        h = (pairs - t) // 2
        axis = [0] * t + [1] * h + [2] * (pairs - t - h)
    return dict(positions=pos.int().contiguous(), cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(), pair_axis=axis, style=case["style"])


def _heads(case, rand, tokens):
    """q, k, v [T, H, D]: tensors of their own, or cut out of one projection's output."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["fused"]:
        return rand(tokens, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    return rand(tokens, hq, d), rand(tokens, hkv, d), rand(tokens, hkv, d)


def _table(g, dev, held, extra):
    """Rows of distinct blocks in any order, -1 behind each row's blocks."""
    nb = sum(held) + extra
    perm = torch.randperm(nb, generator=g, device=dev)
    table = torch.full((len(held), max(1, max(held))), -1, dtype=torch.int32, device=dev)
    req, j = _rows(torch.tensor(held, device=dev), sum(held))
    table[req, j] = perm[: sum(held)].int()
    return nb, table


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    d, hkv, op = case["d"], case["hkv"], case["op"]
    rand = lambda *sh: torch.randn(*sh, generator=g, device=dev).to(dtype)  # noqa: E731
    if op == "rotary":
        q, k, _ = _heads(case, rand, case["tokens"])
        return dict(op=op, dtype=dtype, q=q, k=k, q_out=torch.empty(q.shape, dtype=dtype, device=dev),
                    k_out=torch.empty(k.shape, dtype=dtype, device=dev), **_turning(case, dev, [case["lo"]], [case["tokens"]]))
    cached, new = _lens(case)
    bs, tokens = case["bs"], sum(new)
    nb, table = _table(g, dev, [_blocks(c + n, bs) for c, n in zip(cached, new)], 1 + case["batch"] // 4)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(op=op, dtype=dtype, bs=bs, table=table, lens=i32([c + n for c, n in zip(cached, new)]))
    gain = torch.exp(0.4 * torch.randn(hkv, d, generator=g, device=dev))  # keys have strong and weak channels
    if op == "append":
        q, k, v = _heads(case, rand, tokens)
        req, i = _rows(torch.tensor(new, device=dev), tokens)
        pos = torch.tensor(cached, device=dev)[req] + i
        s.update(q=q, k=k, v=v, k_cache=(rand(nb, bs, hkv, d) * gain).to(dtype), v_cache=rand(nb, bs, hkv, d), bounds=None,
                 slots=(table[req, pos // bs] * bs + pos % bs).int(), q_out=torch.empty(q.shape, dtype=dtype, device=dev),
                 **_turning(case, dev, cached, new))
        if case["bounds"]:
            s["bounds"] = torch.zeros(nb, hkv, 2, d, dtype=dtype, device=dev)
            req, pos = _rows(torch.tensor(cached, device=dev), sum(cached))
            block, off = table[req, pos // bs].long(), pos % bs
            _widen(s["bounds"], block, off, s["k_cache"][block, off])
        return s
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s.update(q=rand(tokens, case["hq"], d), cu_q=i32(cu) if "new_lo" in case else None, counts=new)
    if op == "select":
        # the middle of a block's keys and their spread about it
        mid, up, down = (torch.randn(nb, hkv, d, generator=g, device=dev) for _ in range(3))
        lo, hi = mid - down.mul_(0.3).add_(1.4).clamp_(min=0), mid + up.mul_(0.3).add_(1.4).clamp_(min=0)
        s["bounds"] = torch.stack([lo * gain, hi * gain], 2).to(dtype)
        s.update(top=case["top"], first=1, final=1, selected=torch.empty(tokens, hkv, case["top"], dtype=torch.int32, device=dev))
        return s
    s.update(k_cache=(rand(nb, bs, hkv, d) * gain).to(dtype), v_cache=rand(nb, bs, hkv, d), out=torch.empty_like(s["q"]))
    # the first block, the last one and any others, in order
    width, (req, last) = table.shape[1], _positions(s)
    j, seen = torch.arange(width, device=dev), (last // bs + 1).view(-1, 1, 1)
    chance = torch.rand(tokens, hkv, width, generator=g, device=dev)
    chance = torch.where((j == 0) | (j == seen - 1), 2.0, chance).masked_fill(j >= seen, -1.0)
    pick = chance.topk(min(case["top"], width), -1)
    pick = pick.indices.masked_fill(pick.values < 0, width).sort(-1).values.int()
    pick = pick.masked_fill(pick == width, -1)
    s["selected"] = torch.nn.functional.pad(pick, (0, case["top"] - pick.shape[-1]), value=-1).contiguous()
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_300_gb300 as pa

        if op == "rotary":
            pa.pa_rotary(s["q"], s["k"], s["positions"], s["cos_sin"], q_out=s["q_out"], k_out=s["k_out"], pair_axis=s["pair_axis"],
                         interleaved=s["style"] == "pairs")
            return dict(q=s["q_out"], k=s["k_out"])
        if op == "append":
            pa.pa_cache_append_rotary(s["q"], s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["positions"], s["cos_sin"],
                                      q_out=s["q_out"], bounds=s["bounds"], pair_axis=s["pair_axis"], interleaved=s["style"] == "pairs")
            out = dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
            return out if s["bounds"] is None else dict(out, bounds=s["bounds"])
        if op == "select":
            pa.pa_select_blocks(s["q"], s["bounds"], s["table"], s["lens"], s["top"], s["bs"], first_blocks=s["first"],
                                last_blocks=s["final"], cu_seq_lens_q=s["cu_q"], selected=s["selected"])
            return dict(selected=s["selected"])
        pa.pa_sparse(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["selected"], cu_seq_lens_q=s["cu_q"], out=s["out"])
        return dict(out=s["out"])
    if op == "rotary":
        return dict(q=_turn(s["q"], s, torch.float32).to(s["dtype"]), k=_turn(s["k"], s, torch.float32).to(s["dtype"]))
    return {"append": _plain_append, "select": _plain_select, "sparse": _plain_sparse}[op](s)


# ------------------------------------------------------------------ in 64 bits
def _exact_turn(x, s):
    """Rows turned as complex numbers: pair i of a token by its angle."""
    cs = s["cos_sin"].double()
    half = cs.shape[1] // 2
    pos = s["positions"].view(-1, x.shape[0]).long()
    y = x.double().clone()
    for i in range(half):
        row = pos[s["pair_axis"][i] if s["pair_axis"] else 0]
        w = torch.complex(cs[row, i], cs[row, half + i]).unsqueeze(1)
        a, b = (i, half + i) if s["style"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(y[..., a], y[..., b]) * w
        y[..., a], y[..., b] = z.real, z.imag
    return y


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return dict(q=_exact_turn(s["q"], s), k=_exact_turn(s["k"], s))
    bs, d = case["bs"], case["d"]
    cached, new = _lens(case)
    if case["op"] == "append":
        k, kc, vc = _exact_turn(s["k"], s), s["k_cache"].double(), s["v_cache"].double()
        hkv = kc.shape[2]
        slot = s["slots"].long()
        kc.view(-1, hkv, d)[slot], vc.view(-1, hkv, d)[slot] = k, s["v"].double()
        out = dict(q=_exact_turn(s["q"], s), k_cache=kc, v_cache=vc)
        if s["bounds"] is not None:
            # every block of a request that got tokens, over the keys it now holds
            b = s["bounds"].double()
            req, j = _rows(s["lens"].long().add(bs - 1) // bs, sum(_blocks(c + n, bs) for c, n in zip(cached, new)))
            some = torch.tensor(new, device=b.device)[req] > 0
            req, j = req[some], j[some]
            here = s["table"][req, j].long()
            held = (s["lens"].long()[req] - j * bs).view(-1, 1, 1, 1) > torch.arange(bs, device=b.device).view(1, -1, 1, 1)
            b[here, :, 0] = kc[here].masked_fill(~held, float("inf")).amin(1)
            b[here, :, 1] = kc[here].masked_fill(~held, -float("inf")).amax(1)
            out["bounds"] = b
        return out
    hkv, tokens = case["hkv"], s["q"].shape[0]
    if tokens * hkv > 6000:
        return None  # row by row it takes too long
    q = s["q"].double().view(tokens, hkv, -1, d)
    out = torch.zeros_like(q)
    req = [r for r, n in enumerate(new) for _ in range(n)]
    last = [c + i for c, n in zip(cached, new) for i in range(n)]
    for t in range(tokens):
        for h in range(hkv):
            logical = s["selected"][t, h]
            logical = logical[logical >= 0].long()
            where = s["table"][req[t]][logical].long()
            pos = logical.unsqueeze(1) * bs + torch.arange(bs, device=q.device)
            ok = (pos <= last[t]).view(-1)
            k, v = (s[x][where, :, h].double().reshape(-1, d)[ok] for x in ("k_cache", "v_cache"))
            out[t, h] = torch.softmax(q[t, h] @ k.t() / d ** 0.5, -1) @ v
    return dict(out=out.view(tokens, -1, d))

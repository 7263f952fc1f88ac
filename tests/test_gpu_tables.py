"""pa_block_tables against the plain reference (whole numbers: equal)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import q4

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa.load()


def make(seed, lens, new, bs, spare, wide=None, slack=0):
    rng = np.random.default_rng(seed)
    held = [-(-n // bs) for n in lens]
    nb = sum(held) + spare + slack
    perm = rng.permutation(nb).astype(np.int32)
    wide = wide or max(-(-(n + max(m, 0)) // bs) for n, m in zip(lens, new)) + 1
    table = np.full((len(lens), wide), -1, dtype=np.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += h
    free = np.full(nb, -1, dtype=np.int32)
    free[:spare] = perm[at:at + spare]
    return np.array(lens, dtype=np.int32), np.array(new, dtype=np.int32), table, free


def run(lens, new, table, free, num_free, total, bs, **kw):
    t = lambda x: torch.from_numpy(np.array(x)).to(DEV)  # noqa: E731
    d = dict(lens=t(lens), table=t(table), free=t(free), nf=t(np.array([num_free], dtype=np.int32)),
             slots=torch.full((total,), 12345, dtype=torch.int32, device=DEV),
             err=torch.zeros(1, dtype=torch.int32, device=DEV))
    out = pa.pa_block_tables(d["lens"], t(new), d["table"], d["free"], d["nf"], d["slots"], bs, dev_err=d["err"], **kw)
    torch.cuda.synchronize()
    return d, [x.cpu().numpy() for x in out]


def same(d, out, want):
    table, free, num_free, slots, cu_q, cu_k, after = want
    assert np.array_equal(out[0], cu_q) and np.array_equal(out[1], cu_k) and np.array_equal(out[2], after)
    assert np.array_equal(d["slots"].cpu().numpy(), slots)
    assert np.array_equal(d["table"].cpu().numpy(), table)
    assert int(d["nf"].item()) == num_free
    # the stack is what counts; what lies behind its top is nobody's
    assert np.array_equal(d["free"].cpu().numpy()[:num_free], free[:num_free])


CASES = {
    "one": ([1000], [1], 32),
    "first token": ([0], [1], 16),
    "nothing new": ([5, 0, 16], [0, 0, 0], 16),
    "all end": ([5, 0, 16, 17], [-1, -1, -1, -1], 16),
    "block borders": ([15, 16, 17, 31, 32, 0], [1, 1, 15, 2, 32, 33], 16),
    "odd block size": ([3, 10, 0], [8, 1, 25], 5),
    "one long prompt": ([7] + [100] * 9, [20000] + [1] * 9, 16),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("tail", [0, 37])
def test_small(name, tail):
    lens, new, bs = CASES[name]
    tokens = sum(max(m, 0) for m in new)
    need = sum(-(-(n + m) // bs) - -(-n // bs) for n, m in zip(lens, new) if m > 0)
    lens, new, table, free = make(1, lens, new, bs, need + 1)
    want = q4.block_tables(lens, new, table, free, need + 1, tokens + tail, bs)
    d, out = run(lens, new, table, free, need + 1, tokens + tail, bs)
    assert int(d["err"].item()) == 0
    same(d, out, want)


@pytest.mark.parametrize("batch,new_hi,bs", [(255, 1, 16), (1025, 40, 16), (4097, 9, 32), (16384, 3, 16), (33, 3000, 32)])
def test_random_steps_with_ended_requests(batch, new_hi, bs):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 700, batch)
    new = np.where(rng.random(batch) < 0.2, -1, rng.integers(0, new_hi + 1, batch))
    tokens = int(np.maximum(new, 0).sum())
    take = int(sum(-(-(n + m) // bs) - -(-n // bs) for n, m in zip(lens.tolist(), new.tolist()) if m > 0))
    back = int(sum(-(-n // bs) for n, m in zip(lens.tolist(), new.tolist()) if m < 0))
    spare = max(0, take - back // 2)  # some of the taken blocks have just been given back
    lens, new, table, free = make(batch, lens.tolist(), new.tolist(), bs, spare, slack=5)
    want = q4.block_tables(lens, new, table, free, spare, tokens + 3, bs)
    assert want is not None
    d, out = run(lens, new, table, free, spare, tokens + 3, bs)
    assert int(d["err"].item()) == 0
    same(d, out, want)


def test_empty_batch():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    nf = torch.tensor([3], dtype=torch.int32, device=DEV)
    slots = torch.full((7,), 5, dtype=torch.int32, device=DEV)
    cu_q, cu_k, lens = pa.pa_block_tables(z, z, z.view(0, 4), torch.zeros(9, dtype=torch.int32, device=DEV), nf, slots, 16)
    assert cu_q.tolist() == [0] and cu_k.tolist() == [0] and lens.numel() == 0
    assert slots.tolist() == [-1] * 7 and nf.item() == 3


REFUSED = {
    "no space": ([16, 16], [40, 16], dict(spare=3, total=56), pa.DEVERR_NO_SPACE),
    "slot map short": ([16, 16], [4, 4], dict(spare=3, total=7), pa.DEVERR_NO_SPACE),
    "beyond the row": ([16, 16], [17, 1], dict(spare=9, total=99, wide=2), pa.DEVERR_OVERFLOW),
    "negative length": ([16, -1], [1, 1], dict(spare=9, total=99, wide=4), pa.DEVERR_OVERFLOW),
    "new below -1": ([16, 16], [1, -2], dict(spare=9, total=99, wide=4), pa.DEVERR_OVERFLOW),
    "stack overfull": ([16, 16], [1, -1], dict(spare=3, total=99, count=5), pa.DEVERR_BAD_BLOCK),  # 5 + 1 of 5 blocks
    "count negative": ([16, 16], [0, 0], dict(spare=3, total=9, count=-1), pa.DEVERR_BAD_BLOCK),
    "count too large": ([16, 16], [0, 0], dict(spare=3, total=9, count=6), pa.DEVERR_BAD_BLOCK),
}


@pytest.mark.parametrize("name", REFUSED)
def test_a_refused_step_changes_nothing(name):
    lens, new, o, flag = REFUSED[name]
    safe = [max(n, 0) for n in lens]
    _, _, table, free = make(2, safe, [0, 0], 16, o["spare"], wide=o.get("wide", 8))
    count = o.get("count", o["spare"])
    lens, new = np.array(lens, dtype=np.int32), np.array(new, dtype=np.int32)
    d, out = run(lens, new, table, free, count, o["total"], 16)
    assert int(d["err"].item()) & flag
    assert np.array_equal(d["table"].cpu().numpy(), table) and np.array_equal(d["free"].cpu().numpy(), free)
    assert int(d["nf"].item()) == count
    assert (d["slots"] == -1).all()
    assert not out[0].any() and not out[1].any() and np.array_equal(out[2], lens)


def test_ids_outside_the_pool_become_minus_one():
    lens, new, table, free = make(3, [20, 40, 16], [3, -1, 1], 16, 2, slack=4)
    table[0, 1] = 99   # needed: token 20's block
    table[1, 2] = -7   # given back
    d, out = run(lens, new, table, free, 2, 6, 16)
    want = q4.block_tables(lens, new, table, free, 2, 6, 16)
    assert int(d["err"].item()) == pa.DEVERR_BAD_BLOCK
    same(d, out, want)
    assert d["slots"].cpu().tolist()[:4] == [-1] * 4  # the last block given back was taken next


def test_captured_step_advances_lengths_and_stack_in_place():
    """A step that writes its lengths and its stack back, captured once and
    replayed: every replay is the next step."""
    bs, b, steps = 16, 12, 40
    rng = np.random.default_rng(8)
    lens0 = rng.integers(0, 60, b).tolist()
    lens, new, table, free = make(9, lens0, [1] * b, bs, b * 4, wide=10)
    t = lambda x: torch.from_numpy(np.array(x)).to(DEV)  # noqa: E731
    g_len, g_new, g_tab, g_free = t(lens), t(new), t(table), t(free)
    nf = t(np.array([b * 4], dtype=np.int32))
    slots = torch.empty(b, dtype=torch.int32, device=DEV)
    outs = [torch.empty(b + 1, dtype=torch.int32, device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        pa.pa_block_tables(g_len, g_new, g_tab, g_free, nf, slots, bs, cu_seq_lens_q=outs[0], cu_seq_lens_k=outs[1],
                           seqlens_k=g_len, dev_err=err)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    count = b * 4
    for _ in range(steps):
        graph.replay()
        table, free, count, want, cu_q, cu_k, lens = q4.block_tables(lens, new, table, free, count, b, bs)
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(g_tab.cpu().numpy(), table)
        assert np.array_equal(g_len.cpu().numpy(), lens) and nf.item() == count
        assert np.array_equal(outs[1].cpu().numpy(), cu_k)
    assert err.item() == 0


@pytest.mark.parametrize("new,flag", [([40, 16], 0), ([40, -2], pa.DEVERR_OVERFLOW)])
def test_the_largest_slot_map_is_filled_to_its_end_and_no_further(new, flag):
    """2^31 - 1 slots, served and refused: the index of a thread's last step
    does not fit 32 bits.  The map lies between other data."""
    n, lens, bs = 2 ** 31 - 1, [16, 16], 16
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB")
    memory = torch.full((n + 2048,), 77, dtype=torch.int32, device=DEV)
    slots = memory[1024:1024 + n]
    lens, new, table, free = make(4, lens, new, bs, 5)
    t = lambda x: torch.from_numpy(np.array(x)).to(DEV)  # noqa: E731
    err = t(np.zeros(1, dtype=np.int32))
    nf = t(np.array([5], dtype=np.int32))
    cu_q, _, _ = pa.pa_block_tables(t(lens), t(new), t(table), t(free), nf, slots, bs, dev_err=err)
    assert err.item() == flag
    tokens = int(cu_q[-1].item())
    assert tokens == (0 if flag else 56)
    assert (slots[:tokens] >= 0).all()
    for at in range(tokens, n, 2 ** 28):
        assert (slots[at:min(n, at + 2 ** 28)] == -1).all()
    assert (memory[:1024] == 77).all() and (memory[1024 + n:] == 77).all()


def test_sizes_that_do_not_fit_an_int_are_refused():
    """2^32 entries would reach the library as 0, 2^32 + 4 as 4."""
    if torch.cuda.mem_get_info()[0] < 20 * 2 ** 30:
        pytest.skip("needs 20 GB")
    big = torch.empty(2 ** 32 + 4, dtype=torch.int32, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    args = dict(table=i32(0, 0).view(1, 2), free=i32(0, 0, 0), slots=i32(0))
    for name, t in (("slots", big), ("free", big), ("table", big.view(1, -1))):
        a = {**args, name: t}
        with pytest.raises(ValueError, match="2\\^31"):
            pa.pa_block_tables(i32(3), i32(0), a["table"], a["free"], i32(1), a["slots"], 16)
    rows = lambda: torch.zeros(1, 1, 64, device=DEV)  # noqa: E731
    pool = pa.pa_q4_pool(2, 1, 64, 16)
    with pytest.raises(ValueError, match="2\\^31"):
        pa.pa_decode_q4(rows(), pool, big.view(1, -1), i32(0), rows(), rows())
    with pytest.raises(ValueError, match="2\\^31"):
        pa.pa_cache_gather_q4(pool, big.view(1, -1), i32(0, 1), rows(), rows())


def _decode_lens(lens, new):
    return np.where(np.asarray(new) == 1, lens, pa.PA_LEFT_OUT).astype(np.int32)


@pytest.mark.parametrize("batch,new_hi", [(1, 1), (40, 3), (1025, 1), (4097, 9), (16384, 3)])
def test_decode_lens(batch, new_hi):
    """Lengths before the step where one token is new; everybody else, ended
    requests among them, is left out of the decode behind it."""
    bs = 16
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 300, batch).tolist()
    new = np.where(rng.random(batch) < 0.2, -1, rng.integers(0, new_hi + 1, batch)).tolist()
    tokens = sum(max(m, 0) for m in new)
    lens, new, table, free = make(batch, lens, new, bs, tokens + 1)
    out = torch.full((batch,), 5, dtype=torch.int32, device=DEV)
    want = q4.block_tables(lens, new, table, free, tokens + 1, tokens, bs)
    d, res = run(lens, new, table, free, tokens + 1, tokens, bs, decode_lens=out)
    same(d, res, want)
    assert int(d["err"].item()) == 0 and np.array_equal(out.cpu().numpy(), _decode_lens(lens, new))


@pytest.mark.parametrize("tail", [0, 5000, 20000])
def test_a_refused_step_leaves_everybody_out_of_the_decode(tail):
    lens, new, table, free = make(5, [16, 40, 3], [1, 1, -1], 16, 0)
    new[0] = 400  # longer than its row
    out = torch.full((3,), 5, dtype=torch.int32, device=DEV)
    d, _ = run(lens, new, table, free, 0, 401 + tail, 16, decode_lens=out)
    assert int(d["err"].item()) & pa.DEVERR_OVERFLOW and (out == pa.PA_LEFT_OUT).all()


@pytest.mark.parametrize("total", [4096, 16384])
@pytest.mark.parametrize("name", REFUSED)
def test_a_refused_step_of_a_cluster_changes_nothing(name, total):
    """The refused steps again with slot maps that 8 and 16 CTAs fill."""
    lens, new, o, flag = REFUSED[name]
    if name == "slot map short":
        new, o = [total, 1], dict(o, spare=total // 16 + 9, total=total, wide=total // 16 + 3)
    else:
        o = dict(o, total=o["total"] + total)
    _, _, table, free = make(2, [max(n, 0) for n in lens], [0, 0], 16, o["spare"], wide=o.get("wide", 8))
    count = o.get("count", o["spare"])
    lens, new = np.array(lens, dtype=np.int32), np.array(new, dtype=np.int32)
    d, out = run(lens, new, table, free, count, o["total"], 16)
    assert int(d["err"].item()) & flag
    assert np.array_equal(d["table"].cpu().numpy(), table) and np.array_equal(d["free"].cpu().numpy(), free)
    assert int(d["nf"].item()) == count and (d["slots"] == -1).all()
    assert not out[0].any() and not out[1].any() and np.array_equal(out[2], lens)


@pytest.mark.parametrize("b,total", [(4500, 4500), (200, 17000), (16384, 16384)])
def test_captured_steps_of_a_cluster_in_place(b, total):
    """Lengths and stack written back by 8 and 16 CTAs, every replay the next
    step; requests pause and end."""
    bs, steps = 16, 8
    rng = np.random.default_rng(b)
    lens, _, table, free = make(10, rng.integers(0, 60, b).tolist(), [1] * b, bs, b, wide=6)
    t = lambda x: torch.from_numpy(np.array(x)).to(DEV)  # noqa: E731
    g_len, g_new, g_tab, g_free, nf = t(lens), t(lens), t(table), t(free), t(np.array([b], dtype=np.int32))
    slots = torch.empty(total, dtype=torch.int32, device=DEV)
    cu = [torch.empty(b + 1, dtype=torch.int32, device=DEV) for _ in range(2)]
    at = torch.empty(b, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_block_tables(g_len, g_new, g_tab, g_free, nf, slots, bs, cu_seq_lens_q=cu[0], cu_seq_lens_k=cu[1],
                           seqlens_k=g_len, decode_lens=at, dev_err=err)
    count = b
    for _ in range(steps):
        new = rng.choice([-1, 0, 1, 1, 1, 1], b).astype(np.int32)
        new[lens + 1 > 6 * bs] = -1
        g_new.copy_(t(new))
        graph.replay()
        before = lens
        table, free, count, want, cu_q, cu_k, lens = q4.block_tables(lens, new, table, free, count, total, bs)
        torch.cuda.synchronize()
        assert err.item() == 0 and nf.item() == count
        for got, w in ((slots, want), (g_tab, table), (g_len, lens), (cu[0], cu_q), (cu[1], cu_k),
                       (at, _decode_lens(before, new)), (g_free[:count], free[:count])):
            assert np.array_equal(got.cpu().numpy(), w)

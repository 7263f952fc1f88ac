"""pa_rotary and pa_cache_append_rotary on the GPU against the plain reference."""
import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import sparse as ref
from tests.sparse_util import BF16, F32, angle_table, f64, rotary_bound

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa.load()


def _axes(kind, pairs):
    if kind == 1:
        return None
    if kind == "sections":
        t = pairs // 4
        return [0] * t + [1] * ((pairs - t) // 2) + [2] * (pairs - t - (pairs - t) // 2)
    if kind == "turns":  # time, height, width in turn: no piece of 8 pairs has one axis
        return [i % 3 for i in range(pairs)]
    return [3] * pairs  # all of the pairs on the fourth of four axes


def _positions(kind, tokens, rows, rng):
    n = {1: 1, "sections": 3, "turns": 3, "fourth": 4}[kind]
    p = rng.integers(0, rows, (n, tokens)).astype(np.int32)
    return torch.from_numpy(p[0] if kind == 1 else p)


def _same(a, b):
    assert torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


def _close(got, x, pos, table, axes, style, dtype):
    want, mag = ref.rotary(f64(x), pos.numpy(), table.numpy(), axes, style)
    err = np.abs(f64(got) - want)
    bound = rotary_bound(want, mag, dtype)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("style", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (64, 16), (128, 128), (128, 48), (128, 112)])
@pytest.mark.parametrize("kind", [1, "sections", "turns", "fourth"])
def test_rotary(dtype, style, d, rot, kind):
    rng = np.random.default_rng(d + rot)
    table = angle_table(50, rot)
    for tokens, hq, hkv in ((1, 1, 1), (7, 5, 2), (33, 9, 4)):
        g = torch.Generator().manual_seed(tokens)
        q, k = torch.randn(tokens, hq, d, generator=g).to(dtype), torch.randn(tokens, hkv, d, generator=g).to(dtype)
        pos, axes = _positions(kind, tokens, 50, rng), _axes(kind, rot // 2)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        qo, ko = pa.pa_rotary(q.to(DEV), k.to(DEV), pos.to(DEV), table.to(DEV), interleaved=style, pair_axis=axes, dev_err=err)
        assert err.item() == 0
        _close(qo, q, pos, table, axes, style, dtype)
        _close(ko, k, pos, table, axes, style, dtype)
        _same(qo[..., rot:].cpu(), q[..., rot:])  # what is not turned keeps its bits
        _same(ko[..., rot:].cpu(), k[..., rot:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rotary_of_parts_of_a_projection_in_place_and_alone(dtype):
    d, hq, hkv, tokens, rot = 128, 6, 2, 41, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(tokens, hq + 2 * hkv, d, generator=g).to(dtype)
    table, pos = angle_table(99, rot), torch.randint(0, 99, (tokens,), generator=g, dtype=torch.int32)
    t, p = table.to(DEV), pos.to(DEV)
    whole = x.to(DEV)
    q, k, v = whole.split([hq, hkv, hkv], 1)
    a, b = pa.pa_rotary(q, k, p, t)
    _close(a, x[:, :hq], pos, table, None, False, dtype)
    _close(b, x[:, hq:hq + hkv], pos, table, None, False, dtype)
    _same(whole.cpu(), x)
    only_q, none = pa.pa_rotary(q, None, p, t)
    none2, only_k = pa.pa_rotary(None, k, p, t)
    assert none is None and none2 is None
    _same(only_q, a), _same(only_k, b)
    r = pa.pa_rotary(q, k, p, t, q_out=q, k_out=k)  # in place, the values between untouched
    assert r[0] is q and r[1] is k
    _same(q, a), _same(k, b), _same(v.cpu(), x[:, hq + hkv:])


def test_rotary_positions_outside_the_table():
    d, tokens = 64, 20
    table = angle_table(10, d)
    pos = torch.arange(tokens, dtype=torch.int32) % 10
    pos[3], pos[11] = -1, 10
    q, k = torch.randn(tokens, 3, d).to(BF16), torch.randn(tokens, 5, d).to(BF16)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qo, ko = pa.pa_rotary(q.to(DEV), k.to(DEV), pos.to(DEV), table.to(DEV), dev_err=err)
    assert err.item() == pa.DEVERR_OVERFLOW
    good = [i for i in range(tokens) if i not in (3, 11)]
    for got, x in ((qo, q), (ko, k)):
        assert (got[[3, 11]] == 0).all()
        _close(got[good], x[good], pos[good], table, None, False, BF16)


def test_rotary_far_rows_and_many_tokens():
    """More tokens than one wave of CTAs takes; table rows beyond 2^31 bytes."""
    d, tokens, rows = 128, 70001, (1 << 22) + 5
    table = torch.zeros(rows, d, device=DEV)
    table[:, : d // 2] = 1.0
    table[-1, : d // 2], table[-1, d // 2:] = 0.0, 1.0
    pos = torch.zeros(tokens, dtype=torch.int32, device=DEV)
    pos[::3] = rows - 1
    q = torch.randn(tokens, 2, d, device=DEV).to(BF16)
    k = torch.randn(tokens, 1, d, device=DEV).to(BF16)
    for got, x in zip(pa.pa_rotary(q, k, pos, table), (q, k)):
        want = x.clone()
        want[::3] = torch.cat([-x[::3, :, 64:], x[::3, :, :64]], -1)
        assert torch.equal(got, want)


# ------------------------------------------------------------------ append
def _slots(lens, new, bs, rng, spare=2):
    """Blocks in any order for requests of lens cached and new tokens: (slots, blocks)."""
    held = [-(-(n + m) // bs) for n, m in zip(lens, new)]
    nb = sum(held) + spare
    perm = rng.permutation(nb)
    slots, at = [], 0
    for n, m, h in zip(lens, new, held):
        own = perm[at:at + h]
        at += h
        slots += [int(own[p // bs]) * bs + p % bs for p in range(n, n + m)]
    return np.array(slots, dtype=np.int32), nb


def _check_append(x, slots, pos, table, axes, style, dtype, bs, before, after, refused=()):
    """The pool and bounds after an append of x = (q, k, v), from those before it."""
    (kc, vc, bd), (gk, gv, gb) = before, after
    hkv, d = kc.shape[2:]
    ok = [i for i, s in enumerate(slots) if s >= 0 and i not in refused]
    sl = torch.from_numpy(slots[ok]).long()
    rows = gk.view(-1, hkv, d)[sl]
    if table is None:
        _same(rows, x[1][ok])
    else:
        _close(rows, x[1][ok], pos[..., ok], table, axes, style, dtype)
    _same(gv.view(-1, hkv, d)[sl], x[2][ok])
    mask = torch.ones(kc.shape[0] * bs, dtype=torch.bool)
    mask[sl] = False
    for a, b in ((kc, gk), (vc, gv)):  # every other row has its bits
        _same(a.view(-1, hkv, d)[mask], b.view(-1, hkv, d)[mask])
    if bd is None:
        return
    want = bd.clone()
    for p in sorted(set((sl // bs).tolist())):
        mine = [int(s) for s in slots if s >= 0 and s // bs == p]
        lo, hi = ref.bounds_of(np.stack([f64(gk[p, s % bs]) for s in mine if s in set(sl.tolist())]))
        if mine[0] % bs:  # widened: the least of the least ones, the largest of the largest
            lo, hi = np.minimum(lo, f64(bd[p, :, 0])), np.maximum(hi, f64(bd[p, :, 1]))
        want[p, :, 0], want[p, :, 1] = torch.from_numpy(lo).to(dtype), torch.from_numpy(hi).to(dtype)
    assert torch.equal(torch.isnan(want), torch.isnan(gb))
    assert torch.equal(torch.nan_to_num(want, 7.0), torch.nan_to_num(gb, 7.0))


def _pool(g, nb, bs, hkv, d, dtype, with_bounds):
    r = lambda *s: torch.randn(*s, generator=g).to(dtype)  # noqa: E731
    return r(nb, bs, hkv, d), r(nb, bs, hkv, d), r(nb, hkv, 2, d) if with_bounds else None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot,style,kind", [(128, 128, False, 1), (64, 32, True, "turns"), (128, 64, True, "sections"), (64, 64, False, 1)])
@pytest.mark.parametrize("bs", [16, 32, 5])
@pytest.mark.parametrize("with_bounds", [True, False])
def test_append(dtype, d, rot, style, kind, bs, with_bounds):
    rng = np.random.default_rng(bs + d)
    for lens, new, hq, hkv in (([0], [1], 1, 1), ([7, 16, 0, 100, 31], [1, 1, 1, 1, 1], 8, 2),
                               ([0, 3, 40, 15, 2], [37, 0, 1, 60, 90], 5, 5), ([5], [131], 3, 9)):
        g = torch.Generator().manual_seed(len(lens))
        slots, nb = _slots(lens, new, bs, rng)
        slots = np.concatenate([slots, np.full(3, -1, dtype=np.int32)])  # padding behind the last token
        t = len(slots)
        x = [torch.randn(t, h, d, generator=g).to(dtype) for h in (hq, hkv, hkv)]
        before = _pool(g, nb, bs, hkv, d, dtype, with_bounds)
        after = [None if b is None else b.to(DEV) for b in before]
        table, axes = angle_table(300, rot), _axes(kind, rot // 2)
        pos = _positions(kind, t, 300, rng)
        pos[..., -3:] = -77  # of padding nothing is read
        qo = torch.full((t, hq, d), 5.0, dtype=dtype, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = pa.pa_cache_append_rotary(x[0].to(DEV), x[1].to(DEV), x[2].to(DEV), torch.from_numpy(slots).to(DEV), after[0], after[1],
                                      pos.to(DEV), table.to(DEV), q_out=qo, bounds=after[2], interleaved=style, pair_axis=axes,
                                      dev_err=err)
        assert r is qo and err.item() == 0
        assert (qo[-3:] == 5).all()
        _close(qo[:-3], x[0][:-3], pos[..., :-3], table, axes, style, dtype)
        _check_append(x, slots, pos, table, axes, style, dtype, bs, before, [None if a is None else a.cpu() for a in after])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hkv", [(128, 16, 16), (64, 32, 5), (64, 100, 16), (64, 16, 2), (128, 100, 5)])
def test_append_of_a_long_chunk(dtype, d, bs, hkv):
    """Enough rows for warps that look at one, four and sixteen tokens for the runs that begin
    there; runs of more than 32."""
    rng = np.random.default_rng(9)
    new = [int(n) for n in rng.integers(1, 500, 13)] + [1] * 40
    lens = [int(n) for n in rng.integers(0, 70, len(new))]
    slots, nb = _slots(lens, new, bs, rng)
    t = len(slots)
    assert {2: 0, 5: 3, 16: 12}[hkv] * 24 * 152 < t * hkv <= {2: 3, 5: 12, 16: 1000}[hkv] * 24 * 152
    slots[rng.random(t) < 0.002] = -1
    for i in range(1, t):  # padding only between requests or blocks: rows of a block follow one another
        if slots[i - 1] < 0 and slots[i] >= 0 and slots[i] % bs:
            slots[i] = -1
    g = torch.Generator().manual_seed(1)
    x = [torch.randn(t, h, d, generator=g).to(dtype) for h in (2, hkv, hkv)]
    before = _pool(g, nb, bs, hkv, d, dtype, True)
    after = [b.to(DEV) for b in before]
    table, pos = angle_table(64, d), torch.randint(0, 64, (t,), generator=g, dtype=torch.int32)
    pa.pa_cache_append_rotary(None, x[1].to(DEV), x[2].to(DEV), torch.from_numpy(slots).to(DEV), after[0], after[1], pos.to(DEV),
                              table.to(DEV), bounds=after[2])
    _check_append(x, slots, pos, table, None, False, dtype, bs, before, [a.cpu() for a in after])


def test_append_of_special_keys_without_turning():
    """NaN, infinities and zeros of both signs in keys: bounds take them as numbers do,
    NaN wins; no positions: the keys keep their bits."""
    d, bs, hkv = 64, 16, 2
    slots = np.arange(3, 3 + 40, dtype=np.int32)
    g = torch.Generator().manual_seed(2)
    x = [torch.randn(40, h, d, generator=g).to(BF16) for h in (4, hkv, hkv)]
    x[1][5, 0, 7], x[1][20, 1, 3], x[1][21, 1, 3], x[1][30, 0, :] = float("nan"), float("inf"), -float("inf"), -0.0
    x[2][9] = float("nan")
    before = _pool(g, 4, bs, hkv, d, BF16, True)
    before[2][0, 1, 0, 5] = float("nan")  # in a block that has keys already
    after = [b.to(DEV) for b in before]
    qo = pa.pa_cache_append_rotary(x[0].to(DEV), x[1].to(DEV), x[2].to(DEV), torch.from_numpy(slots).to(DEV), after[0], after[1],
                                   bounds=after[2])
    _same(qo.cpu(), x[0])
    _check_append(x, slots, None, None, None, False, BF16, bs, before, [a.cpu() for a in after])


@pytest.mark.parametrize("with_bounds", [True, False])
def test_append_refuses_slots_and_positions(with_bounds):
    d, bs, hkv, nb = 128, 16, 2, 3
    slots = np.array([0, 1, 2, nb * bs, 20, 21, 22, -1, 2**31 - 1, 40], dtype=np.int32)
    pos = torch.tensor([0, 99, 2, 3, 4, -1, 6, 500, 8, 9], dtype=torch.int32)
    g = torch.Generator().manual_seed(6)
    x = [torch.randn(10, h, d, generator=g).to(BF16) for h in (4, hkv, hkv)]
    before = _pool(g, nb, bs, hkv, d, BF16, with_bounds)
    after = [None if b is None else b.to(DEV) for b in before]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = angle_table(20, d)
    qo = torch.full((10, 4, d), 5.0, dtype=BF16, device=DEV)
    pa.pa_cache_append_rotary(x[0].to(DEV), x[1].to(DEV), x[2].to(DEV), torch.from_numpy(slots).to(DEV), after[0], after[1],
                              pos.to(DEV), table.to(DEV), q_out=qo, bounds=after[2], dev_err=err)
    assert err.item() == pa.DEVERR_OVERFLOW | pa.DEVERR_BAD_BLOCK
    refused = [1, 3, 5, 8]
    assert (qo[refused] == 0).all() and (qo[7] == 5).all()
    _check_append(x, slots, pos, table, None, False, BF16, bs, before, [None if a is None else a.cpu() for a in after], refused)


def test_append_beyond_two_to_the_31_elements():
    """Rows whose place in the pool passes 32 bits."""
    d, bs, hkv, nb = 128, 16, 8, 150000
    k, v = (torch.zeros(nb, bs, hkv, d, dtype=BF16, device=DEV) for _ in range(2))
    bounds = torch.zeros(nb, hkv, 2, d, dtype=BF16, device=DEV)
    assert k.numel() > 2**31
    slots = torch.tensor([nb * bs - 2, nb * bs - 1, 5], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 3, hkv, d, device=DEV).to(BF16)
    pa.pa_cache_append_rotary(None, x[0], x[1], slots, k, v, bounds=bounds)
    assert torch.equal(k[-1, -2:], x[0, :2]) and torch.equal(v[-1, -2:], x[1, :2]) and torch.equal(k[0, 5], x[0, 2])
    assert torch.equal(bounds[-1, :, 1], torch.maximum(x[0, :2].amax(0), torch.zeros_like(x[0, 0])))
    assert int((k != 0).any(-1).any(-1).sum()) == 3

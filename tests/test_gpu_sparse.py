"""pa_select_blocks and pa_sparse on the GPU against the plain reference, and the step
that they and pa_cache_append_rotary make up."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import sparse as ref
from tests.sparse_util import BF16, F32, angle_table, attend_bound, f64, make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _bounds(seed, nb, hkv, d, dtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    mid, a, b = (torch.randn(nb, hkv, d, generator=g) for _ in range(3))
    return torch.stack([mid - spread * a.abs(), mid + spread * b.abs()], 2).to(dtype)


def _table(rng, blocks, width, nb):
    perm = rng.permutation(nb)
    table, at = np.full((len(blocks), width), -1, dtype=np.int32), 0
    for r, n in enumerate(blocks):
        table[r, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table)


def _select(q, bounds, table, lens, top, bs, first=1, last=1, cu=None, dev_err=None):
    got = torch.full((q.shape[0], bounds.shape[1], top), -9, dtype=torch.int32, device=DEV)
    r = pa.pa_select_blocks(q.to(DEV), bounds.to(DEV), table.to(DEV), lens.to(DEV), top, bs, first_blocks=first, last_blocks=last,
                            cu_seq_lens_q=None if cu is None else cu.to(DEV), selected=got, dev_err=dev_err)
    assert r is got
    return got.cpu().numpy()


def _want(q, bounds, table, lens, top, bs, first=1, last=1, cu=None):
    return ref.select(f64(q), f64(bounds), table.numpy(), lens.numpy(), top, bs, first, last, None if cu is None else cu.numpy())


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 8, 1), (128, 32, 14, 2), (64, 16, 3, 3), (64, 32, 10, 5), (128, 16, 32, 8), (64, 7, 6, 1)])
@pytest.mark.parametrize("top,first,last", [(2, 1, 1), (9, 1, 1), (16, 0, 0), (64, 3, 2), (5, 0, 1), (7, 4, 3)])
def test_select_for_single_tokens(dtype, d, bs, hq, hkv, top, first, last):
    lens = [1, bs, 5 * bs + 1, 40 * bs, 17 * bs + 3, 300 * bs - 1, 0]
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks) + 3
    rng = np.random.default_rng(top)
    table = _table(rng, blocks, max(blocks) + 2, nb)
    bounds = _bounds(top + d, nb, hkv, d, dtype)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(top)).to(dtype)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _select(q, bounds, table, i32(lens), top, bs, first, last, dev_err=err)
    assert err.item() == 0
    assert np.array_equal(got, _want(q, bounds, table, i32(lens), top, bs, first, last))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 8, 2), (64, 32, 7, 1), (128, 16, 3, 3), (64, 16, 8, 1)])
@pytest.mark.parametrize("top", [3, 33])
def test_select_for_chunks(dtype, d, bs, hq, hkv, top):
    """Requests with chunks, single tokens and none; queries before the first key;
    rows behind the last request, left as they were."""
    new, lens = [5, 0, 1, 37, 3], [100 * bs + 3, 50, 77 * bs, 37, 2]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks)
    table = _table(np.random.default_rng(1), blocks, max(blocks), nb)
    bounds = _bounds(5, nb, hkv, d, dtype)
    q = torch.randn(int(cu[-1]) + 4, hq, d, generator=torch.Generator().manual_seed(8)).to(dtype)
    got = _select(q, bounds, table, i32(lens), top, bs, cu=torch.from_numpy(cu))
    want = _want(q, bounds, table, i32(lens), top, bs, cu=torch.from_numpy(cu))
    assert (want[43] == -1).all()  # the first of three queries over two keys
    assert np.array_equal(got[:cu[-1]], want[:cu[-1]])
    assert (got[cu[-1]:] == -9).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hq,hkv,first,last", [(64, 16, 32, 8, 1, 1), (128, 16, 24, 24, 0, 2), (64, 32, 36, 18, 2, 0), (128, 16, 48, 16, 1, 1),
                                                    (64, 16, 40, 8, 1, 1), (128, 32, 64, 8, 0, 0)])
@pytest.mark.parametrize("tokens", [800, 210, 1500])
def test_select_for_tiles_of_tokens(dtype, d, bs, hq, hkv, first, last, tokens):
    """Enough tokens a request for CTAs that take up to 16 of them: requests that end
    inside a tile, single tokens between, queries before the first key, rows whose blocks
    all fit, one request with a bad entry, rows behind the last request; heads in every
    packing of eight columns."""
    top = 9
    part = tokens // 5
    new = [part + 3, 0, 1, 2 * part, 17, part - 21, 16]
    lens = [60 * bs + 5, 40, 33 * bs, 2 * part - 5, 21 * bs - 1, 25 * bs + part, 50 * bs]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks)
    table = _table(np.random.default_rng(1), blocks, max(blocks) + 1, nb)
    bounds = _bounds(5, nb, hkv, d, dtype)
    q = torch.randn(int(cu[-1]) + 5, hq, d, generator=torch.Generator().manual_seed(8)).to(dtype)
    want = _want(q, bounds, table, i32(lens), top, bs, first, last, torch.from_numpy(cu))
    broken = table.clone()
    broken[6, 20] = nb + 7
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _select(q, bounds, broken, i32(lens), top, bs, first, last, torch.from_numpy(cu), err)
    assert err.item() == pa.DEVERR_BAD_BLOCK
    assert np.array_equal(got[:cu[6]], want[:cu[6]])
    assert (got[cu[6]:cu[7]] == -1).all() and (got[cu[7]:] == -9).all()
    # an entry that only a request's later tokens need fails theirs alone
    broken = table.clone()
    broken[5, 30] = -1
    got = _select(q, bounds, broken, i32(lens), top, bs, first, last, torch.from_numpy(cu), err)
    rows = np.array([r == 5 and p // bs - last >= 30 for r, p in ref.query_positions(lens, cu)])
    assert (bs == 32 or part < 60 or rows.any()) and not rows.all()
    assert (got[:cu[7]][rows] == -1).all() and np.array_equal(got[:cu[7]][~rows], want[:cu[7]][~rows])
    for bad in ([1] + cu[1:].tolist(), cu[:3].tolist() + [cu[-1] + 3] + cu[4:].tolist()):
        err.zero_()
        _select(q, bounds, table, i32(lens), top, bs, first, last, i32(bad), err)
        assert err.item() & pa.DEVERR_BAD_CU  # (rows may be taken for another request's, and fail as such)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,most", [(75, 9), (1100, 6), (40, 60)])
def test_select_for_tiles_of_many_requests(dtype, batch, most):
    """More requests than a warp looks at in one step; with nothing, one token or chunks, and
    a token behind the last that belongs to none."""
    d, bs, top, hkv = 64, 16, 4, 2
    rng = np.random.default_rng(batch)
    new = rng.integers(0, most + 1, batch)
    new[rng.random(batch) < 0.1] = 0
    lens = new + rng.integers(0, 300, batch)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    assert cu[-1] >= 2 * batch
    nb = 500
    table = torch.from_numpy(rng.integers(0, nb, (batch, 25)).astype(np.int32))
    bounds = _bounds(5, nb, hkv, d, dtype)
    q = torch.randn(int(cu[-1]) + 1, 6, d, generator=torch.Generator().manual_seed(8)).to(dtype)
    lens = torch.from_numpy(lens.astype(np.int32))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _select(q, bounds, table, lens, top, bs, cu=torch.from_numpy(cu), dev_err=err)
    assert err.item() == 0 and (got[-1] == -9).all()
    assert np.array_equal(got[:-1], _want(q, bounds, table, lens, top, bs, cu=torch.from_numpy(cu))[:-1])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,width", [(137, 90), (271, 200), (271, 120), (541, 90), (547, 40)])
@pytest.mark.parametrize("d,group,packed", [(64, 3, False), (128, 8, False), (64, 1, True), (128, 4, True)])
def test_select_of_many_rows(dtype, batch, width, d, group, packed):
    """Rows enough for four, two and one warps each, in numbers that leave places empty:
    short and long ones side by side, close scores, a row with a bad entry and one with a bad length, rows of
    requests left out; as packed queries, some requests without any and rows behind the last."""
    bs, hkv, top = 16, 3, 7
    assert (batch * hkv) % 8 != 0
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, width * bs + 1, batch).astype(np.int32)
    lens[5], lens[9], lens[12], lens[20] = pa.PA_LEFT_OUT, width * bs, width * bs, 1
    nb = 300
    table = rng.integers(0, nb, (batch, width)).astype(np.int32)
    bounds = _bounds(5, nb, hkv, d, dtype)
    bounds[: nb // 2] = bounds[nb // 2:]  # scores that are equal
    cu = new = None
    if packed:
        new = np.ones(batch, dtype=np.int64)
        new[[3, 30, batch - 1]] = 0
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    q = torch.randn(batch, hkv * group, d, generator=torch.Generator().manual_seed(8)).to(dtype)
    tokens = batch if cu is None else int(cu[-1])
    want = np.full((batch, hkv, top), -9, dtype=np.int32)
    clean = np.where(lens < 0, 0, lens)
    want[:tokens] = _want(q[:tokens], bounds, torch.from_numpy(table), torch.from_numpy(clean), top, bs, cu=cu)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _select(q, bounds, torch.from_numpy(table), torch.from_numpy(lens), top, bs, cu=cu, dev_err=err)
    assert err.item() == 0 and np.array_equal(got, want)
    table[9, width // 2], lens[12] = nb, width * bs + 1
    rows = np.arange(batch) if cu is None else np.cumsum(new) - 1
    want[rows[9]], want[rows[12]] = -1, -1
    got = _select(q, bounds, torch.from_numpy(table), torch.from_numpy(lens), top, bs, cu=cu, dev_err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK | pa.DEVERR_OVERFLOW
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,hkv,part", [(3, 2, 25), (2, 1, 70), (5, 3, 4), (2, 2, 9)])
def test_select_for_tiles_on_clusters(dtype, batch, hkv, part):
    """Few tiles of tokens over long contexts: a cluster of CTAs for each, in which the first
    chooses; tiles that hold nothing among them."""
    d, bs, top = 64, 16, 40
    new = [part - 3 * r % 4 for r in range(batch)]
    new[-1] = 0 if batch > 2 else new[-1]
    lens = [(300 + 90 * r) * bs - 5 for r in range(batch)]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks)
    table = _table(np.random.default_rng(1), blocks, 900, nb)
    bounds = _bounds(5, nb, hkv, d, dtype)
    q = torch.randn(int(cu[-1]) + 2, 4 * hkv, d, generator=torch.Generator().manual_seed(8)).to(dtype)
    got = _select(q, bounds, table, i32(lens), top, bs, cu=torch.from_numpy(cu))
    want = _want(q, bounds, table, i32(lens), top, bs, cu=torch.from_numpy(cu))
    assert np.array_equal(got[:cu[-1]], want[:cu[-1]]) and (got[cu[-1]:] == -9).all()
    table[0, 100] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _select(q, bounds, table, i32(lens), top, bs, cu=torch.from_numpy(cu), dev_err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK and (got[:cu[1]] == -1).all() and np.array_equal(got[cu[1]:cu[-1]], want[cu[1]:cu[-1]])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_among_equal_and_nearly_equal_scores(dtype):
    """Blocks whose scores are equal (ties: the lowest block) or differ by less than the
    rounding of an fp32 sum; the exact scores decide."""
    d, bs, n, top = 128, 16, 400, 60
    rng = np.random.default_rng(4)
    base = _bounds(1, 1, 1, d, dtype)
    bounds = base.repeat(n, 1, 1, 1).clone()
    table = torch.from_numpy(rng.permutation(n).astype(np.int32)).view(1, n)
    q = torch.randn(1, 8, d, generator=torch.Generator().manual_seed(3)).to(dtype)
    assert np.array_equal(_select(q, bounds, table, i32([n * bs]), top, bs),
                          np.array([0] + list(range(1, top - 1)) + [n - 1]).reshape(1, 1, top))
    # one channel that contributes less than 2^-24 of the sum moves by steps
    tiny = torch.zeros(1, 8, d)
    tiny[0, :, 0] = 2.0 ** -20
    tiny[0, :, 1:] = torch.randn(8, d - 1, generator=torch.Generator().manual_seed(5)).abs() + 1
    q = tiny.to(dtype)
    bounds[:, 0, 1, 0] = torch.from_numpy(rng.integers(1, 200, n)).to(dtype) * 2.0 ** -6
    got, want = _select(q, bounds, table, i32([n * bs]), top, bs), _want(q, bounds, table, i32([n * bs]), top, bs)
    assert np.array_equal(got, want)
    # and all scores 0
    assert np.array_equal(_select(q, bounds * 0, table, i32([n * bs]), top, bs).ravel(), [0] + list(range(1, top - 1)) + [n - 1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_with_many_close_scores(dtype):
    """Scores in a narrow band far from 0: most of the blocks are within the error of
    the fp32 sums of the last one taken."""
    d, bs, n, top = 64, 16, 3000, 700
    bounds = _bounds(2, n, 2, d, dtype, spread=0.0) * 2.0 ** -12 + 4
    bounds = bounds.to(dtype)
    if dtype == BF16:  # bf16 numbers about 4 are 2^-6 apart: two channels carry the difference
        bounds[:, :, :, :2] = (_bounds(3, n, 2, d, F32)[:, :, :, :2] * 2.0 ** -14).to(dtype)
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2)).int().view(1, n)
    q = (torch.randn(1, 4, d, generator=torch.Generator().manual_seed(7)).abs() * 3 + 2).to(dtype)
    assert np.array_equal(_select(q, bounds, table, i32([n * bs]), top, bs), _want(q, bounds, table, i32([n * bs]), top, bs))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_select_with_nan_and_infinite_bounds(dtype):
    """NaN ranks above all numbers, infinities as they are; in the queries as well."""
    d, bs, n, top, hkv = 64, 16, 90, 11, 2
    bounds = _bounds(1, n, hkv, d, dtype)
    bounds[7, 0, 1, 3], bounds[50, 1, 0, 9] = float("nan"), float("nan")
    bounds[12, 0, 1, :], bounds[13, 1, 1, 4], bounds[60, 0, 0, 5] = float("inf"), float("inf"), -float("inf")
    table = torch.arange(n, dtype=torch.int32).view(1, n).repeat(4, 1)
    q = torch.randn(4, 6, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    q[1, 2] = 0  # 0 times an infinity
    q[2, 0, 5] = float("nan")
    q[3, 4, 6] = float("inf")
    lens = i32([n * bs] * 4)
    assert np.array_equal(_select(q, bounds, table, lens, top, bs), _want(q, bounds, table, lens, top, bs))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [1, 19])
@pytest.mark.parametrize("nans", [1, 3, 20, 40, 300])
def test_select_where_the_last_chosen_is_nan(dtype, tokens, nans):
    """The keys of NaN are the largest 32-bit numbers: nothing is added to them."""
    d, bs, n, hkv = 64, 16, 600, 2
    bounds = _bounds(1, n, hkv, d, dtype)
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2)).int().view(1, n)
    some = np.random.default_rng(nans).permutation(n)[:nans]
    bounds[some, 0, 0, 2] = float("nan")
    bounds[some, 1, 1, 60] = float("inf")
    q = torch.randn(tokens, 6, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    lens, cu = i32([n * bs - 3]), i32([0, tokens])
    for top in (2 + nans // 2, 3 + nans // 2, nans, nans + 1, nans + 2, nans + 3, nans + 9):
        if top >= 2:
            assert np.array_equal(_select(q, bounds, table, lens, top, bs, cu=cu), _want(q, bounds, table, lens, top, bs, cu=cu)), top


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [1, 19])
@pytest.mark.parametrize("head", [0, 2])
@pytest.mark.parametrize("step", [2.0 ** -14, 2.0 ** -9])
def test_select_of_close_scores_beside_an_infinite_head(dtype, tokens, head, step):
    """A head whose scores are all minus infinity takes nothing from the others, whose
    scores are in doubt."""
    d, bs, n, hkv = 64, 16, 500, 2
    bounds = torch.full((n, hkv, 2, d), 4.0)
    bounds[:, :, :, :2] = _bounds(3, n, hkv, d, F32)[:, :, :, :2] * step
    bounds[:, :, :, 7] = -1
    bounds = bounds.to(dtype)
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2)).int().view(1, n)
    q = (torch.randn(tokens, 6, d, generator=torch.Generator().manual_seed(1)).abs() * 3 + 2).to(dtype)
    q[:, head, 7] = float("inf")
    lens, cu = i32([n * bs - 3]), i32([0, tokens])
    for top in (5, 40, 300):
        assert np.array_equal(_select(q, bounds, table, lens, top, bs, cu=cu), _want(q, bounds, table, lens, top, bs, cu=cu)), top


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hq,hkv", [(64, 6, 2), (128, 8, 1), (64, 2, 2), (128, 10, 2)])
def test_select_for_tiles_with_nan_infinite_and_close_scores(dtype, d, hq, hkv):
    """The same in tiles of tokens, with heads of every number; scores of a narrow band, few and
    many of them in doubt."""
    bs, n, tokens = 16, 500, 43
    bounds = _bounds(1, n, hkv, d, dtype)
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2)).int().view(1, n)
    g = torch.Generator().manual_seed(1)
    q = torch.randn(tokens, hq, d, generator=g).to(dtype)
    lens, cu = i32([n * bs - 3]), i32([0, tokens])
    bounds[7, 0, 1, 3], bounds[50, hkv - 1, 0, 9] = float("nan"), float("nan")
    bounds[12, 0, 1, :], bounds[13, hkv - 1, 1, 4], bounds[60, 0, 0, 5] = float("inf"), float("inf"), -float("inf")
    q[3, 1], q[9, 0, 5], q[20, hq - 1, 6] = 0, float("nan"), float("inf")
    for top in (5, 90):
        assert np.array_equal(_select(q, bounds, table, lens, top, bs, cu=cu), _want(q, bounds, table, lens, top, bs, cu=cu))
    for step in (2.0 ** -14, 2.0 ** -9):
        close = torch.full((n, hkv, 2, d), 4.0)
        close[:, :, :, :2] = _bounds(3, n, hkv, d, F32)[:, :, :, :2] * step
        close = close.to(dtype)
        q = (torch.randn(tokens, hq, d, generator=g).abs() * 3 + 2).to(dtype)
        for top in (40, 300):
            assert np.array_equal(_select(q, close, table, lens, top, bs, cu=cu), _want(q, close, table, lens, top, bs, cu=cu))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (F32, 64)])
@pytest.mark.parametrize("n,top", [(49152, 1000), (20000, 19999), (49150, 3)])
def test_select_from_as_many_blocks_as_there_can_be(dtype, d, n, top):
    bs = 16
    bounds = _bounds(1, 3000, 1, d, dtype)  # blocks appear many times: whole runs of ties
    table = torch.randint(0, 3000, (2, 49152), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    q = torch.randn(2, 2, d, generator=torch.Generator().manual_seed(2)).to(dtype)
    lens = i32([n * bs, n * bs - 5])
    assert np.array_equal(_select(q, bounds, table, lens, top, bs), _want(q, bounds, table, lens, top, bs))


@pytest.mark.parametrize("rows", [1, 4, 9, 19, 28, 38, 45, 60, 76, 100, 200])
def test_select_is_the_same_for_every_split(rows):
    """As many CTAs a row as the number of rows allows: one to sixteen of them."""
    d, bs, n, top = 64, 16, 700, 50
    bounds = _bounds(1, n, 1, d, BF16)
    table = torch.randperm(n, generator=torch.Generator().manual_seed(2)).int().view(1, n).repeat(rows, 1)
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(3)).to(BF16).repeat(rows, 1, 1)
    lens = i32([n * bs] * rows)
    got = _select(q, bounds, table, lens, top, bs)
    assert (got == _want(q[:1], bounds, table[:1], lens[:1], top, bs)).all()


def test_select_refuses_what_the_device_sees():
    d, bs, n, top = 64, 16, 30, 5
    bounds = _bounds(1, n, 1, d, BF16)
    q = torch.randn(8, 2, d).to(BF16)
    table = torch.arange(n, dtype=torch.int32).view(1, n).repeat(8, 1)
    table[1, 9], table[2, 4] = -1, n
    table[3, 0], table[4, 29] = -1, 2**31 - 1  # of first and last blocks the entries are not read
    lens = i32([n * bs, n * bs, n * bs, n * bs, n * bs, n * bs + 1, -3, pa.PA_LEFT_OUT])
    want = _want(q[:1], bounds, table[:1], lens[:1], top, bs)[0]
    for rows, bits in (([0, 3, 4, 7], 0), ([1], pa.DEVERR_BAD_BLOCK), ([2], pa.DEVERR_BAD_BLOCK), ([5], pa.DEVERR_OVERFLOW),
                       ([6], pa.DEVERR_OVERFLOW)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = _select(q[:1].repeat(len(rows), 1, 1), bounds, table[rows], lens[rows], top, bs, dev_err=err)
        assert err.item() == bits
        for r, g in zip(rows, got):
            assert np.array_equal(g, want if r in (0, 3, 4) else np.full_like(want, -1))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _select(q[:6], bounds, table[[0, 0, 0]], lens[[0, 0, 0]], top, bs, cu=i32([2, 3, 1, 6]), dev_err=err)
    assert err.item() == pa.DEVERR_BAD_CU and (got[:2] == -1).all()


# ------------------------------------------------------------------ attention
def _random_choice(rng, lens, hkv, bs, top, cu=None):
    rows = ref.query_positions(lens, cu)
    out = np.full((len(rows), hkv, top), -1, dtype=np.int32)
    for t, (_, pos) in enumerate(rows):
        n = max(0, pos // bs + 1)
        for h in range(hkv):
            some = rng.permutation(n)[:top]
            out[t, h, :len(some)] = np.sort(some)
    return out


def _attend(c, q, sel, scale=0.0, cu=None, dev_err=None, out=None):
    up = lambda x: x.to(DEV) if isinstance(x, torch.Tensor) else torch.from_numpy(x).to(DEV)  # noqa: E731
    return pa.pa_sparse(up(q), up(c["k"]), up(c["v"]), up(c["table"]), up(c["lens"]), up(sel),
                        cu_seq_lens_q=None if cu is None else up(cu), softmax_scale=scale, dev_err=dev_err, out=out)


def _check(got, c, q, sel, scale=None, cu=None):
    d = q.shape[2]
    rows = q.shape[0] if cu is None else int(cu[-1])
    want, info = ref.attend(f64(q), f64(c["k"]), f64(c["v"]), c["table"].numpy(), c["lens"].numpy(), sel, scale or d ** -0.5, cu)
    err, bound = np.abs(f64(got) - want)[:rows], attend_bound(want, info, d, q.dtype)[:rows]
    assert np.isfinite(f64(got)[:rows]).all()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 8, 1), (128, 32, 14, 2), (64, 16, 3, 3), (64, 32, 10, 5), (128, 48, 6, 2), (64, 16, 32, 4)])
@pytest.mark.parametrize("top", [1, 3, 20, 90])
def test_sparse_for_single_tokens(dtype, d, bs, hq, hkv, top):
    lens = [1, bs, 5 * bs + 1, 30 * bs, 17 * bs + 3, 0, 2]
    rng = np.random.default_rng(top)
    c = make_cache(top, lens, hkv, d, bs, dtype, gain=1.5)
    q = torch.randn(len(lens), hq, d, generator=torch.Generator().manual_seed(d)).to(dtype)
    sel = _random_choice(rng, lens, hkv, bs, top)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _attend(c, q, sel, dev_err=err)
    assert err.item() == 0
    _check(got, c, q, sel)
    assert (got[5] == 0).all()


@pytest.mark.parametrize("d,bs", [(64, 1), (64, 7), (128, 20), (64, 33)])
def test_sparse_with_blocks_of_any_size_in_fp32(d, bs):
    """Blocks that are no whole number of the kernel's units of tokens."""
    lens = [1, bs, 5 * bs + 1, 30 * bs, 17 * bs + bs // 2, 9]
    c = make_cache(bs, lens, 2, d, bs, F32)
    q = torch.randn(len(lens), 6, d, generator=torch.Generator().manual_seed(d)).to(F32)
    for top in (2, 40):
        sel = _random_choice(np.random.default_rng(top), lens, 2, bs, top)
        _check(_attend(c, q, sel), c, q, sel)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 8, 2), (64, 32, 7, 1), (128, 16, 3, 3)])
def test_sparse_for_chunks(dtype, d, bs, hq, hkv):
    new, lens = [5, 0, 1, 21, 3], [20 * bs + 3, 50, 7 * bs, 21, 2]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    c = make_cache(1, lens, hkv, d, bs, dtype)
    q = torch.randn(int(cu[-1]) + 3, hq, d, generator=torch.Generator().manual_seed(8)).to(dtype)
    sel = _random_choice(np.random.default_rng(2), lens, hkv, bs, 6, cu)
    sel = np.concatenate([sel, np.zeros((3, hkv, 6), dtype=np.int32)])
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    got = _attend(c, q, sel, cu=cu, out=out)
    _check(got, c, q, sel, cu=cu)
    assert (got[int(cu[-1]):] == 7).all() and (got[27] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_lists_of_any_kind(dtype):
    """Unordered lists, entries of nothing between, blocks behind the query, a block twice,
    an empty list, a scale of the caller's."""
    d, bs, hkv = 64, 32, 2
    lens = [200, 70, 129, 33]
    c = make_cache(4, lens, hkv, d, bs, dtype, width=9)
    q = torch.randn(4, 6, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    sel = np.full((4, hkv, 7), -1, dtype=np.int32)
    sel[0, 0], sel[0, 1] = [6, -1, 2, 5, -7, 0, 3], [4, 4, 1, -1, -1, 1, 4]
    sel[1, 0, 5:], sel[1, 1] = [2, 1], [8, 3, 2, 2**31 - 1, 100, 0, -2**31]
    sel[2, 0, 3] = 4
    for scale in (0.0, 0.7):
        got = _attend(c, q, sel, scale)
        seen = sel.copy()
        seen[1, 1, [0, 1, 3, 4]] = -1
        _check(got, c, q, seen, scale or None)
        assert (got[3] == 0).all() and (got[2, 3:] == 0).all() and (got[2, :3] != 0).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,top", [(1, 300), (3, 129), (10, 64), (28, 300), (40, 64), (90, 64), (120, 40), (150, 64), (200, 40), (400, 40)])
def test_sparse_for_every_split(dtype, rows, top):
    """One to sixteen CTAs a row; lists longer than a warp looks up at once."""
    d, bs = 64, 16
    n = 320
    c = make_cache(7, [n * bs - 3], 1, d, bs, dtype)
    c["table"], c["lens"] = c["table"].repeat(rows, 1), c["lens"].repeat(rows)
    q = torch.randn(1, 8, d, generator=torch.Generator().manual_seed(2)).to(dtype).repeat(rows, 1, 1)
    sel = _random_choice(np.random.default_rng(3), [n * bs - 3], 1, bs, top)
    got = _attend(c, q, np.repeat(sel, rows, 0))
    assert torch.equal(got, got[:1].expand_as(got))
    c["table"], c["lens"] = c["table"][:1], c["lens"][:1]
    _check(got[:1], c, q[:1], sel)


@pytest.mark.parametrize("d,hkv,rows", [(128, 1, 913), (128, 3, 307), (64, 8, 761), (64, 5, 1217)])
def test_sparse_of_many_rows(d, hkv, rows):
    """Two rows a CTA: an odd number of them, lists of different lengths side by side,
    rows without anything, a bad entry in one, rows behind the last request."""
    assert rows * hkv >= (6 if d == 128 else 40) * 152 and rows % 2 == 1
    bs, lens = 16, [90, 333, 17, 0]
    c = make_cache(11, lens, hkv, d, bs, BF16, width=21)
    pick = np.arange(rows) % 4
    big = dict(c, table=c["table"][pick].clone(), lens=c["lens"][pick].clone())
    q = torch.randn(rows, 2 * hkv, d, generator=torch.Generator().manual_seed(1)).to(BF16)
    sel = _random_choice(np.random.default_rng(5), [lens[i] for i in pick], hkv, bs, 9)
    sel[4:8, 0] = -1
    big["table"][1, :] = -1  # the second request's first row
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _attend(big, q, sel, dev_err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK and (got[1] == 0).all() and (got[3::4] == 0).all()
    rest = np.setdiff1d(np.arange(rows)[:40], [1])
    _check(got[rest], dict(big, table=big["table"][rest], lens=big["lens"][rest]), q[rest], sel[rest])
    last = np.arange(rows - 9, rows)
    _check(got[last], dict(big, table=big["table"][last], lens=big["lens"][last]), q[last], sel[last])
    # the same rows as packed queries of one request: all see its last positions
    n = rows - 2
    one = dict(c, table=c["table"][1:2], lens=i32([n + 20 * bs]))
    one["table"] = torch.nn.functional.pad(one["table"], (0, n // bs + 2), value=0)
    sel2 = np.tile(_random_choice(np.random.default_rng(6), [300], hkv, bs, 9), (rows, 1, 1))
    out = torch.full(q.shape, 3.0, dtype=BF16, device=DEV)
    got = _attend(one, q, sel2, cu=np.array([0, n], dtype=np.int32), out=out)
    assert (got[n:] == 3).all()
    _check(got[:30], dict(one, lens=i32([n + 20 * bs - n + 30])), q[:30], sel2[:30], cu=np.array([0, 30], dtype=np.int32))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_of_a_list_beyond_one_look_up(dtype):
    d, bs, top = 64, 16, 16 * 4 * 64 * 2 + 77  # three look-ups of sixteen CTAs' warps
    c = make_cache(7, [16], 1, d, bs, dtype, width=top)
    c["table"][0, :] = c["table"][0, 0]
    c["lens"][0] = top * bs - 9
    q = torch.randn(1, 2, d, generator=torch.Generator().manual_seed(2)).to(dtype)
    sel = np.arange(top, dtype=np.int32)[::-1].copy().reshape(1, 1, top)
    got = _attend(c, q, sel)
    # the same block over and over, the last one less nine keys
    k, v = (f64(c[x])[c["table"][0, 0]][:, 0] for x in "kv")
    s = f64(q)[0] @ k.T * d ** -0.5
    w = np.exp(s - s.max(1, keepdims=True)) * np.where(np.arange(bs) < bs - 9, top, top - 1)
    want = ((w @ v) / w.sum(1, keepdims=True))[None]
    info = np.array([[[d ** -0.5 * (np.abs(f64(q)[0]) @ np.abs(k).T).max(), np.abs(v).max(), top * bs]]])
    assert (np.abs(f64(got) - want) <= attend_bound(want, info, d, dtype)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_special_values(dtype):
    """NaN in unused slots counts nothing (make_cache leaves it there); a NaN or infinity
    that is seen reaches the outputs of its rows and no others."""
    d, bs, hkv = 128, 16, 2
    c = make_cache(3, [70, 70, 70], hkv, d, bs, dtype)
    q = torch.randn(3, 4, d, generator=torch.Generator().manual_seed(1)).to(dtype)
    sel = np.tile(np.arange(5, dtype=np.int32), (3, hkv, 1))
    clean = _attend(c, q, sel)
    _check(clean, c, q, sel)
    c["k"][c["table"][0, 1], 3, 0, 5] = float("nan")
    c["v"][c["table"][1, 4], 5, 1, 7] = float("inf")
    q[2, 3, 9] = float("nan")
    got = _attend(c, q, sel)
    assert torch.isnan(got[0, :2]).all() and torch.equal(got[0, 2:], clean[0, 2:])
    # a bf16 weight is the sum of two numbers, the second of either sign or 0: w * inf may be NaN
    assert (torch.isinf(got[1, 2:, 7]) if dtype == F32 else ~torch.isfinite(got[1, 2:, 7])).all() and torch.isnan(got[2, 3]).all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[0, :2], keep[1, 2:, 7], keep[2, 3] = False, False, False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_of_large_scores(dtype):
    """Scores of some hundreds: one key takes all of the weight."""
    d, bs = 64, 16
    c = make_cache(5, [200], 1, d, bs, dtype, gain=30.0)
    q = (torch.randn(1, 8, d, generator=torch.Generator().manual_seed(1)) * 20).to(dtype)
    sel = np.arange(13, dtype=np.int32).reshape(1, 1, 13)
    s = f64(q)[0] @ np.concatenate(f64(c["k"])[c["table"][0, :13]])[:200, 0].T * d ** -0.5
    assert np.abs(s).max() > 500
    got = f64(_attend(c, q, sel))[0]
    v = np.concatenate(f64(c["v"])[c["table"][0, :13]])[:200, 0]
    best = np.sort(s, 1)
    for g in range(8):
        if best[g, -1] - best[g, -2] > 40:  # e^-40 is below every rounding
            assert np.array_equal(got[g], v[s[g].argmax()])
    assert (best[:, -1] - best[:, -2] > 40).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sparse_refuses_what_the_device_sees(dtype):
    d, bs, n = 64, 16, 10
    c = make_cache(5, [n * bs - 2] * 6, 1, d, bs, dtype)
    q = torch.randn(6, 2, d).to(dtype)
    sel = np.tile(np.array([0, 3, 9], dtype=np.int32), (6, 1, 1))
    clean = _attend(c, q, sel)
    _check(clean, c, q, sel)
    c["table"][0, 5], c["table"][1, 3], c["table"][2, 9] = -1, -1, 10**6  # entry 5 is not needed
    c["lens"][3], c["lens"][4], c["lens"][5] = n * bs + 1, -5, pa.PA_LEFT_OUT
    for r, bits in enumerate((0, pa.DEVERR_BAD_BLOCK, pa.DEVERR_BAD_BLOCK, pa.DEVERR_OVERFLOW, pa.DEVERR_OVERFLOW, 0)):
        one = dict(c, table=c["table"][r:r + 1], lens=c["lens"][r:r + 1])
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = _attend(one, q[r:r + 1], sel[r:r + 1], dev_err=err)
        assert err.item() == bits
        assert torch.equal(got[0], clean[0]) if r == 0 else (got == 0).all()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = _attend(dict(c, table=c["table"][:2], lens=c["lens"][:2]), q, sel, cu=np.array([1, 3, 2], dtype=np.int32), dev_err=err,
                  out=torch.full(q.shape, 3.0, dtype=dtype, device=DEV))
    assert err.item() & pa.DEVERR_BAD_CU and (got[0] == 0).all() and (got[3:] == 3).all()


def test_sparse_beyond_two_to_the_31_elements():
    d, bs, hkv, nb = 128, 16, 8, 150000
    k, v = (torch.zeros(nb, bs, hkv, d, dtype=BF16, device=DEV) for _ in range(2))
    assert k.numel() > 2**31
    k[-1], v[-1] = torch.randn(bs, hkv, d), torch.randn(bs, hkv, d)
    q = torch.randn(1, 8 * hkv, d).to(BF16).to(DEV)
    table = torch.tensor([[0, nb - 1]], dtype=torch.int32, device=DEV)
    sel = torch.ones(1, hkv, 1, dtype=torch.int32, device=DEV)
    out = pa.pa_sparse(q, k, v, table, torch.tensor([32], dtype=torch.int32, device=DEV), sel)
    c = dict(k=k[-1:].cpu(), v=v[-1:].cpu(), table=i32([[0]]), lens=i32([16]))
    _check(out, c, q.cpu(), np.zeros((1, hkv, 1), dtype=np.int32))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,d,bs", [(BF16, 128, 16), (BF16, 64, 32), (F32, 64, 16)])
def test_serving_steps(dtype, d, bs):
    """Prompts, then steps with new tokens, chunks, pauses and ends: tables on the GPU,
    rotated append with bounds, selection, attention over it.  The cache and its bounds
    are followed by the plain reference step by step; with every block selected the
    outputs are those of dense attention."""
    rng = np.random.default_rng(1)
    hq, hkv, nb, mb, b, top = 8, 2, 120, 24, 5, 6
    table = torch.full((b, mb), -1, dtype=torch.int32, device=DEV)
    free, count = torch.arange(nb, dtype=torch.int32, device=DEV), torch.tensor([nb], dtype=torch.int32, device=DEV)
    lens = torch.zeros(b, dtype=torch.int32, device=DEV)
    k_cache, v_cache = (torch.full((nb, bs, hkv, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    bounds = torch.full((nb, hkv, 2, d), float("nan"), dtype=dtype, device=DEV)
    angles = angle_table(mb * bs, d).to(DEV)
    g = torch.Generator().manual_seed(3)
    steps = [[100, 37, 1, 16, 7 * bs], [1, 1, 1, 1, 1], [1, 0, 30, 1, 5], [-1, 1, 1, 1, 0], [50, 1, bs, 1, 1]]
    for new in steps:
        before = lens.cpu().numpy()
        tokens = sum(max(n, 0) for n in new)
        slots = torch.empty(tokens + 2, dtype=torch.int32, device=DEV)
        n = torch.tensor(new, dtype=torch.int32, device=DEV)
        cu, _, _ = pa.pa_block_tables(lens, n, table, free, count, slots, bs, seqlens_k=lens)
        q, k, v = torch.randn(tokens + 2, hq + 2 * hkv, d, generator=g).to(dtype).to(DEV).split([hq, hkv, hkv], 1)
        pos = np.concatenate([np.arange(before[r], before[r] + m) for r, m in enumerate(new) if m > 0] + [[0, 0]])
        q_out = torch.zeros(q.shape, dtype=dtype, device=DEV)
        pa.pa_cache_append_rotary(q, k, v, slots, k_cache, v_cache, torch.from_numpy(pos).int().to(DEV), angles, q_out=q_out,
                                  bounds=bounds)
        sel = pa.pa_select_blocks(q_out, bounds, table, lens, top, bs, cu_seq_lens_q=cu,
                                  selected=torch.full((tokens + 2, hkv, top), -1, dtype=torch.int32, device=DEV))
        out = pa.pa_sparse(q_out, k_cache, v_cache, table, lens, sel, cu_seq_lens_q=cu)
        c = dict(k=k_cache.cpu(), v=v_cache.cpu(), table=table.cpu(), lens=lens.cpu(), bounds=bounds.cpu())
        now = lens.cpu().numpy()
        for r in range(b):  # bounds are those of the keys that are there
            for j in range(-(-int(now[r]) // bs)):
                p, rows = int(c["table"][r, j]), min(bs, int(now[r]) - j * bs)
                lo, hi = ref.bounds_of(f64(c["k"])[p, :rows])
                assert np.array_equal(f64(c["bounds"])[p, :, 0], lo) and np.array_equal(f64(c["bounds"])[p, :, 1], hi)
        cu_h = cu.cpu().numpy()
        got_sel = sel.cpu().numpy()
        # bounds of blocks that later tokens of the same chunk are in: as they stand after the step
        assert np.array_equal(got_sel[:tokens], _want(q_out.cpu(), c["bounds"], c["table"], c["lens"], top, bs, cu=cu.cpu())[:tokens])
        _check(out, c, q_out.cpu(), got_sel, cu=cu_h)
        every = np.tile(np.arange(mb, dtype=np.int32), (tokens + 2, hkv, 1))
        dense = pa.pa_sparse(q_out, k_cache, v_cache, table, lens, torch.from_numpy(every).to(DEV), cu_seq_lens_q=cu)
        seen = every.copy()
        for t, (_, p) in enumerate(ref.query_positions(now, cu_h)):
            seen[t][seen[t] > p // bs] = -1
        _check(dense, c, q_out.cpu(), seen, cu=cu_h)
    assert rng is not None


def _step_args(dtype=BF16, d=128, bs=16, hkv=2, seed=0):
    c = make_cache(seed, [100, 333, 17], hkv, d, bs, dtype)
    g = torch.Generator().manual_seed(seed)
    s = {k: v.to(DEV) for k, v in c.items()}
    s["qkv"] = torch.randn(3, 4 + 2 * hkv, d, generator=g).to(dtype).to(DEV)
    s["slots"] = torch.tensor([int(c["table"][r, (n - 1) // bs]) * bs + (n - 1) % bs for r, n in enumerate([100, 333, 17])],
                              dtype=torch.int32, device=DEV)
    s["pos"] = (s["lens"] - 1).contiguous()
    s["angles"] = angle_table(400, d).to(DEV)
    return s


def _step(s, hkv=2, bs=16, **kw):
    q, k, v = s["qkv"].split([4, hkv, hkv], 1)
    q = pa.pa_cache_append_rotary(q, k, v, s["slots"], s["k"], s["v"], s["pos"], s["angles"], bounds=s["bounds"], **kw)
    sel = pa.pa_select_blocks(q, s["bounds"], s["table"], s["lens"], 5, bs, **kw)
    return pa.pa_sparse(q, s["k"], s["v"], s["table"], s["lens"], sel, **kw), sel


def test_a_captured_step_replays_on_new_inputs():
    s = _step_args()
    _step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, sel = _step(s)
    for seed in (1, 2):
        fresh = _step_args(seed=seed)
        for k in s:
            s[k].copy_(fresh[k]) if s[k].shape == fresh[k].shape else None
        graph.replay()
        want, want_sel = _step(fresh)
        torch.cuda.synchronize()
        assert torch.equal(sel, want_sel) and torch.equal(out, want)
        assert torch.equal(s["k"].nan_to_num(9.0), fresh["k"].nan_to_num(9.0))
        assert torch.equal(s["bounds"].nan_to_num(9.0), fresh["bounds"].nan_to_num(9.0))


_FIRST_CALL_CAPTURED = """
import torch
import paged_kv_cache_300_gb300 as pa
from tests.test_gpu_sparse import F32, BF16, _step, _step_args
for dtype in (BF16, F32):
    s, fresh = _step_args(dtype), _step_args(dtype)
    q, k = s["qkv"][:, :4], s["qkv"][:, 4:6]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, sel = _step(s)
        turned = pa.pa_rotary(q, k, s["pos"], s["angles"])
    for _ in range(2):
        graph.replay()
    want, want_sel = _step(fresh)
    assert torch.equal(sel, want_sel) and torch.equal(out, want)
    assert all(torch.equal(a, b) for a, b in zip(turned, pa.pa_rotary(q, k, s["pos"], s["angles"])))
print("captured first")
"""


def test_the_first_call_of_a_process_can_be_captured():
    r = subprocess.run([sys.executable, "-c", _FIRST_CALL_CAPTURED], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_on_another_stream_and_several_at_once():
    want = [_step(_step_args(seed=i)) for i in range(4)]
    args = [_step_args(seed=i) for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [None] * 4
    for _ in range(3):
        for i, st in enumerate(streams):
            got[i] = _step(args[i], stream=st)
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(got, want):
        assert torch.equal(a, c) and torch.equal(b, d)


def test_small_calls_without_rows():
    s = _step_args()
    q = s["qkv"][:0, :4]
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    cu = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert pa.pa_rotary(q, None, none, s["angles"])[0].shape == (0, 4, 128)
    before = s["k"].clone()
    pa.pa_cache_append_rotary(None, s["qkv"][:0, 4:6], s["qkv"][:0, 6:], none, s["k"], s["v"], none, s["angles"], bounds=s["bounds"])
    assert torch.equal(before.view(torch.int16), s["k"].view(torch.int16))
    sel = pa.pa_select_blocks(q.contiguous(), s["bounds"], s["table"], s["lens"], 3, 16, cu_seq_lens_q=cu)
    assert sel.shape == (0, 2, 3)
    assert pa.pa_sparse(q.contiguous(), s["k"], s["v"], s["table"], s["lens"], sel, cu_seq_lens_q=cu).shape == (0, 4, 128)

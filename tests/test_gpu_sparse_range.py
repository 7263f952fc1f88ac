"""Block-sparse calls where the numbers are hardest: weights whose sums cancel, long sums,
values near the end of the numbers, scores that differ by less than any float shows."""
import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import sparse as ref
from tests.sparse_util import BF16, F32, f64, half_step, make_cache
from tests.test_gpu_sparse import _attend, _bounds, _check, _random_choice, _select, i32

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa.load()


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [9, 1300])
def test_sparse_holds_weights_to_fp32(dtype, d, rows):
    """Values whose weighted sum cancels to some 2^-24 of its terms show what the weights are held to.

    A score is one exact product k of 8 bits, at most 1 in magnitude, and the scale is ln 2, so a weight is
    2^k: scale and its product with log2 e are off by 2^-24 each, the power by 2^-22 (ex2's bound), a difference
    from the reference by 2^-24, so a weight by 2^-22 + 4 ln 2 2^-24 < 2^-22 + 2^-22 of itself.  What 24 bits hold it to:
    2^-24.  The products' sums, 16 terms in three steps of at most 2^-21 of their magnitudes (bf16) or 16 fmas
    and one join of two sides (fp32): 3 2^-21.  Numerator and the sum of weights each: (2 2^-22 + 2^-24 + 3 2^-21)
    of their magnitudes; one division and the output's rounding."""
    bs, hkv, group = 16, 2, 4
    rng = np.random.default_rng(d + rows)
    lens = [bs] * rows
    c = make_cache(3, lens, hkv, d, bs, dtype)
    k = torch.zeros_like(c["k"])
    k[..., 0] = -torch.from_numpy(rng.integers(0, 128, tuple(k.shape[:3]))).to(dtype) / 128
    q = torch.zeros(rows, hkv * group, d, dtype=dtype)
    q[..., 0] = 1
    # the last three values of a channel take back what the sum of those before has left, 8 bits each
    w = np.exp2(f64(k)[..., 0])[..., None]
    v = f64(torch.randn(c["v"].shape, generator=torch.Generator().manual_seed(d)).to(dtype))
    v[:, -3:] = 0
    for t in (-3, -2, -1):
        left = -(w * v).sum(1) / w[:, t]
        v[:, t] = f64(torch.from_numpy(left).to(BF16))
    c["k"], c["v"] = k, torch.from_numpy(v).to(dtype)
    sel = np.zeros((rows, hkv, 1), dtype=np.int32)
    got = f64(_attend(c, q, sel, float(np.log(2.0)))).reshape(rows, hkv, group, d)
    block = c["table"].numpy()[:, 0]
    w, v = w[block].astype(np.longdouble), v[block].astype(np.longdouble)  # [rows, 16, hkv, 1 or d]
    total = w.sum(1)
    want, size = ((w * v).sum(1) / total)[:, :, None], ((w * np.abs(v)).sum(1) / total)[:, :, None]
    assert (np.abs(want) < 2.0 ** -20 * size).mean() > 0.9
    off = 2 * 2.0 ** -22 + 2.0 ** -24 + 3 * 2.0 ** -21
    bound = off * (size + np.abs(want)) + (half_step(dtype) + 2.0 ** -23) * np.abs(want)
    err = np.abs(got - want)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("d", [64, 128])
def test_sparse_adds_units_with_rounding(d):
    """Many keys of positive values, then a few that take their weighted sum back: each unit of 16
    keys may cost its warp's sum half a step, and a sum that is cut off loses some two.

    512 units a warp, whose sum grows evenly: 512 / 2 half steps of 2^-24 of its end.  Within a unit 3
    products that cut off, each at most (17 / 4 + 1) 2^-23 of its magnitudes (addends at 2^-25 of the largest, the
    sum at 2^-23).  A weight: 2 2^-22 as above and 2^-24.  Joins of warps: 3 2^-24 and 4 powers.  All of the
    magnitudes' sum; the division and the output's rounding of what is left."""
    bs, hkv, rows, top = 16, 1, 310, 2048
    rng = np.random.default_rng(d)
    c = make_cache(3, [4 * bs], hkv, d, bs, BF16, width=top)
    turn = c["table"][0, :3].tolist()
    table = np.array([turn[i % 3] for i in range(top - 1)] + [int(c["table"][0, 3])], dtype=np.int32)
    c["table"] = torch.from_numpy(table).view(1, top).repeat(rows, 1)
    c["lens"] = i32([top * bs] * rows)
    c["k"] = torch.zeros_like(c["k"])
    c["k"][..., 0] = -torch.from_numpy(rng.integers(0, 128, tuple(c["k"].shape[:3]))).to(BF16) / 128
    w = np.exp2(f64(c["k"])[:, :, 0, 0])  # [blocks, bs]
    v = f64((torch.rand(c["v"].shape, generator=torch.Generator().manual_seed(d)) + 1).to(BF16))[:, :, 0]
    last, many = table[-1], [int((table[:-1] == p).sum()) for p in turn]
    v[last] = 0
    for t in range(4):
        left = sum(n * (w[p][:, None] * v[p]).sum(0) for n, p in zip(many, turn)) + (w[last][:, None] * v[last]).sum(0)
        v[last, t] = f64(torch.from_numpy(-left / w[last, t]).to(BF16))
    c["v"][:, :, 0] = torch.from_numpy(v).to(BF16)
    q = torch.zeros(rows, 2, d, dtype=BF16)
    q[..., 0] = 1
    sel = np.tile(np.arange(top, dtype=np.int32), (rows, 1, 1))
    got = f64(_attend(c, q, sel, float(np.log(2.0))))
    assert (got == got[:1, :1]).all()
    w, v = w.astype(np.longdouble), v.astype(np.longdouble)
    parts = [(n, w[p][:, None], v[p]) for n, p in zip(many + [1], turn + [last])]
    total = sum(n * a.sum(0) for n, a, _ in parts)
    want, size = sum(n * (a * b).sum(0) for n, a, b in parts) / total, sum(n * (a * abs(b)).sum(0) for n, a, b in parts) / total
    assert (abs(want) < 2.0 ** -22 * size).all()
    off = 256 * 2.0 ** -24 + 3 * 5.25 * 2.0 ** -23 + 2 * 2.0 ** -22 + 2.0 ** -24 + 3 * 2.0 ** -24 + 4 * 2.0 ** -22
    bound = off * size + 2.0 ** -8 * abs(want)
    assert (abs(got[0, 0] - want) <= bound).all(), float((abs(got[0, 0] - want) / bound).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rows", [(64, 1), (128, 1), (128, 40), (128, 930), (64, 6200)])
def test_sparse_of_values_near_the_end_of_the_numbers(dtype, d, rows):
    """Weights never pass 1, so that sums of as many values as have one stay finite: first keys of
    score 0, then as many of score 7.5 (log2), as far as a maximum may grow before it is followed."""
    bs, n = 16, 64
    c = make_cache(2, [n * bs], 1, d, bs, dtype)
    c["k"][:] = 0
    c["k"][c["table"][0, n // 2:].long(), :, 0, 0] = 7.5
    c["v"] = ((torch.rand(c["v"].shape, generator=torch.Generator().manual_seed(1)) + 1) * 2.0 ** 117).to(dtype)
    q = torch.zeros(rows, 2, d, dtype=dtype)
    q[..., 0] = 1
    sel = np.arange(n, dtype=np.int32).reshape(1, 1, n)
    big = dict(c, table=c["table"].repeat(rows, 1), lens=c["lens"].repeat(rows))
    got = _attend(big, q, np.repeat(sel, rows, 0), float(np.log(2.0)))
    assert torch.equal(got, got[:1].expand_as(got))
    _check(got[:1], c, q[:1], sel, float(np.log(2.0)))


# ------------------------------------------------------------------ selection
def _whole(x, bits):
    """float64 -> whole numbers of 2^-bits, Python's own."""
    m, e = np.frexp(x)
    return np.array([int(f * 2.0 ** 53) * 2 ** (int(k) - 53 + bits) if f else 0 for f, k in zip(m.ravel(), e.ravel())],
                    dtype=object).reshape(x.shape)


def _exact_choice(q, bounds, top, bits):
    """The choice of a single row among blocks 0 .. n - 1, the first and the last forced: q [G, D] and bounds
    [n, 2, D] in whole numbers."""
    x, lo, hi = _whole(q, bits), _whole(bounds[:, 0], bits), _whole(bounds[:, 1], bits)
    score = [max(sum(u * (h if u > 0 else l) for u, h, l in zip(row, b_hi, b_lo)) for row in x) for b_hi, b_lo in zip(hi, lo)]
    n = len(score)
    rank = sorted(range(1, n - 1), key=lambda j: (-score[j], j))
    return np.array(sorted([0, n - 1] + rank[:top - 2]), dtype=np.int32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,top", [(26, 9), (400, 60)])
@pytest.mark.parametrize("step", [-20, -30, -35, -37, -44])
@pytest.mark.parametrize("rows,chunk", [(1, False), (19, True), (700, False)])
def test_select_of_scores_that_no_float_tells_apart(dtype, n, top, step, rows, chunk):
    """One channel's share of the scores is 2^step of the others', the same in all blocks; its
    steps decide, however few or many blocks are in doubt and whoever chooses.  Channels 24 and on
    and 56 and on are added up apart from the others: there, it is the only one that is not 0."""
    d, bs = 64, 16
    for seed, at in ((4, 0), (5, 24)):
        rng = np.random.default_rng(seed)
        bounds = _bounds(seed, 1, 1, d, dtype).repeat(n, 1, 1, 1).clone()
        bounds[:, 0, 1, at] = torch.from_numpy(rng.integers(1, 200, n)).to(dtype) * 2.0 ** -6
        q = torch.randn(4, d, generator=torch.Generator().manual_seed(seed)).abs() + 1
        if at:
            q[:, 24:32] = q[:, 56:] = 0
        q[:, at] = 2.0 ** step
        q, bounds = q.to(BF16).to(dtype), bounds.to(BF16).to(dtype)
        table = torch.from_numpy(rng.permutation(n).astype(np.int32)).view(1, n)
        want = _exact_choice(f64(q), f64(bounds[table[0].long(), 0]), top, 140)
        many = q.view(1, 4, d).repeat(rows, 1, 1)
        if chunk:
            got = _select(many, bounds, table, i32([n * bs]), top, bs, cu=i32([0, rows]))
            got = got[rows - bs:]  # (the others see a block less)
        else:
            got = _select(many, bounds, table.repeat(rows, 1), i32([n * bs] * rows), top, bs)
        assert (got == want).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,top", [(26, 9), (400, 60)])
@pytest.mark.parametrize("tokens", [1, 16])
def test_select_of_heads_whose_largest_channels_differ(dtype, n, top, tokens):
    """Each head's products add up to less than 2^128, those of the largest |q| of all heads do not: the
    scores are in doubt all the same, and 24 bits of them are equal."""
    d, bs = 64, 16
    rng = np.random.default_rng(n)
    bounds = torch.ones(n, 1, 2, d, dtype=dtype)
    bounds[:, 0, 0] = -1
    bounds[:, 0, 1, 5] = torch.from_numpy(rng.integers(1, 200, n)).to(dtype) * 2.0 ** -8
    q = torch.zeros(tokens, 4, d, dtype=dtype)
    for g in range(4):  # 2^127 and a half each
        q[:, g, 16 * g] = 1.5 * 2.0 ** 126 if g else 2.0 ** 127
        q[:, g, 5] = 2.0 ** 100
    table = torch.from_numpy(rng.permutation(n).astype(np.int32)).view(1, n)
    got = _select(q, bounds, table, i32([n * bs]), top, bs, cu=i32([0, tokens]))
    step = f64(bounds[table[0].long(), 0, 1, 5])
    rank = sorted(range(1, n - 1), key=lambda j: (-step[j], j))
    assert (got == np.array(sorted([0, n - 1] + rank[:top - 2]), dtype=np.int32)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 24])
def test_select_of_one_large_product_beside_many_small_ones(dtype, d, tokens):
    """A large product first and d - 1 small ones behind it that a matrix product drops whole: positive ones in
    some blocks, negative ones in the others, which hold one more product that makes up for most of the difference."""
    bs, n, top = 16, 120, 42
    rng = np.random.default_rng(d)
    q = torch.full((tokens, 2, d), 1.9921875 * 2.0 ** -13)
    q[..., 0] = 1
    small = (d - 1) * 1.9921875 * 2.0 ** -26  # what is dropped
    more = 0.95 * 2 * small  # the others are less by 2 small - more
    high = rng.permutation(n - 2)[:top - 2] + 1
    bounds = torch.full((n, 1, 2, d), -2.0 ** -13)
    bounds[high, 0, 1, 1:] = 2.0 ** -13
    bounds[..., 0] = 1
    other = np.setdiff1d(np.arange(n), high)
    bounds[other, 0, 1, 1] = more / (1.9921875 * 2.0 ** -13)
    q, bounds = q.to(dtype), bounds.to(dtype)
    want = np.array(sorted([0, n - 1] + high.tolist()), dtype=np.int32)
    table = torch.arange(n, dtype=torch.int32).view(1, n)
    assert np.array_equal(_exact_choice(f64(q)[0], f64(bounds)[:, 0], top, 140), want)
    got = _select(q, bounds, table, i32([n * bs]), top, bs, cu=i32([0, tokens]))
    assert (got[-bs:] == want).all()


# ------------------------------------------------------------------ the error of whole outputs
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hq,hkv", [(128, 8, 2), (64, 6, 1), (64, 16, 2)])
@pytest.mark.parametrize("chunk", [False, True])
def test_sparse_error_of_whole_outputs(dtype, d, hq, hkv, chunk):
    """The relative 2-norm of the error, which is that of fp32 arithmetic and not of less.

    Roundings are half a step at most and of any sign, so sums of n of them grow as the root of n.  A score's
    d products: root(d) 2^-24 of scale times the root of their squares' sum, less than 3 here; ex2: 2^-22.  Weighted
    values: root(300) 2^-25 of their sum.  Together e < (3 root(128) + 4 + 9) 2^-24 = 47 2^-24 of the output: the bound in
    fp32.  A bf16 output is the neighbour of the rounded exact value with a chance of e over a step, 2^-8 to
    2^-7 of it, and then off by a step: in the 2-norm root(e 2^-7) of the outputs."""
    bs, top, batch = 16, 20, 24
    rng = np.random.default_rng(d)
    lens = [int(n) for n in rng.integers(200, 1500, batch)]
    cu = None
    if chunk:
        cu = np.concatenate([[0], np.cumsum(rng.integers(1, 6, batch))]).astype(np.int32)
    c = make_cache(d, lens, hkv, d, bs, dtype)
    q = torch.randn(batch if cu is None else int(cu[-1]), hq, d, generator=torch.Generator().manual_seed(d)).to(dtype)
    sel = _random_choice(rng, lens, hkv, bs, top, cu)
    got = f64(_attend(c, q, sel, cu=cu))
    want, _ = ref.attend(f64(q), f64(c["k"]), f64(c["v"]), c["table"].numpy(), np.array(lens), sel, d ** -0.5, cu)
    e = 47 * 2.0 ** -24
    if dtype == BF16:
        want, e = f64(torch.from_numpy(want).to(BF16)), (e * 2.0 ** -7) ** 0.5
    assert np.linalg.norm(got - want) <= e * np.linalg.norm(want), np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("n,top", [(40, 14), (400, 60)])
@pytest.mark.parametrize("rows,chunk", [(1, False), (19, True), (700, False)])
def test_select_of_products_that_fp32_rounds(n, top, rows, chunk):
    """fp32 operands of 24 bits whose products are rounded: blocks in which two channels' shares are
    moved against each other, so that sums differ by the last bits of the bounds."""
    d, bs = 64, 16
    for seed in (1, 2, 3):
        rng = np.random.default_rng(seed)
        q = (rng.random((4, d)) + 1).astype(np.float32)
        q[1:] *= np.float32(0.5)  # the first head decides
        one = (rng.random((2, d)) + 1).astype(np.float32)
        one[0] = -one[0]
        bounds = np.repeat(one[None], n, 0)
        for j in range(n):
            a, b = rng.permutation(d)[:2]
            more = rng.random() / 4
            bounds[j, 1, a] += np.float32(more)
            bounds[j, 1, b] -= np.float32(more * q[0, a] / q[0, b])
        want = _exact_choice(q.astype(np.float64), bounds.astype(np.float64), top, 60)
        table = torch.arange(n, dtype=torch.int32).view(1, n)
        many, held = torch.from_numpy(q).view(1, 4, d).repeat(rows, 1, 1), torch.from_numpy(bounds).view(n, 1, 2, d)
        if chunk:
            got = _select(many, held, table, i32([n * bs]), top, bs, cu=i32([0, rows]))[rows - bs:]
        else:
            got = _select(many, held, table.repeat(rows, 1), i32([n * bs] * rows), top, bs)
        assert (got == want).all()

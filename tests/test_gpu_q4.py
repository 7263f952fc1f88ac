"""The 4-bit pool on the GPU: update, read-back and decode against the plain
reference."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import q4
from tests.q4_util import NORM, check, decode_bound, edge_rows, make, write_rows

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa.load()


def _dev(c):
    return {k: (v if isinstance(v, torch.Tensor) else torch.from_numpy(v)).to(DEV)
            for k, v in c.items() if k != "bs"}


def _f32(t):
    return t.float().numpy()


def _same_pool(got, want, bs, d):
    """Codes and scales equal (a NaN scale is a NaN scale)."""
    got = got.cpu().numpy()
    assert np.array_equal(got[:, :, :bs * d], want[:, :, :bs * d])
    g, w = (np.ascontiguousarray(x[:, :, bs * d:]).view("<u2").astype(np.int64) for x in (got, want))
    nan = lambda x: (x & 0x7FFF) > 0x7F80  # noqa: E731
    zero = lambda x: (x & 0x7FFF) == 0  # noqa: E731
    assert ((g == w) | (nan(g) & nan(w)) | (zero(g) & zero(w))).all()


# ------------------------------------------------------------------ update
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hkv", [(64, 16, 1), (64, 32, 3), (128, 16, 8), (128, 32, 5), (64, 32, 2)])
@pytest.mark.parametrize("total", [1, 2, 37, 200])
def test_update(dtype, d, bs, hkv, total):
    rng = np.random.default_rng(total + d)
    g = torch.Generator().manual_seed(total)
    nb = -(-total // bs) + 3
    start = int(rng.integers(0, 2 * bs))
    slots = (start + np.arange(total)).astype(np.int32)  # a run that starts anywhere in a block
    if total == 200:
        slots = rng.permutation(nb * bs)[:total].astype(np.int32)  # and slots in any order
    slots[rng.random(total) < 0.1] = -1
    x = torch.randn(2, total, hkv, d, generator=g) * torch.exp(3 * torch.randn(2, total, hkv, 1, generator=g))
    x[0, 0, 0] = 1.5                   # a row of one value
    x[1, 0, hkv - 1] = 0.0
    x[0, total // 2, 0, 3] = float("nan")
    x[1, total // 2, 0, 9] = float("inf")
    x = x.to(dtype)
    pool = rng.integers(0, 256, (nb, hkv, q4.record_bytes(d, bs)), dtype=np.uint8)
    got = torch.from_numpy(pool).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_cache_update_q4(x[0].to(DEV), x[1].to(DEV), torch.from_numpy(slots).to(DEV), got, dev_err=err)
    torch.cuda.synchronize()
    for i, s in enumerate(slots):
        if s >= 0:
            q4.write(pool, int(s), _f32(x[0, i]), _f32(x[1, i]), bs)
    assert err.item() == 0
    _same_pool(got, pool, bs, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs", [(64, 32), (128, 16)])
@pytest.mark.parametrize("total,hkv,heads", [(1700, 5, 2), (1600, 8, 3), (2600, 5, 3), (4200, 3, 3), (4099, 8, 8)])
def test_update_with_several_heads_a_warp(dtype, d, bs, total, hkv, heads):
    """Chunks large enough that a warp takes several heads, of which the last
    warps have fewer: a run of slots that begins in the middle of a token pair,
    then lone and neighbouring ones in any order, padding between."""
    assert min(hkv, total * hkv // 4096) == heads
    rng = np.random.default_rng(total)
    nb = -(-total // bs) + 3
    slots = np.arange(3, 3 + total, dtype=np.int32)
    rest = np.setdiff1d(np.arange(nb * bs), slots[:total // 2])
    slots[total // 2:] = rng.permutation(rest)[:total - total // 2]
    slots[rng.random(total) < 0.1] = -1
    g = torch.Generator().manual_seed(total)
    x = (torch.randn(2, total, hkv, d, generator=g) * torch.exp(torch.randn(2, total, hkv, 1, generator=g))).to(dtype)
    pool = rng.integers(0, 256, (nb, hkv, q4.record_bytes(d, bs)), dtype=np.uint8)
    got = torch.from_numpy(pool).to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_cache_update_q4(x[0].to(DEV), x[1].to(DEV), torch.from_numpy(slots).to(DEV), got, dev_err=err)
    write_rows(pool, slots, _f32(x[0]), _f32(x[1]), bs)
    assert err.item() == 0
    _same_pool(got, pool, bs, d)


def test_update_with_every_step_there_is():
    """A row for each bf16 step above 2^-100, with values at the borders of
    its codes and one number beside them: 16 / step has to be correctly rounded."""
    bs, d = 32, 64
    step = (np.arange(0x0D81, 0x7F80, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)
    step = step[15 * step < q4.BF16_MAX]
    assert step[0] < 1.01 * 2.0 ** -100 and step[-1] > 2.0 ** 124 and len(step) == 28679
    edge = (step[:, None] * (np.arange(15) + 0.5)).astype(np.float32)
    up, down = np.nextafter(edge, np.float32(np.inf)), np.nextafter(edge, np.float32(0))
    top = (15 * step * (1 - 2.0 ** -10)).astype(np.float32)[:, None]
    more = np.random.default_rng(3).random((len(step), 17)).astype(np.float32)
    x = np.concatenate([np.zeros_like(top), top, np.minimum(edge, top), np.minimum(up, top), down, more * top], 1)
    n, s, _ = q4.quantise(x)
    assert np.array_equal(q4.bf16_bits_to_f64(s), step) and n.max() == 15
    t = len(x)
    pool = np.zeros((-(-t // bs), 1, q4.record_bytes(d, bs)), dtype=np.uint8)
    got = torch.from_numpy(pool).to(DEV)
    k, v = x[:, None], np.ascontiguousarray(x[:, None, ::-1])
    slots = np.arange(t, dtype=np.int32)
    pa.pa_cache_update_q4(torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV), torch.from_numpy(slots).to(DEV), got)
    write_rows(pool, slots, k, v, bs)
    _same_pool(got, pool, bs, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_update_of_extreme_rows(dtype):
    """Rows from the smallest to the largest numbers, and rows whose range
    passes the largest one."""
    d, bs, hkv = 128, 16, 2
    g = torch.Generator().manual_seed(3)
    mag = 10.0 ** torch.linspace(-37, 38, 32)
    x = torch.rand(2, 32, hkv, d, generator=g) * 2 - 1
    x = (x * mag.view(1, -1, 1, 1)).clamp(-3.3e38, 3.3e38).to(dtype)
    x[0, -1, 0, 0], x[0, -1, 0, 1] = 3.3e38, -3.3e38
    pool = np.zeros((2, hkv, q4.record_bytes(d, bs)), dtype=np.uint8)
    got = torch.from_numpy(pool).to(DEV)
    pa.pa_cache_update_q4(x[0].to(DEV), x[1].to(DEV), torch.arange(32, dtype=torch.int32, device=DEV), got)
    for i in range(32):
        q4.write(pool, i, _f32(x[0, i]), _f32(x[1, i]), bs)
    _same_pool(got, pool, bs, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_finite_rows_at_the_end_of_the_numbers(dtype, d):
    """Stored as the format says, and read back without an infinity."""
    bs, x = 16, edge_rows(dtype)
    x = torch.cat([x, x[:, torch.arange(63, -1, -1)]], 1)[:, :d].unsqueeze(1)
    t = len(x)
    nb = t // bs + 1
    pool = np.zeros((nb, 1, q4.record_bytes(d, bs)), dtype=np.uint8)
    got = torch.from_numpy(pool).to(DEV)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    xd = x.to(DEV)
    pa.pa_cache_update_q4(xd, xd, i32(list(range(t))), got)
    for i in range(t):
        q4.write(pool, i, _f32(x[i]), _f32(x[i]), bs)
    _same_pool(got, pool, bs, d)
    kf, vf = torch.empty_like(xd), torch.empty_like(xd)
    pa.pa_cache_gather_q4(got, i32([list(range(nb))]), i32([0, t]), kf, vf)
    assert torch.isfinite(kf).all() and torch.isfinite(vf).all()
    # each row once more as the one token of a sequence
    lens, tab = i32([0] * t), torch.arange(t, dtype=torch.int32, device=DEV).view(-1, 1)
    alone = pa.pa_q4_pool(t, 1, d, bs)
    ks, vs = torch.empty_like(xd), torch.empty_like(xd)
    pa.pa_decode_q4(torch.zeros_like(xd), alone, tab, lens, xd, xd, k_stored=ks, v_stored=vs)
    assert torch.equal(ks, kf) and torch.equal(vs, vf)


def test_update_skips_slots_beyond_the_pool():
    d, bs, hkv = 64, 16, 2
    x = torch.randn(3, hkv, d, device=DEV)
    pool = torch.zeros(2, hkv, q4.record_bytes(d, bs), dtype=torch.uint8, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_cache_update_q4(x, x, torch.tensor([32, 2**31 - 1, -5], dtype=torch.int32, device=DEV), pool, dev_err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK and not pool.any()


# ------------------------------------------------------------------ gather
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hkv", [(64, 16, 2), (64, 32, 5), (128, 16, 8), (128, 32, 1)])
def test_gather(dtype, d, bs, hkv):
    lens = [0, 1, bs - 1, bs, bs + 1, 77, 0, 3 * bs, 130]
    c = make(5, lens, hkv, hkv, d, bs, dtype)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    extra = 9  # rows behind the last request stay as they were
    kf = torch.full((cu[-1] + extra, hkv, d), 7.0, dtype=dtype, device=DEV)
    vf = torch.full_like(kf, -7.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = _dev(c)
    pa.pa_cache_gather_q4(g["pool"], g["table"], torch.from_numpy(cu).to(DEV), kf, vf, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert (kf[cu[-1]:] == 7).all() and (vf[cu[-1]:] == -7).all()
    for b, n in enumerate(lens):
        k, v, _, _ = q4.read(c["pool"], c["table"][b], n, d, bs)
        for got, want in ((kf, k), (vf, v)):
            # b + n s is at most 15 bits of fp32 wide where the two are of one
            # size; its fp32 rounding, then the one to dtype
            w = torch.from_numpy(want).float().to(dtype)
            assert torch.equal(got[cu[b]:cu[b + 1]].cpu(), w), (b, n)


@pytest.mark.parametrize("batch", [31, 33, 1100])
def test_gather_many_requests(batch):
    """Lengths 0 to 40 in a large batch: finding a tile's request."""
    d, bs, hkv = 64, 16, 1
    lens = [(7 * i * i) % 41 if i % 3 else 0 for i in range(batch)]
    c = make(8, lens, hkv, hkv, d, bs, BF16)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    kf = torch.zeros(int(cu[-1]), hkv, d, dtype=BF16, device=DEV)
    vf = torch.zeros_like(kf)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = _dev(c)
    pa.pa_cache_gather_q4(g["pool"], g["table"], torch.from_numpy(cu).to(DEV), kf, vf, dev_err=err)
    assert err.item() == 0
    want = [q4.read(c["pool"], c["table"][b], n, d, bs)[:2] for b, n in enumerate(lens)]
    for got, i in ((kf, 0), (vf, 1)):
        assert torch.equal(got.cpu(), torch.from_numpy(np.concatenate([w[i] for w in want])).float().to(BF16))


def test_gather_zeroes_what_it_cannot_read():
    d, bs, hkv = 128, 16, 2
    c = make(6, [40, 40, 40], hkv, hkv, d, bs, BF16)
    c["table"] = np.ascontiguousarray(c["table"][:, :3])
    c["table"][0, 1] = -1
    c["table"][1, 2] = 10 ** 6
    cu = torch.tensor([0, 40, 80, 130], dtype=torch.int32, device=DEV)  # the third runs over its row of 48
    kf = torch.full((130, hkv, d), 3.0, dtype=BF16, device=DEV)
    vf = torch.full_like(kf, 3.0)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = _dev(c)
    pa.pa_cache_gather_q4(g["pool"], g["table"], cu, kf, vf, dev_err=err)
    assert err.item() == pa.DEVERR_BAD_BLOCK | pa.DEVERR_OVERFLOW
    for t in (kf, vf):
        assert not t[16:32].any() and not t[72:80].any() and not t[128:].any()
    k, _, _, _ = q4.read(c["pool"], c["table"][0], 16, d, bs)
    assert torch.equal(kf[:16].cpu(), torch.from_numpy(k).float().to(BF16))


def test_gather_with_bad_cumulative_lengths_stays_inside():
    d, bs, hkv = 64, 16, 2
    c = make(6, [40, 40], hkv, hkv, d, bs, F32)
    g = _dev(c)
    for cu in ([0, 50, 40], [3, 20, 40], [0, 20, 90], [0, -5, 40]):
        kf = torch.full((60, hkv, d), 3.0, device=DEV)
        vf = torch.full_like(kf, 3.0)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        pa.pa_cache_gather_q4(g["pool"], g["table"], torch.tensor(cu, dtype=torch.int32, device=DEV), kf[:40], vf[:40],
                              dev_err=err)
        assert err.item() & pa.DEVERR_BAD_CU, cu
        assert (kf[40:] == 3).all() and (vf[40:] == 3).all()


# ------------------------------------------------------------------ decode
def _decode(c, **kw):
    g = _dev(c)
    dtype = c["q"].dtype
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ks, vs = torch.empty_like(g["k_new"]), torch.empty_like(g["v_new"])
    out = pa.pa_decode_q4(g["q"], g["pool"], g["table"], g["lens"], g["k_new"], g["v_new"], k_stored=ks, v_stored=vs,
                          dev_err=err, **kw)
    torch.cuda.synchronize()
    assert out.dtype == dtype
    return out, g["pool"], ks, vs, err.item()


def _against_reference(c, scale=None, norm=True, **kw):
    dtype, bs, d = c["q"].dtype, c["bs"], c["q"].shape[2]
    out, pool, ks, vs, err = _decode(c, **kw)
    assert err == 0
    want_pool = c["pool"].copy()
    ref, seen = q4.decode(_f32(c["q"]), want_pool, c["table"], c["lens"], _f32(c["k_new"]), _f32(c["v_new"]), bs, scale)
    _same_pool(pool, want_pool, bs, d)
    for b, (k, v, _, _) in enumerate(seen):
        assert torch.equal(ks[b].cpu(), torch.from_numpy(k[-1]).float().to(dtype))
        assert torch.equal(vs[b].cpu(), torch.from_numpy(v[-1]).float().to(dtype))
    bound = decode_bound(c["q"], seen, ref, dtype, d ** -0.5 if scale is None else scale)
    check(out, ref, bound, norm=NORM[dtype] if norm else None)
    return out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 8), (32, 8), (8, 1), (21, 3), (12, 6), (40, 5), (16, 16)])
def test_decode(dtype, d, bs, hq, hkv):
    lens = [0, 1, bs - 2, bs - 1, bs, bs + 1, 2 * bs - 1, 63, 64, 200, 517]
    _against_reference(make(hq * 100 + hkv, lens, hq, hkv, d, bs, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[0], [5000], [3, 20000, 900], [1500] * 40, list(range(0, 300))])
def test_decode_lengths(dtype, lens):
    _against_reference(make(11, lens, 8, 2, 128, 16, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hq,hkv", [(128, 7, 7), (64, 26, 13), (64, 32, 32), (128, 48, 12), (128, 64, 8), (64, 88, 11)])
def test_decode_many_rows(dtype, d, hq, hkv):
    """Batches in which a warp has a head of its own, or two share one."""
    _against_reference(make(hkv, [(37 * i) % 211 for i in range(60)], hq, hkv, d, 16, dtype))


@pytest.mark.parametrize("batch", [511, 512, 513, 1500])
def test_decode_batches_around_the_cached_lengths(batch):
    _against_reference(make(batch, [(5 * i) % 40 for i in range(batch)], 2, 2, 64, 16, BF16))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_one_long_sequence(dtype):
    _against_reference(make(12, [70001], 8, 1, 64, 32, dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 8, 8), (64, 32, 16, 2), (64, 16, 16, 16)])
def test_decode_long_walks(dtype, d, bs, hq, hkv):
    """Enough tokens that every warp walks hundreds of blocks; the pool is
    made on the GPU and four sequences are checked."""
    b, lo, hi = 72, 6000, 12000
    rng = np.random.default_rng(d + hkv)
    lens = rng.integers(lo, hi, b).astype(np.int32)
    held = lens // bs + 1
    nb = int(held.sum())
    perm = rng.permutation(nb).astype(np.int32)
    table = np.full((b, held.max()), -1, dtype=np.int32)
    for i, at in enumerate(np.cumsum(held) - held):
        table[i, :held[i]] = perm[at:at + held[i]]
    g = torch.Generator(device=DEV).manual_seed(5)
    pool = torch.randint(0, 256, (nb, hkv, q4.record_bytes(d, bs)), dtype=torch.uint8, device=DEV, generator=g)
    scales = torch.randn(nb, hkv, bs, 4, device=DEV, generator=g) * torch.tensor([0.02, 0.2, 0.02, 0.4], device=DEV)
    scales += torch.tensor([0.3, -2.2, 0.3, -2.2], device=DEV)
    pool[:, :, bs * d:] = scales.to(BF16).view(torch.uint8).view(nb, hkv, bs * 8)
    rand = lambda *s: torch.randn(*s, device=DEV, generator=g).to(dtype)  # noqa: E731
    q, kn, vn = rand(b, hq, d), rand(b, hkv, d), rand(b, hkv, d)
    pick = [0, 17, 40, b - 1]
    rows = [table[i, :held[i]].astype(np.int64) for i in pick]
    blocks = pool[torch.from_numpy(np.concatenate(rows)).to(DEV)].cpu().numpy()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = pa.pa_decode_q4(q, pool, torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV), kn, vn, dev_err=err)
    assert err.item() == 0
    small = np.full((4, held.max()), -1, dtype=np.int32)
    at = 0
    for j, r in enumerate(rows):
        small[j, :len(r)] = np.arange(at, at + len(r))
        at += len(r)
    sel = lambda x: x[torch.tensor(pick, device=DEV)].cpu()  # noqa: E731
    ref, seen = q4.decode(_f32(sel(q)), blocks, small, lens[pick], _f32(sel(kn)), _f32(sel(vn)), bs)
    check(sel(out), ref, decode_bound(sel(q), seen, ref, dtype, d ** -0.5), norm=NORM[dtype])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs", [(64, 32), (128, 16)])
def test_decode_peaked_and_scaled(dtype, d, bs):
    """Scores that span hundreds (one key takes nearly all), and another scale."""
    c = make(13, [40, 333, 1000], 8, 2, d, bs, dtype)
    c["q"] = (c["q"].float() * 30).to(dtype)
    _against_reference(c, norm=False)
    c["q"] = (c["q"].float() / 60).to(dtype)
    _against_reference(c, scale=0.7, softmax_scale=0.7, norm=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("k_gain,v_gain,q_gain", [(1e-6, 1.0, 1e6), (1e6, 1e-6, 1e-6), (1.0, 1e-20, 1.0),
                                                  (1.0, 1e20, 1.0), (1e-15, 3e4, 1e15)])
def test_decode_magnitudes(dtype, k_gain, v_gain, q_gain):
    """Keys, values and queries far from 1: the 16-bit operands of the
    products must not leave their range."""
    c = make(14, [100, 17, 400], 8, 2, 128, 16, dtype, k_gain=k_gain, v_gain=v_gain)
    c["q"] = (c["q"].float() * q_gain).to(dtype)
    _against_reference(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("step", [2.0 ** 110, 2.0 ** 120, 2.0 ** 123])
def test_decode_of_the_largest_steps(dtype, group, step):
    """One key that outweighs 4000 others by 2^18 each: together they are a
    64th of the sum, and none of them may be lost because its value's step is
    large.  Their lows are the opposite of the one's."""
    d, bs, n = 128, 16, 4000
    c = make(35, [n], group, 1, d, bs, dtype)
    sc = np.ascontiguousarray(c["pool"][:, :, bs * d:]).view("<u2").reshape(-1, 1, bs, 4).copy()
    bits = lambda x: torch.tensor(x).to(BF16).view(torch.int16).numpy().view("<u2")  # noqa: E731
    sc[..., 0], sc[..., 1] = 0, 0                    # keys of zeros
    sc[..., 2], sc[..., 3] = bits(step), bits(-2.0 * step)
    blk = c["table"][0, 5]
    sc[blk, 0, 7, 1] = bits(1.0)                     # the one key
    sc[blk, 0, 7, 3] = bits(-8.0 * step)
    c["pool"][:, :, bs * d:] = sc.reshape(*c["pool"].shape[:2], -1).view(np.uint8)
    c["k_new"][:], c["v_new"][:] = 0, 0
    c["q"][:] = 18 * 0.6931471805599453 / d ** 0.5    # scale q.k = 18 log 2
    _against_reference(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_values_of_very_different_sizes(dtype):
    """Tokens whose values differ by 2^40 in size, the large ones hardly seen."""
    c = make(15, [300, 300], 8, 2, 64, 16, dtype)
    d, bs = 64, 16
    sc = np.ascontiguousarray(c["pool"][:, :, bs * d:]).view("<u2")
    f = (sc.astype(np.uint32) << 16).view(np.float32).reshape(*sc.shape[:2], bs, 4)
    f[:, :, ::3, 2:] *= 2.0 ** -40
    c["pool"][:, :, bs * d:] = (f.reshape(sc.shape).view(np.uint32) >> 16).astype("<u2").view(np.uint8)
    _against_reference(c)


def test_decode_of_constant_rows():
    """Every value row holds one number (step 0)."""
    c = make(16, [50, 3], 4, 2, 64, 16, F32)
    sc = np.ascontiguousarray(c["pool"][:, :, 16 * 64:]).view("<u2").reshape(*c["pool"].shape[:2], 16, 4).copy()
    sc[..., 2] = 0
    c["pool"][:, :, 16 * 64:] = sc.reshape(*c["pool"].shape[:2], -1).view(np.uint8)
    c["v_new"][:] = 0.25
    _against_reference(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 16, 2)])
@pytest.mark.parametrize("size", [1e9, 1e12, 1e30, 3.3e38])
@pytest.mark.parametrize("every", [1, 3])
def test_decode_of_large_constant_rows(dtype, d, hq, hkv, size, every):
    """Value rows of one large number (step 0), all or one in three: what they
    weigh is held back by their size, not by their step."""
    bs = 16
    c = make(34, [50, 3, 700, 2000], hq, hkv, d, bs, dtype)
    sc = np.ascontiguousarray(c["pool"][:, :, bs * d:]).view("<u2").reshape(*c["pool"].shape[:2], bs, 4).copy()
    low = torch.tensor(size).to(BF16).view(torch.int16).item() & 0xFFFF
    held = (sc[..., 2] & 0x7FFF) <= 0x7F80  # slots that hold a token
    held[:, :, np.arange(bs) % every != 0] = False
    sc[..., 2][held], sc[..., 3][held] = 0, low
    c["pool"][:, :, bs * d:] = sc.reshape(*c["pool"].shape[:2], -1).view(np.uint8)
    if every == 1:
        c["v_new"][:] = size
    _against_reference(c)


def test_decode_zero_query_is_the_mean():
    c = make(17, [100], 2, 1, 64, 16, F32)
    c["q"].zero_()
    _against_reference(c)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_nan_rows_reach_their_heads_only(dtype):
    d, bs = 128, 16
    c = make(18, [200, 200, 200], 8, 2, d, bs, dtype)
    at = lambda b, t: (c["table"][b, t // bs], bs * d + 8 * (t % bs))  # noqa: E731
    blk, o = at(0, 77)
    c["pool"][blk, 1, o:o + 4] = 255       # a key of kv head 1, sequence 0
    blk, o = at(2, 5)
    c["pool"][blk, 0, o + 4:o + 8] = 255   # a value of kv head 0, sequence 2
    out, _, _, _, err = _decode(c)
    assert err == 0
    nan = torch.isnan(out).cpu()
    want = torch.zeros_like(nan)
    want[0, 4:] = True
    want[2, :4] = True
    assert torch.equal(nan, want)
    c["q"][1, 3, 9] = float("nan")
    out, _, _, _, _ = _decode(c)
    want[1, 3] = True
    assert torch.equal(torch.isnan(out).cpu(), want)


def test_decode_nan_new_token():
    c = make(19, [33, 20], 4, 2, 64, 16, BF16)
    c["k_new"][0, 1, 3] = float("inf")
    c["v_new"][1, 0, 0] = float("nan")
    out, pool, ks, vs, err = _decode(c)
    want_pool = c["pool"].copy()
    q4.decode(_f32(c["q"]), want_pool, c["table"], c["lens"], _f32(c["k_new"]), _f32(c["v_new"]), 16)
    _same_pool(pool, want_pool, 16, 64)
    assert torch.isnan(ks[0, 1]).all() and torch.isfinite(ks[0, 0]).all() and torch.isnan(vs[1, 0]).all()
    assert torch.isnan(out[0, 2:]).all() and torch.isfinite(out[0, :2]).all()
    assert torch.isnan(out[1, :2]).all() and torch.isfinite(out[1, 2:]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 32)])
def test_decode_bad_blocks_and_lengths(dtype, d, bs):
    lens = [100, 100, 5, 100, 900]
    c = make(20, lens, 8, 2, d, bs, dtype)
    good, pool_good, _, _, _ = _decode(c)
    c["table"][0, 1] = -1
    c["table"][1, 100 // bs] = len(c["pool"])   # the append's own block
    c["table"][4, 900 // bs - 3] = 2 ** 31 - 1
    c["lens"][2] = -1
    before = c["pool"].copy()
    out, pool, _, _, err = _decode(c)
    assert err == pa.DEVERR_BAD_BLOCK | pa.DEVERR_OVERFLOW
    for b in (0, 1, 2, 4):
        assert not out[b].any()
    assert torch.equal(out[3], good[3])
    # no append was written where the block or the length is bad
    for b in (1, 2):
        own = c["table"][b][(c["table"][b] >= 0) & (c["table"][b] < len(before))]
        assert np.array_equal(pool.cpu().numpy()[own], before[own])
    for n in (c["table"].shape[1] * bs, 2 ** 31 - 1):
        c["lens"][2] = n
        out, _, _, _, err = _decode(c)
        assert err & pa.DEVERR_OVERFLOW and not out[2].any() and torch.equal(out[3], good[3])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_does_not_depend_on_placement(dtype):
    c = make(21, [1000, 37, 512], 16, 4, 128, 16, dtype)
    a = _decode(c)[0]
    rng = np.random.default_rng(0)
    perm = rng.permutation(len(c["pool"]))
    moved = np.empty_like(c["pool"])
    moved[perm] = c["pool"]
    c["table"] = np.where(c["table"] >= 0, perm[c["table"]], -1).astype(np.int32)
    c["pool"] = moved
    assert torch.equal(a, _decode(c)[0])


def test_decode_with_shared_prefix_blocks():
    _against_reference(make(22, [300, 290, 161, 300], 8, 2, 128, 16, BF16, shared_blocks=10))


def test_decode_again_gives_the_same_bits():
    c = make(23, [4000, 100, 2500], 32, 8, 128, 16, BF16)
    a = _decode(c)[0]
    assert all(torch.equal(a, _decode(c)[0]) for _ in range(3))


def test_decode_on_a_stream_of_its_own():
    c = make(24, [700, 30], 8, 2, 128, 16, BF16)
    want = _decode(c)[0]
    g = _dev(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(g["q"])
    pa.pa_decode_q4(g["q"], g["pool"], g["table"], g["lens"], g["k_new"], g["v_new"], out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_outputs_made_for_another_stream_take_no_memory_in_use():
    """A tensor that the current stream has yet to read is given up; what a call
    on a side stream allocates must not lie there."""
    c = make(37, [700, 30], 8, 2, 128, 16, BF16)
    g = _dev(c)
    n = 4096
    lens, new, free, count = (torch.zeros(k, dtype=torch.int32, device=DEV) for k in (n, n, 8, 1))
    table = torch.full((n, 1), -1, dtype=torch.int32, device=DEV)
    slots = torch.empty(4, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    calls = [((2, 8, 128), BF16, lambda: pa.pa_decode_q4(g["q"], g["pool"], g["table"], g["lens"], g["k_new"],
                                                         g["v_new"], stream=side)),
             ((n + 1,), torch.int32, lambda: pa.pa_block_tables(lens, new, table, free, count, slots, 16, stream=side))]
    for shape, dtype, call in calls:
        call()  # workspaces and code are there
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        x = [torch.full(shape, 3, dtype=dtype, device=DEV) for _ in range(3)]
        y = [torch.zeros(shape, dtype=dtype, device=DEV) for _ in range(3)]
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # a tenth of a second
        for a, b in zip(x, y):
            b.copy_(a)
        del x, a
        kept = call()
        torch.cuda.synchronize()
        assert all((b == 3).all() for b in y)
        del kept


def test_a_refused_launch_is_not_reported_again_by_a_later_call():
    """Launches into a capture that has become void fail on the host.  The next
    good call of another kind must not answer with that error."""
    cudart = ctypes.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")
    c = make(38, [20, 30], 8, 2, 128, 16, BF16)
    g = _dev(c)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    out, ws = torch.empty_like(g["q"]), torch.zeros(4 << 20, dtype=torch.uint8, device=DEV)
    slots, cu, one = i32(0, 1), i32(0, 1, 2), i32(0)
    chunk, pool = g["k_new"], torch.zeros(4, 16, 2, 128, dtype=BF16, device=DEV)
    table, free = torch.full((2, 2), -1, dtype=torch.int32, device=DEV), i32(0, 1, 2, 3)
    outs = dict(cu_seq_lens_q=cu.clone(), cu_seq_lens_k=cu.clone(), seqlens_k=i32(0, 0))
    calls = [lambda s: pa.pa_cache_update_q4(chunk, chunk, slots, g["pool"], stream=s),
             lambda s: pa.pa_cache_gather_q4(g["pool"], g["table"], cu, chunk.clone(), chunk.clone(), stream=s),
             lambda s: pa.pa_decode_q4(g["q"], g["pool"], g["table"], g["lens"], chunk, chunk, out, workspace=ws, stream=s),
             lambda s: pa.pa_block_tables(i32(0, 0), i32(0, 0), table, free, one, slots, 16, stream=s, **outs)]
    good = lambda: pa.pa_cache_update(chunk, chunk, cu, i32(0, 0), i32(0, 1).view(2, 1), pool, pool)  # noqa: E731
    for call in calls:
        call(None)
        torch.cuda.synchronize()
        side, graph = torch.cuda.Stream(), ctypes.c_void_p()
        handle = ctypes.c_void_p(side.cuda_stream)
        assert cudart.cudaStreamBeginCapture(handle, 2) == 0  # relaxed
        try:
            assert cudart.cudaStreamSynchronize(handle) != 0  # voids the capture
            cudart.cudaGetLastError()
            with pytest.raises(pa.PAError):
                call(side)
        finally:
            cudart.cudaStreamEndCapture(handle, ctypes.byref(graph))
            cudart.cudaGetLastError()
        good()
    torch.cuda.synchronize()


def test_two_captured_graphs_replay_at_once():
    """Graphs captured without a workspace of their own have one each."""
    cases = [make(25 + i, [3000, 2000, 2600], 8, 2, 128, 16, BF16) for i in range(2)]
    want = [_decode(c)[0] for c in cases]
    graphs, outs, keep = [], [], []
    for c in cases:
        g = _dev(c)
        out = torch.zeros_like(g["q"])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.pa_decode_q4(g["q"], g["pool"], g["table"], g["lens"], g["k_new"], g["v_new"], out)
        graphs.append(graph), outs.append(out), keep.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w)


def test_capture_over_two_streams():
    """A call captured on a stream that is not the current one has a workspace
    of the graph's too, and leaves none of it to later calls on that stream."""
    c = make(27, [3000, 100, 2600], 8, 2, 128, 16, BF16)
    want = _decode(c)[0]
    a, b = _dev(c), _dev(c)
    outs = [torch.zeros_like(a["q"]) for _ in range(3)]
    side = torch.cuda.Stream()
    call = lambda g, out, **kw: pa.pa_decode_q4(  # noqa: E731
        g["q"], g["pool"], g["table"], g["lens"], g["k_new"], g["v_new"], out, **kw)
    held = dict(pa._q4_workspaces)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        call(b, outs[1], stream=side)
        call(a, outs[0])
        torch.cuda.current_stream().wait_stream(side)
    assert pa._q4_workspaces == held
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    call(b, outs[2], stream=side)
    side.synchronize()
    for out in outs:
        assert torch.equal(out, want)


def test_one_workspace_for_calls_of_different_sizes():
    cases = [make(30, [900, 20], 8, 2, 128, 16, BF16), make(31, list(range(0, 900, 9)), 16, 16, 64, 32, F32),
             make(32, [6000], 8, 1, 128, 32, BF16)]
    size = max(pa.pa_decode_q4_workspace_size(c["q"].shape[0], c["q"].shape[1], c["k_new"].shape[1], c["q"].shape[2],
                                              c["bs"], c["q"].dtype) for c in cases)
    ws = torch.zeros(max(size, 16), dtype=torch.uint8, device=DEV)
    for _ in range(2):
        for c in cases:
            _against_reference(c, workspace=ws)


def test_reset_zeroes_the_kept_workspaces():
    """What a call that gave up may leave behind: counters that are not zero,
    and sums of another call."""
    c = make(36, [3000, 20, 2500], 8, 2, 128, 16, BF16)
    want = _decode(c)[0]
    key = torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream
    kept = pa._q4_workspaces[key]
    for left in (1, 2, 17):
        kept[:4 * 6].view(torch.int32).fill_(left)
        pa.pa_reset_workspaces()
        assert not kept.any() and pa._q4_workspaces[key] is kept
        assert torch.equal(_decode(c)[0], want)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 8, 2), (128, 32, 16, 8)])
def test_serving_steps(d, bs, hq, hkv):
    """Prompts and tokens of four requests through all four operators: tables
    and slots on the GPU, the chunk into the pool, whole sequences read back
    for the varlen attention, then decode steps; one request ends and its
    blocks serve the others."""
    g = torch.Generator().manual_seed(77)
    rnd = lambda *s: torch.randn(*s, generator=g).to(BF16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    b, mb, nb = 4, 12, 30
    pool = pa.pa_q4_pool(nb, hkv, d, bs)
    table = torch.full((b, mb), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(nb, generator=g).int().to(DEV)
    count, err = i32([nb]), i32([0])
    lens = i32([0] * b)
    hpool, hist = np.zeros((nb, hkv, q4.record_bytes(d, bs)), dtype=np.uint8), [0] * b
    for new in ([37, 1, 0, 64], [3, 20, 50, 9]):  # two prefill chunks
        total = sum(new)
        slots = torch.empty(total + 5, dtype=torch.int32, device=DEV)
        cu_q, cu_k, after = pa.pa_block_tables(lens, i32(new), table, free, count, slots, bs, dev_err=err)
        k, v, q = rnd(total + 5, hkv, d), rnd(total + 5, hkv, d), rnd(total, hq, d)
        pa.pa_cache_update_q4(k.to(DEV), v.to(DEV), slots, pool, dev_err=err)
        tk = sum(hist) + total
        kf = torch.empty(tk, hkv, d, dtype=BF16, device=DEV)
        vf = torch.empty_like(kf)
        pa.pa_cache_gather_q4(pool, table, cu_k, kf, vf, dev_err=err)
        hist = [h + n for h, n in zip(hist, new)]
        out = pa.pa_varlen(q.to(DEV), kf, vf, cu_q, cu_k, max(new), max(hist), True, dev_err=err)
        assert err.item() == 0
        for i, s in enumerate(slots.cpu().tolist()):
            if s >= 0:
                q4.write(hpool, s, _f32(k[i]), _f32(v[i]), bs)
        at = 0
        for r in range(b):
            kk, vv, _, _ = q4.read(hpool, table[r].cpu().numpy(), hist[r], d, bs)
            kk, vv = (torch.from_numpy(x).float().to(BF16).double() for x in (kk, vv))
            for i in range(new[r]):
                n = hist[r] - new[r] + i + 1
                w = torch.einsum("hgd,thd->hgt", q[at].double().view(hkv, -1, d), kk[:n]) * d ** -0.5
                ref = torch.einsum("hgt,thd->hgd", torch.softmax(w, -1), vv[:n]).reshape(hq, d)
                assert (out[at].cpu().double() - ref).abs().max() <= 1e-2 + 1e-2 * ref.abs().max()
                at += 1
        lens = after
    ending = 3
    for step in range(bs + 2):
        new = [1] * b
        if step == 2:  # a step between, in which one request only leaves
            new = [0] * b
            new[ending] = -1
        slots = torch.empty(b, dtype=torch.int32, device=DEV)
        before = lens
        _, _, lens = pa.pa_block_tables(before, i32(new), table, free, count, slots, bs, dev_err=err)
        if step == 2:
            hist[ending] = 0
            continue
        q, kn, vn = rnd(b, hq, d), rnd(b, hkv, d), rnd(b, hkv, d)
        out = pa.pa_decode_q4(q.to(DEV), pool, table, before, kn.to(DEV), vn.to(DEV), dev_err=err)
        assert err.item() == 0
        tab = table.cpu().numpy()
        ref, seen = q4.decode(_f32(q), hpool, tab, np.array(hist), _f32(kn), _f32(vn), bs)
        check(out, ref, decode_bound(q, seen, ref, BF16, d ** -0.5), f"step {step}", norm=NORM[BF16])
        hist = [h + 1 for h in hist]
        assert lens.cpu().tolist() == hist
    used = sum(-(-h // bs) for h in hist)
    assert count.item() == nb - used
    assert np.unique(np.concatenate([table[r].cpu().numpy()[:-(-hist[r] // bs)] for r in range(b)])).size == used


# ------------------------------------------------------------------ exactness
@pytest.mark.parametrize("d,bs,hq,hkv,left", [(128, 16, 32, 8, 2.0 ** -13), (128, 32, 6, 3, 2.0 ** -13),
                                              (64, 32, 16, 16, 2.0 ** -13), (64, 16, 16, 4, 2.0 ** -13),
                                              (128, 16, 64, 8, 2.1e-4), (64, 32, 40, 8, 2.1e-4)])
def test_decode_bf16_is_off_by_little_but_its_own_rounding(d, bs, hq, hkv, left):
    """The 2-norm of the error is h, that of the reference's own rounding to
    bf16, and beside it e, what the sums before the rounding are off by:
    sqrt(h^2 + e^2), the two being independent.

    Up to 4 heads a kv head: weights are sums of two f16 numbers (2^-22), and a
    score is off by 2^-17 of its largest product, 15 s max|q| scale <= 15 x 0.4 x
    5 x 0.125 < 4, in each of up to 8 steps that add up as roots: < 2^-13 of p, and
    as much of the result at most.

    5 to 8: a weight m 2^k, 1 <= m < 2, is off by an even spread over +-2^-11 2^k,
    2^-11 / (m sqrt(3)) of itself in the root mean square, and 1 / m^2 is
    (1 - 1/4) / (2 log 2) = 0.54 on average over logarithms that are spread evenly:
    2.1e-4.  That meets s (n - 7.5), which is no larger than the spread of the
    values that the result is a mean of.

    The two meet in 2 e h over the root of 16384 elements, 0.3% of h^2 for e = 0.2 h.
    """
    c = make(40 + d + hq, [1100 + 37 * i for i in range(max(4, 16384 // (hq * d)))], hq, hkv, d, bs, BF16)
    codes = c["pool"][:, :, :bs * d]  # middle codes are more frequent than those at the ends, as in normal data
    more = np.random.default_rng(hq).integers(0, 256, codes.shape, dtype=np.uint8)
    codes[:] = ((codes & 15) + (more & 15)) // 2 | ((codes >> 4) + (more >> 4)) // 2 << 4
    out, _, _, _, err = _decode(c)
    assert err == 0
    ref, _ = q4.decode(_f32(c["q"]), c["pool"], c["table"], c["lens"], _f32(c["k_new"]), _f32(c["v_new"]), bs)
    ref = torch.from_numpy(ref)
    size = ref.norm()
    h = float((ref.to(BF16).double() - ref).norm() / size)
    got = float((out.cpu().double() - ref).norm() / size)
    assert got <= (h * h + left * left) ** 0.5 * 1.002, (got, h)


# ------------------------------------------------------------------ the step's tables and its decode
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_decode_of_sequences_left_out(dtype):
    """No output, no append, no error; the others within their bound."""
    c = make(50, [100, 900, 5, 40], 8, 2, 128, 16, dtype)
    _, pool_good, ks_good, _, _ = _decode(c)
    ref, seen = q4.decode(_f32(c["q"]), c["pool"].copy(), c["table"], c["lens"], _f32(c["k_new"]), _f32(c["v_new"]), 16)
    bound = decode_bound(c["q"], seen, ref, dtype, 128 ** -0.5)
    lens = c["lens"].copy()
    for out_of in ([1], [0, 3], [0, 1, 2, 3]):
        c["lens"] = lens.copy()
        c["lens"][out_of] = pa.PA_LEFT_OUT
        out, pool, ks, _, err = _decode(c)
        assert err == 0
        for b in range(4):
            own = c["table"][b][c["table"][b] >= 0]
            if b in out_of:
                assert not out[b].any()
                assert np.array_equal(pool.cpu().numpy()[own], c["pool"][own])
            else:
                # the work is cut in other places, so the sums differ by roundings
                check(out[b:b + 1], ref[b:b + 1], bound[b:b + 1], norm=NORM[dtype])
                assert torch.equal(ks[b], ks_good[b]) and torch.equal(pool[own], pool_good[own])
    c["lens"][2] = -2 ** 31 + 1  # any other negative length is an error
    assert _decode(c)[4] == pa.DEVERR_OVERFLOW


@pytest.mark.parametrize("captured", [False, True])
def test_tables_and_decode_of_one_step(captured):
    """Steps of a server over a fixed batch: lengths and free list in place,
    tables and decode in one graph.  Requests pause and end, others take an ended
    one's blocks in the same step, and its row stays empty for a while: nothing of
    another request may change, and no step raises an error."""
    d, bs, hq, hkv, b, mb, nb = 64, 16, 4, 2, 5, 8, 14
    g = torch.Generator().manual_seed(5)
    rng = np.random.default_rng(5)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    z = lambda *s: torch.zeros(*s, dtype=BF16, device=DEV)  # noqa: E731
    pool, table = pa.pa_q4_pool(nb, hkv, d, bs), torch.full((b, mb), -1, dtype=torch.int32, device=DEV)
    free, count, lens, new, at, err = i32(list(range(nb))), i32([nb]), i32([0] * b), i32([0] * b), i32([0] * b), i32([0])
    slots, cu_q, cu_k = i32([0] * b), i32([0] * (b + 1)), i32([0] * (b + 1))
    q, kn, vn, out = z(b, hq, d), z(b, hkv, d), z(b, hkv, d), z(b, hq, d)

    def step():
        pa.pa_block_tables(lens, new, table, free, count, slots, bs, cu_seq_lens_q=cu_q, cu_seq_lens_k=cu_k,
                           seqlens_k=lens, decode_lens=at, dev_err=err)
        pa.pa_decode_q4(q, pool, table, at, kn, vn, out, dev_err=err)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    hist = [0] * b
    rows = [np.zeros((0, 2, hkv, d), dtype=np.float32) for _ in range(b)]  # every request's own tokens
    taken_over = 0
    for i in range(90):
        todo = [1 if rng.random() < 0.8 else 0 for _ in range(b)]
        for r in range(b):
            if hist[r] == 0 and rng.random() < 0.6:
                todo[r] = 0  # an empty row waits for its next request
            if hist[r] > 20 and rng.random() < 0.06:
                todo[r] = -1
        if sum(-(-(h + max(m, 0)) // bs) for h, m in zip(hist, todo) if m >= 0) > nb:
            todo = [0] * b
            todo[int(np.argmax(hist))] = -1
        xs = [torch.randn(*t.shape, generator=g).to(BF16) for t in (q, kn, vn)]
        for t, x in zip((q, kn, vn), xs):
            t.copy_(x)
        new.copy_(i32(todo))
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert err.item() == 0, i
        tab = table.cpu().numpy()
        for r in range(b):
            if todo[r] < 0:
                hist[r], rows[r] = 0, rows[r][:0]
            elif todo[r] == 1:
                new_row = np.stack([_f32(xs[1][r]), _f32(xs[2][r])])[None]
                rows[r] = np.concatenate([rows[r], new_row])
                hist[r] += 1
        assert lens.tolist() == hist
        owned = [set(tab[r, :-(-hist[r] // bs)].tolist()) for r in range(b)]
        taken_over += sum(hist[r] == 0 and any(o & set(tab[r].tolist()) for o in owned) for r in range(b))
        small = np.zeros((nb, hkv, q4.record_bytes(d, bs)), dtype=np.uint8)
        for r in range(b):
            if todo[r] != 1:
                assert not out[r].any()
            for p in range(hist[r]):
                q4.write(small, int(tab[r, p // bs]) * bs + p % bs, rows[r][p, 0], rows[r][p, 1], bs)
        # the pool holds every living request's tokens, and the outputs are theirs
        for r in range(b):
            got = q4.read(pool.cpu().numpy(), tab[r], hist[r], d, bs)
            want = q4.read(small, tab[r], hist[r], d, bs)
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (i, r)
            if todo[r] == 1:
                ref, seen = q4.decode(_f32(xs[0][r:r + 1]), small, tab[r:r + 1], np.array([hist[r] - 1]),
                                      _f32(xs[1][r:r + 1]), _f32(xs[2][r:r + 1]), bs)
                check(out[r:r + 1], ref, decode_bound(xs[0][r:r + 1], seen, ref, BF16, d ** -0.5), (i, r))
    assert taken_over > 10  # rows of ended requests that name another's blocks


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("b,d,bs,hq,hkv,chunk", [(3, 128, 16, 8, 2, 5), (40, 64, 32, 8, 8, 3), (600, 64, 16, 4, 2, 2)])
def test_steps_back_to_back_are_the_steps_one_by_one(captured, b, d, bs, hq, hkv, chunk):
    """Every call starts while the one before it runs: tables (in place), update by
    their slots and read-back, tables and decode, 24 times without a pause, give
    the bits that the same steps give with a pause behind every call."""
    steps, mb = 24, -(-24 * (chunk + 2) // bs) + 1
    nb = b * mb
    g = torch.Generator(device=DEV).manual_seed(b)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    rows, most = b * chunk, b * steps * (chunk + 1)
    k, v, q, kn, vn = rnd(steps, rows, hkv, d), rnd(steps, rows, hkv, d), rnd(steps, b, hq, d), rnd(steps, b, hkv, d), rnd(
        steps, b, hkv, d)
    grow = torch.randint(0, chunk + 1, (steps, b), generator=g, device=DEV).int()
    one = torch.randint(0, 2, (steps, b), generator=g, device=DEV).int()
    order = torch.randperm(nb, generator=g, device=DEV).int()
    results = []
    for pause in (True, False):
        pool, table, free, count = pa.pa_q4_pool(nb, hkv, d, bs), i32(b, mb) - 1, order.clone(), i32(1) + nb
        lens, at, slots, cu, ck, err = i32(b), i32(b), i32(rows), i32(b + 1), i32(b + 1), i32(1)
        out, kf, vf = rnd(steps, b, hq, d) * 0, torch.zeros(steps, most, hkv, d, dtype=BF16, device=DEV), None
        vf = torch.zeros_like(kf)
        ws = torch.zeros(pa.pa_decode_q4_workspace_size(b, hq, hkv, d, bs), dtype=torch.uint8, device=DEV)
        stop = torch.cuda.synchronize if pause else (lambda: None)

        def tables(new):
            pa.pa_block_tables(lens, new, table, free, count, slots, bs, cu_seq_lens_q=cu, cu_seq_lens_k=ck,
                               seqlens_k=lens, decode_lens=at, dev_err=err)
            stop()

        def chain():
            for i in range(steps):
                tables(grow[i])
                pa.pa_cache_update_q4(k[i], v[i], slots, pool, dev_err=err)
                stop()
                pa.pa_cache_gather_q4(pool, table, ck, kf[i], vf[i], dev_err=err)
                stop()
                tables(one[i])
                pa.pa_decode_q4(q[i], pool, table, at, kn[i], vn[i], out[i], workspace=ws, dev_err=err)
                stop()

        if captured and not pause:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                chain()
            graph.replay()
        else:
            chain()
        torch.cuda.synchronize()
        assert err.item() == 0
        results.append([out, pool, table, lens, free, count, kf, vf])
    for x, y in zip(*results):
        assert torch.equal(x, y)
    assert torch.isfinite(results[0][0]).all() and results[0][3].float().mean() > steps

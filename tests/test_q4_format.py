"""The 4-bit pool's format and the plain references themselves (CPU)."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import q4
from paged_kv_cache_300_gb300 import _build
from tests.q4_util import edge_rows, write_rows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_build.LIB) and shutil.which("nvcc") is None and not os.path.exists(
            "/usr/local/cuda/bin/nvcc"):
        pytest.skip("library not built and no nvcc")
    _build.build()
    return pa.load()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bs", [16, 32])
def test_value_units_are_a_permutation(d, bs):
    t, x = np.meshgrid(np.arange(bs), np.arange(d // 4), indexing="ij")
    assert sorted(q4.v_unit(t, x, d).ravel().tolist()) == list(range(bs * d // 4))


def test_codes_are_within_half_a_step():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((400, 64)) * np.exp(8 * rng.standard_normal((400, 1)))).astype(np.float32)
    n, s, b = q4.quantise(x)
    step = q4.bf16_bits_to_f64(s)[:, None]
    # half a step, and the three fp32 roundings of at most 16 steps in all
    assert (np.abs(q4.values(n, s, b) - x) <= step * (0.5 + 48 * 2.0 ** -24)).all()
    assert n.max() == 15 and n.min() == 0


@pytest.mark.parametrize("row,expect", [
    ([0.0] * 64, [0.0] * 64),
    ([2.5] * 64, [2.5] * 64),
    ([-1.0] + [2.75] * 63, [-1.0] + [2.75] * 63),
    (list(range(16)) * 4, list(range(16)) * 4),
])
def test_rows_that_are_held_exactly(row, expect):
    n, s, b = q4.quantise(np.array([row], dtype=np.float32))
    assert q4.values(n, s, b)[0].tolist() == expect


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan, -3.4e38])
def test_rows_without_a_finite_low_read_as_nan(bad):
    x = np.ones((1, 64), dtype=np.float32)
    x[0, 5] = bad
    n, s, b = q4.quantise(x)
    assert np.isnan(q4.values(n, s, b)).all() and n.max() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_finite_rows_at_the_end_of_the_numbers_read_back_finite(dtype):
    x = edge_rows(dtype)
    assert torch.isfinite(x).all()
    n, s, b = q4.quantise(x.float().numpy())
    v = q4.values(n, s, b)
    step = q4.bf16_bits_to_f64(s)[:, None]
    # half a step, and the three fp32 roundings of at most 16 steps in all
    assert (np.abs(v - x.double().numpy()) <= step * (0.5 + 48 * 2.0 ** -24)).all()
    assert (np.abs(v) <= torch.finfo(torch.float32).max).all()
    if dtype == torch.bfloat16:
        assert torch.isfinite(torch.from_numpy(v).to(dtype)).all()


def test_write_then_read():
    rng = np.random.default_rng(1)
    for d, bs in ((64, 16), (128, 32)):
        pool = np.zeros((3, 2, q4.record_bytes(d, bs)), dtype=np.uint8)
        x = rng.standard_normal((bs + 3, 2, 2, d)).astype(np.float32)
        row = [2, 0]
        for t in range(bs + 3):
            q4.write(pool, row[t // bs] * bs + t % bs, x[t, 0], x[t, 1], bs)
        k, v, _, _ = q4.read(pool, row, bs + 3, d, bs)
        assert np.array_equal(k, q4.values(*q4.quantise(x[:, 0])))
        assert np.array_equal(v, q4.values(*q4.quantise(x[:, 1])))


@pytest.mark.parametrize("d,bs", [(64, 32), (128, 16)])
def test_write_of_many_rows(d, bs):
    rng = np.random.default_rng(2)
    one = rng.integers(0, 256, (6, 3, q4.record_bytes(d, bs)), dtype=np.uint8)
    many = one.copy()
    x = rng.standard_normal((2, 40, 3, d)).astype(np.float32)
    slots = rng.permutation(6 * bs)[:40].astype(np.int32)
    slots[[3, 20]] = -1
    for i, s in enumerate(slots):
        if s >= 0:
            q4.write(one, int(s), x[0, i], x[1, i], bs)
    write_rows(many, slots, x[0], x[1], bs)
    assert np.array_equal(one, many)


def test_block_bytes(lib):
    assert lib.pa_q4_block_bytes(8, 128, 16) == 8 * 16 * 136
    assert lib.pa_q4_block_bytes(3, 64, 32) == 3 * 32 * 72
    for bad in ((8, 96, 16), (8, 128, 8), (0, 128, 16), (8, 128, 64)):
        assert lib.pa_q4_block_bytes(*bad) == 0


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _update(lib, **o):
    a = dict(k=4096, v=4096, slots=4096, pool=4096, t=4, hkv=2, d=128, nb=8, bs=16, dt=1)
    a.update(o)
    return lib.pa_cache_update_q4(_p(a["k"]), _p(a["v"]), _p(a["slots"]), _p(a["pool"]), a["t"], a["hkv"], a["d"],
                                  a["nb"], a["bs"], a["dt"], None, None)


def _gather(lib, **o):
    a = dict(pool=4096, tab=4096, cu=4096, k=4096, v=4096, b=2, t=4, hkv=2, d=128, nb=8, bs=16, mb=4, dt=1)
    a.update(o)
    return lib.pa_cache_gather_q4(_p(a["pool"]), _p(a["tab"]), _p(a["cu"]), _p(a["k"]), _p(a["v"]), a["b"], a["t"],
                                  a["hkv"], a["d"], a["nb"], a["bs"], a["mb"], a["dt"], None, None)


def _decode(lib, **o):
    a = dict(q=4096, pool=4096, tab=4096, sl=4096, kn=4096, vn=4096, out=4096, ks=None, vs=None, b=2, hq=8, hkv=2,
             d=128, nb=8, bs=16, mb=4, dt=1, ws=None, wsb=0)
    a.update(o)
    return lib.pa_decode_q4(_p(a["q"]), _p(a["pool"]), _p(a["tab"]), _p(a["sl"]), _p(a["kn"]), _p(a["vn"]),
                            _p(a["out"]), _p(a["ks"]), _p(a["vs"]), a["b"], a["hq"], a["hkv"], a["d"], a["nb"],
                            a["bs"], a["mb"], a["dt"], 0.0, _p(a["ws"]), a["wsb"], None, None)


def _tables(lib, **o):
    a = dict(sl=4096, new=4096, tab=4096, free=4096, nf=4096, slots=4096, cq=4096, ck=4096, lens=4096, nfo=4096, b=2,
             n=4, nb=8, bs=16, mb=4)
    a.update(o)
    return lib.pa_block_tables(_p(a["sl"]), _p(a["new"]), _p(a["tab"]), _p(a["free"]), _p(a["nf"]), _p(a["slots"]),
                               _p(a["cq"]), _p(a["ck"]), _p(a["lens"]), _p(a["nfo"]), a["b"], a["n"], a["nb"],
                               a["bs"], a["mb"], None, None)


COMMON = [(dict(dt=7), -2), (dict(hkv=0), -3), (dict(nb=0), -3), (dict(d=96), -4), (dict(bs=8), -4),
          (dict(bs=64), -4), (dict(nb=1 << 28), -4), (dict(pool=None), -1), (dict(pool=4096 + 8), -3)]


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(t=-1), -3), (dict(k=None), -1), (dict(slots=None), -1), (dict(v=4096 + 4), -3), (dict(slots=4098), -3),
    (dict(t=0, k=None), 0), (dict(t=(1 << 30) - 32, hkv=2), -4)])
def test_update_refuses_before_any_launch(lib, over, status):
    assert _update(lib, **over) == status


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(t=-1), -3), (dict(b=-1), -3), (dict(mb=0), -3), (dict(v=None), -1), (dict(cu=None), -1),
    (dict(k=4096 + 4), -3), (dict(tab=4097), -3), (dict(t=0, k=None), 0), (dict(b=0, cu=None), 0)])
def test_gather_refuses_before_any_launch(lib, over, status):
    assert _gather(lib, **over) == status


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(hq=0), -3), (dict(hq=7), -3), (dict(mb=0), -3), (dict(b=-1), -3), (dict(hq=18), -4),
    (dict(b=1 << 18, hkv=2), -4), (dict(q=None), -1), (dict(out=None), -1), (dict(sl=None), -1),
    (dict(vn=4096 + 8), -3), (dict(ks=4096 + 2), -3), (dict(tab=4099), -3), (dict(b=0, q=None), 0)])
def test_decode_refuses_before_any_launch(lib, over, status):
    assert _decode(lib, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(b=-1), -3), (dict(n=-1), -3), (dict(nb=0), -3), (dict(bs=0), -3), (dict(mb=0), -3), (dict(b=16385), -4),
    (dict(nb=1 << 27), -4), (dict(mb=1 << 27), -4), (dict(cq=None), -1), (dict(nf=None), -1), (dict(free=None), -1),
    (dict(sl=None), -1), (dict(tab=None), -1), (dict(slots=None), -1), (dict(slots=4097), -3), (dict(lens=4098), -3)])
def test_tables_refuse_before_any_launch(lib, over, status):
    assert _tables(lib, **over) == status


def test_tables_with_decode_lens_refuse_before_any_launch(lib):
    p = _p(4096)
    call = lambda **o: lib.pa_block_tables_decode(*[p] * 10, o.get("at", p), o.get("b", 2), 4, 8, 16, 4, None, None)  # noqa: E731
    assert call(at=_p(4098)) == -3 and call(b=-1) == -3 and call(b=16385, at=None) == -4


def test_binding_refuses_what_it_cannot_take():
    z = torch.zeros
    with pytest.raises(ValueError):  # not on a GPU
        pa.pa_cache_update_q4(z(1, 2, 64).bfloat16(), z(1, 2, 64).bfloat16(), z(1, dtype=torch.int32),
                              z(4, 2, 16 * 72, dtype=torch.uint8))
    with pytest.raises(ValueError):
        pa.pa_block_tables(*(z(1, dtype=torch.int32),) * 2, z(1, 4, dtype=torch.int32),
                           *(z(1, dtype=torch.int32),) * 3, 16)


def test_reset_zeroes_what_is_kept(monkeypatch):
    kept = [torch.ones(16, dtype=torch.uint8) for _ in range(3)]
    monkeypatch.setattr(pa, "_workspaces", {(0, 0): kept[0], (0, 7): kept[1]})
    monkeypatch.setattr(pa, "_q4_workspaces", {(0, 0): kept[2]})
    pa.pa_reset_workspaces()
    assert not any(t.any() for t in kept)


def test_table_reference_worked_example():
    """Three requests of 30, 32 and 70 tokens in blocks of 32, one new token
    each: only the second needs a block; then the first ends and the third
    takes its block."""
    table = np.full((3, 4), -1, dtype=np.int32)
    table[0, 0], table[1, 0], table[2, :3] = 2, 0, [3, 5, 6]
    free = np.full(8, -1, dtype=np.int32)
    free[:3] = [7, 4, 1]
    t, f, n, slots, cu_q, cu_k, lens = q4.block_tables([30, 32, 70], [1, 1, 1], table, free, 3, 5, 32)
    assert t[1].tolist() == [0, 1, -1, -1] and n == 2 and slots.tolist() == [2 * 32 + 30, 32, 6 * 32 + 6, -1, -1]
    assert cu_q.tolist() == [0, 1, 2, 3] and cu_k.tolist() == [0, 31, 64, 135] and lens.tolist() == [31, 33, 71]
    t, f, n, slots, _, _, lens = q4.block_tables([31, 33, 71], [-1, 0, 26], t, f, n, 26, 32)
    assert t[2].tolist() == [3, 5, 6, 2] and n == 2 and slots[-1] == 2 * 32 and lens.tolist() == [0, 33, 97]
    assert q4.block_tables([0], [200], table[:1], free, 3, 300, 32) is None  # longer than the row
    assert q4.block_tables([0, 0], [64, 64], table[:2], free, 3, 300, 32) is None  # three free blocks


def test_gather_refuses_a_grid_past_31_bits(lib):
    assert _gather(lib, b=2 ** 31 - 1, t=64) == -4
    assert _gather(lib, b=2 ** 31 - 4, t=64, k=None) == -4
    assert _gather(lib, b=2 ** 31 - 5, t=64, k=None) == -1

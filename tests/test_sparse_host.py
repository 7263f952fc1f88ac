"""Refusals of the rotary and block-sparse calls that the host sees, and the plain
references (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_300_gb300 as pa
from oracle import sparse as ref
from tests.test_abi import lib  # noqa: F401  (the module's fixture)

P = ctypes.c_void_p


def _call(lib, name, order, args, over):
    a = dict(args, **over)
    return getattr(lib, name)(*[a[k] for k in order])


ROT = dict(q=P(4096), k=P(8192), positions=P(4096), cos_sin=P(4096), q_out=P(4096), k_out=P(4096), tokens=4, hq=8, hkv=2, d=128, rot=128,
           maxpos=10, axes=1, pair_axis=None, inter=0, qs=1024, ks=256, qos=1024, kos=256, dtype=1, err=None, stream=None)
APP = dict(q=P(4096), k=P(4096), v=P(4096), slots=P(4096), kc=P(4096), vc=P(4096), bounds=P(4096), positions=P(4096), cos_sin=P(4096),
           q_out=P(4096), tokens=4, hq=8, hkv=2, d=128, rot=64, maxpos=10, axes=1, pair_axis=None, inter=0, qs=1024, ks=256, vs=256,
           qos=1024, nb=4, bs=16, dtype=1, err=None, stream=None)
SEL = dict(q=P(4096), bounds=P(4096), table=P(4096), lens=P(4096), cu=None, selected=P(4096), batch=2, tq=2, hq=8, hkv=2, d=128, nb=4,
           bs=16, mb=9, top=4, first=1, last=1, dtype=1, err=None, stream=None)
SPA = dict(q=P(4096), kc=P(4096), vc=P(4096), table=P(4096), lens=P(4096), cu=None, selected=P(4096), out=P(4096), batch=2, tq=2, hq=8,
           hkv=2, d=128, nb=4, bs=16, mb=9, top=4, dtype=1, scale=0.0, err=None, stream=None)


def _axes(*x):
    return (ctypes.c_uint8 * len(x))(*x)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=5), -2), (dict(tokens=-1), -3), (dict(d=96, rot=96), -4), (dict(rot=0), -3), (dict(rot=130), -3), (dict(rot=24), -4),
    (dict(axes=0), -3), (dict(axes=5), -4), (dict(axes=3), -1), (dict(axes=3, pair_axis=_axes(*[3] * 64)), -3),
    (dict(pair_axis=_axes(*[1] * 64)), -3), (dict(maxpos=0), -3), (dict(q=None), -1), (dict(k_out=None), -1), (dict(positions=None), -1),
    (dict(cos_sin=P(4100)), -3), (dict(q=P(4104)), -3), (dict(qos=1016), -3), (dict(ks=250), -3), (dict(ks=-256), -3),
    (dict(tokens=0, q=None), 0), (dict(hq=0, hkv=0), 0), (dict(hkv=-1), -3),
])
def test_rotary_refusals(lib, over, status):  # noqa: F811
    order = "q k positions cos_sin q_out k_out tokens hq hkv d rot maxpos axes pair_axis inter qs ks qos kos dtype err stream".split()
    assert _call(lib, "pa_rotary", order, ROT, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=-1), -2), (dict(tokens=-1), -3), (dict(d=80, rot=16), -4), (dict(hkv=0), -3), (dict(nb=0), -3), (dict(bs=0), -3),
    (dict(nb=1 << 28), -4), (dict(axes=9), -4), (dict(axes=2), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(kc=None), -1),
    (dict(q_out=None), -1), (dict(positions=None), -1), (dict(bounds=P(4104)), -3), (dict(vc=P(4104)), -3), (dict(slots=P(4098)), -3),
    (dict(vs=12), -3), (dict(qos=1000), -3), (dict(tokens=0, k=None), 0), (dict(rot=0, cos_sin=None, positions=None, kc=None), -1),
])
def test_append_refusals(lib, over, status):  # noqa: F811
    order = ("q k v slots kc vc bounds positions cos_sin q_out tokens hq hkv d rot maxpos axes pair_axis inter qs ks vs qos nb bs dtype "
             "err stream").split()
    assert _call(lib, "pa_cache_append_rotary", order, APP, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), -2), (dict(batch=-1), -3), (dict(tq=3), -3), (dict(hq=7), -3), (dict(hq=18), -4), (dict(d=32), -4), (dict(top=0), -3),
    (dict(first=-1), -3), (dict(first=3, last=2), -3), (dict(first=2**31 - 1, last=2**31 - 1), -3), (dict(mb=49153), -4),
    (dict(nb=1 << 27, bs=16), -4), (dict(mb=40000, bs=1 << 16), -4), (dict(tq=1 << 26, batch=1 << 26), -4), (dict(top=(1 << 20) + 1), -4),
    (dict(q=None), -1), (dict(selected=None), -1), (dict(bounds=P(4104)), -3), (dict(lens=P(4097)), -3),
    (dict(batch=0, tq=0, q=None), 0), (dict(cu=P(4096), tq=0, q=None), 0),
])
def test_select_refusals(lib, over, status):  # noqa: F811
    order = "q bounds table lens cu selected batch tq hq hkv d nb bs mb top first last dtype err stream".split()
    assert _call(lib, "pa_select_blocks", order, SEL, over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), -2), (dict(batch=-1), -3), (dict(tq=1), -3), (dict(hq=7), -3), (dict(hq=18), -4), (dict(d=96), -4), (dict(top=-4), -3),
    (dict(bs=24), -4), (dict(bs=8), -4), (dict(nb=1 << 27), -4), (dict(kc=None), -1), (dict(out=None), -1), (dict(vc=P(4104)), -3),
    (dict(selected=P(4098)), -3), (dict(batch=0, tq=0, q=None), 0), (dict(top=1 << 20, bs=1 << 10), -4), (dict(top=(1 << 20) + 1), -4),
])
def test_sparse_refusals(lib, over, status):  # noqa: F811
    order = "q kc vc table lens cu selected out batch tq hq hkv d nb bs mb top dtype scale err stream".split()
    assert _call(lib, "pa_sparse", order, SPA, over) == status


def test_bindings_refuse_cpu_tensors(lib):  # noqa: F811
    t = torch.zeros(1, 8, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    c = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: pa.pa_rotary(t, t, i, torch.zeros(4, 64)), lambda: pa.pa_rotary(None, None, i, torch.zeros(4, 64)),
                 lambda: pa.pa_cache_append_rotary(t, t, t, i, c, c), lambda: pa.pa_select_blocks(t, c, i.view(1, 1), i, 4, 16),
                 lambda: pa.pa_sparse(t, c, c, i.view(1, 1), i, i.view(1, 1, 1))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the references
def test_reference_rotary_turns_as_complex_numbers_do():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 8))
    angle = rng.standard_normal((9, 3))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = np.array([[3, 1, 4, 1, 5], [2, 7, 1, 8, 2]])
    for inter in (False, True):
        y, mag = ref.rotary(x, pos, table, [0, 1, 0], inter)
        a, b = (x[..., 0:6:2], x[..., 1:6:2]) if inter else (x[..., :3], x[..., 3:6])
        z = (a + 1j * b) * np.exp(1j * np.stack([angle[pos[0], 0], angle[pos[1], 1], angle[pos[0], 2]], 1))[:, None]
        c, d = (y[..., 0:6:2], y[..., 1:6:2]) if inter else (y[..., :3], y[..., 3:6])
        assert np.allclose(c, z.real, atol=1e-15) and np.allclose(d, z.imag, atol=1e-15)
        assert np.array_equal(y[..., 6:], x[..., 6:]) and (mag >= abs(y) - 1e-15).all()


def test_reference_score_bounds_every_key():
    rng = np.random.default_rng(1)
    keys, q = rng.standard_normal((6, 10, 16)), rng.standard_normal((3, 16))
    lo, hi = zip(*(ref.bounds_of(k) for k in keys))
    s = ref.scores(q, np.array(lo), np.array(hi))
    assert (s >= np.einsum("gd,bnd->bgn", q, keys).max((1, 2))).all()
    one = ref.scores(q, keys[:, 0], keys[:, 0])  # a block of one key: its own score
    assert np.allclose(one, (keys[:, 0] @ q.T).max(1))


def test_reference_choice():
    s = np.array([1.0, 5, 5, 3, np.nan, 0, 9])
    assert ref.choose(s, 7, 4, 1, 1).tolist() == [0, 1, 4, 6]
    assert ref.choose(s, 7, 4, 0, 0).tolist() == [1, 2, 4, 6]
    assert ref.choose(s, 3, 5, 1, 1).tolist() == [0, 1, 2, -1, -1]
    assert ref.choose(s, 0, 2, 1, 1).tolist() == [-1, -1]


def test_reference_attention_is_dense_attention_when_all_is_selected():
    rng = np.random.default_rng(2)
    kc, vc, q = rng.standard_normal((4, 2, 1, 8)), rng.standard_normal((4, 2, 1, 8)), rng.standard_normal((3, 2, 8))
    table = np.array([[2, 0, 3]])
    sel = np.tile(np.arange(3), (3, 1, 1))
    out, info = ref.attend(q, kc, vc, table, [5], sel, 0.3, [0, 3])
    k, v = kc[table[0]].reshape(-1, 8), vc[table[0]].reshape(-1, 8)
    for t in range(3):
        w = np.exp(q[t] @ k[:3 + t].T * 0.3)
        assert np.allclose(out[t], w @ v[:3 + t] / w.sum(1, keepdims=True))
    assert info[:, 0, 2].tolist() == [3, 4, 5]

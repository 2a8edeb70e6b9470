"""Head norms, position rotation and the append: the oracle's pins, the host table, and the
refusals that the host makes before anything is enqueued."""

import math

import numpy as np
import pytest
import torch

from oracle import append_oracle as ao

DUMMY = 1 << 20


@pytest.fixture(scope="module")
def tq():
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


# ---------------------------------------------------------------- pins

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [2, 6, 8])
def test_a_rotation_keeps_norms_and_adds_angles(rot, interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 3, 8))
    table = ao.rope_table(rot, 40)
    one = ao.rotate(x, np.full(7, 11), table, interleaved)[0]
    assert np.allclose(np.linalg.norm(one, axis=2), np.linalg.norm(x, axis=2))
    assert np.array_equal(one[:, :, rot:], x[:, :, rot:])
    twice = ao.rotate(one, np.full(7, 9), table, interleaved)[0]
    assert np.allclose(twice, ao.rotate(x, np.full(7, 20), table, interleaved)[0])
    # a score depends on the distance of the two positions alone
    y = rng.standard_normal((7, 3, 8))
    near = [(ao.rotate(x, np.full(7, p), table, interleaved)[0] * ao.rotate(y, np.full(7, p + 4), table, interleaved)[0]).sum(2)
            for p in (0, 30)]
    assert np.allclose(*near)


def test_pairs_of_both_styles_are_the_same_up_to_channel_order():
    x = np.random.default_rng(1).standard_normal((5, 2, 16))
    table, pos = ao.rope_table(16, 50), np.array([0, 1, 7, 30, 49])
    order = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    assert np.allclose(ao.rotate(x, pos, table, True)[0][:, :, order], ao.rotate(x[:, :, order], pos, table, False)[0])


def test_norm():
    x = np.array([[[3.0, -4.0, 0.0, 0.0]]])
    assert np.allclose(ao.norm_heads(x, np.array([1, 2, 3, 4.0]), 0.0), [[[3 / 2.5, -8 / 2.5, 0, 0]]])
    assert np.allclose(ao.norm_heads(x, np.ones(4), 6.25), x / math.sqrt(12.5))


# ---------------------------------------------------------------- the table

@pytest.mark.parametrize("rot,rows,base", [(2, 5, 10000.0), (64, 300, 10000.0), (128, 70, 500000.0), (6, 4, 7.0)])
def test_table_matches_the_oracle(tq, rot, rows, base):
    got = tq.tq_build_rope(rot, rows, base).numpy()
    want = ao.rope_table(rot, rows, base)
    assert got.dtype == np.float32 and got.shape == want.shape
    # fp64 angles and functions, rounded once: half a step of a number up to 1, and what the two
    # powers' last bits move an angle below 300
    assert np.abs(got - want).max() <= 2.0 ** -25 + 300 * 2.0 ** -51


def test_table_far_positions_and_given_frequencies(tq):
    freq = np.array([1.0, 0.25, 1e-3])
    got = tq.tq_build_rope(6, 131072, inv_freq=torch.from_numpy(freq)).numpy()
    for p in (0, 1, 999, 65537, 131071):
        angle = p * freq
        assert np.abs(got[p] - np.concatenate([np.cos(angle), np.sin(angle)])).max() <= 2.0 ** -25 + 2.0 ** -50
    assert tq.tq_build_rope(8, 0).shape == (0, 8)


def test_table_refusals(tq):
    f = tq.lib().tq_build_rope
    assert f(7, 4, 10.0, None, DUMMY) == tq.TQ_ERR_UNSUPPORTED
    assert f(0, 4, 10.0, None, DUMMY) == tq.TQ_ERR_UNSUPPORTED
    assert f(258, 4, 10.0, None, DUMMY) == tq.TQ_ERR_UNSUPPORTED
    assert f(8, -1, 10.0, None, DUMMY) == tq.TQ_ERR_INVALID_ARG
    assert f(8, 4, 10.0, None, None) == tq.TQ_ERR_INVALID_ARG
    assert f(8, 4, 0.0, None, DUMMY) == tq.TQ_ERR_INVALID_ARG
    assert f(8, 4, float("nan"), None, DUMMY) == tq.TQ_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="inv_freq"):
        tq.tq_build_rope(8, 4, inv_freq=torch.ones(3))


# ---------------------------------------------------------------- refusals

ROPE = dict(pos=DUMMY, off=0, table=DUMMY, rows=64, rot=128, pairs=0, qw=DUMMY, kw=None, eps=1e-6)


def _rope(tq, **kw):
    a = dict(q=DUMMY, qs=4096, hq=32, k=DUMMY, ks=1024, h=8, t=1, n=4, d=128, **ROPE, qo=DUMMY * 2, qos=4096, ko=DUMMY * 2,
             kos=1024)
    a.update(kw)
    return tq.lib().tq_norm_rope(*a.values(), None, None)


def _append(tq, **kw):
    a = dict(q=DUMMY, qs=4096, hq=32, qo=DUMMY * 2, qos=4096, k=DUMMY, ks=1024, v=DUMMY, vs=1024, t=1, n=4, h=8, d=128,
             slots=DUMMY, kp=DUMMY, kb=4, vp=DUMMY, vb=2, nb=8, bs=16, signs=DUMMY, kc=DUMMY, vc=DUMMY, **ROPE)
    a.update(kw)
    return tq.lib().tq_append_kv(*a.values(), None, None)


BOTH = [(dict(n=-1), 1), (dict(n=1 << 31), 1), (dict(hq=20000, qs=1 << 23, qos=1 << 23), 2), (dict(d=96), 2), (dict(d=512), 2), (dict(t=3), 1), (dict(rot=0), 1), (dict(rot=130), 1),
        (dict(rot=7), 1), (dict(rows=-1), 1), (dict(pos=None), 1), (dict(pos=DUMMY + 2), 1), (dict(table=DUMMY + 1), 1),
        (dict(qw=DUMMY + 2), 1), (dict(kw=DUMMY + 1), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1),
        (dict(eps=float("inf")), 1), (dict(hq=-1), 1), (dict(qo=None), 1), (dict(q=DUMMY + 1), 1), (dict(qo=DUMMY + 1), 1),
        (dict(qs=4095), 1), (dict(qos=4095), 1), (dict(qo=DUMMY, qos=5000), 1)]


@pytest.mark.parametrize("kw,code", BOTH + [(dict(h=-1), 1), (dict(h=20000, ks=1 << 23, kos=1 << 23), 2), (dict(ko=None), 1), (dict(ks=1023), 1), (dict(k=DUMMY + 1), 1)])
def test_norm_rope_host_refusals(tq, kw, code):
    assert _rope(tq, **kw) == code
    assert tq.lib().tq_last_error().decode()


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(h=0), 1), (dict(h=20000, ks=1 << 23, vs=1 << 23), 2), (dict(nb=-1), 1), (dict(bs=0), 1), (dict(kb=1), 2), (dict(vb=6), 2), (dict(slots=None), 1),
    (dict(slots=DUMMY + 4), 1), (dict(kp=None), 1), (dict(vp=DUMMY + 8), 1), (dict(signs=None), 1), (dict(vc=None), 1),
    (dict(ks=1023), 1), (dict(vs=1000), 1), (dict(v=DUMMY + 1), 1), (dict(kc=DUMMY + 2), 1)])
def test_append_host_refusals(tq, kw, code):
    assert _append(tq, **kw) == code
    assert tq.lib().tq_last_error().decode()


def test_bindings_refuse(tq):
    q, k = torch.zeros(4, 8, 64), torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="same CUDA device"):
        tq.tq_norm_rope(q, k)
    with pytest.raises(ValueError, match="expected"):
        tq.tq_norm_rope(None, None)
    with pytest.raises(ValueError, match="expected"):
        tq.tq_norm_rope(q.long(), k)
    with pytest.raises(ValueError, match="same CUDA device"):
        tq.tq_append_kv(q, k, k, None, None, torch.zeros(4, dtype=torch.int64), torch.ones(64), None, None)
    with pytest.raises(ValueError, match="expected"):
        tq.tq_append_kv(None, None, None, None, None, torch.zeros(4, dtype=torch.int64), torch.ones(64), None, None)

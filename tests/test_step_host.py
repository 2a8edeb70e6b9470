"""Refusals of the serving-step calls that the host makes before anything is enqueued."""

import pytest
import torch

DUMMY = 1 << 20


@pytest.fixture(scope="module")
def tq():
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


def _plan(tq, **kw):
    a = dict(lens=DUMMY, new=DUMMY, blocks=DUMMY, s=2, table=DUMMY, w=4, ring=DUMMY, state=DUMMY, nb=8, bs=16, rows=4,
             slots=DUMMY, q_seq=DUMMY, q_len=DUMMY, starts=DUMMY, lo=DUMMY, bo=DUMMY, fo=DUMMY)
    a.update(kw)
    return tq.lib().tq_plan_step(*a.values(), None, None)


@pytest.mark.parametrize("kw", [dict(s=-1), dict(w=-1), dict(nb=-1), dict(nb=1 << 31), dict(bs=0), dict(rows=-1),
                                dict(rows=1 << 31), dict(lens=None), dict(new=None), dict(table=None), dict(ring=None),
                                dict(state=None), dict(slots=None), dict(starts=None), dict(fo=None),
                                dict(slots=DUMMY + 4), dict(q_len=DUMMY + 2), dict(lens=DUMMY + 1)])
def test_plan_host_refusals(tq, kw):
    assert _plan(tq, **kw) == tq.TQ_ERR_INVALID_ARG
    assert tq.lib().tq_last_error().decode().startswith("tq_plan_step")


def _commit(tq, **kw):
    a = dict(k=DUMMY, rk=68, v=DUMMY, rv=68, nb=8, bs=16, h=2, table=DUMMY, s=2, w=4, ctx=DUMMY, path=DUMMY, n=DUMMY,
             p=3, out=DUMMY)
    a.update(kw)
    return tq.lib().tq_commit_tree(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [(dict(k=None, v=None), 1), (dict(s=-1), 1), (dict(bs=0), 1), (dict(h=0), 1),
                                     (dict(rk=0), 1), (dict(rv=-4), 1), (dict(p=-1), 1), (dict(path=None), 1),
                                     (dict(out=None), 1), (dict(k=DUMMY + 8), 1), (dict(ctx=DUMMY + 2), 1),
                                     (dict(h=1 << 20), 2)])
def test_commit_host_refusals(tq, kw, code):
    assert _commit(tq, **kw) == code
    assert tq.lib().tq_last_error().decode().startswith("tq_commit_tree")


def _attn(tq, which, **kw):
    a = dict(q=DUMMY, qt=1, t=4, hq=16, h=4, d=128, k=DUMMY, kb=4, v=DUMMY, vb=4, nb=8, bs=16, table=DUMMY, s=2, w=4,
             q_seq=DUMMY)
    a.update(dict(ctx=DUMMY, mask=DUMMY, words=1) if which == "tree" else
             dict(q_len=DUMMY, prefix=None, docs=None, window=0, slopes=None))
    a.update(signs=DUMMY, kc=DUMMY, vc=DUMMY, scale=0.0, cap=0.0, out=DUMMY, ot=1, ws=DUMMY, wb=1 << 40)
    a.update(kw)
    f = tq.lib().tq_paged_tree if which == "tree" else tq.lib().tq_paged_prefill_biased
    return f(*a.values(), None, None)


COMMON = [(dict(hq=15), 1), (dict(hq=12), 2), (dict(d=96), 2), (dict(kb=6), 2), (dict(vb=1), 2), (dict(qt=3), 1),
          (dict(ot=7), 1), (dict(t=-1), 1), (dict(s=-1), 1), (dict(nb=-1), 1), (dict(bs=0), 1), (dict(q=None), 1),
          (dict(out=None), 1), (dict(table=None), 1), (dict(q_seq=None), 1), (dict(signs=None), 1), (dict(vc=None), 1),
          (dict(cap=-1.0), 1), (dict(cap=float("nan")), 1), (dict(cap=float("inf")), 1), (dict(wb=1000), 1),
          (dict(ws=None), 1), (dict(ws=DUMMY + 16), 1), (dict(k=DUMMY + 4), 1), (dict(q=DUMMY + 1), 1),
          (dict(w=1 << 28), 2), (dict(t=1 << 24, w=1 << 20), 2)]


@pytest.mark.parametrize("which,kw,code", [(w, kw, c) for w in ("tree", "biased") for kw, c in COMMON] + [
    ("tree", dict(words=0), 1), ("tree", dict(words=1025), 1), ("tree", dict(mask=None), 1), ("tree", dict(ctx=None), 1),
    ("tree", dict(mask=DUMMY + 2), 1), ("biased", dict(window=-1), 1), ("biased", dict(q_len=None), 1),
    ("biased", dict(prefix=DUMMY + 1), 1), ("biased", dict(slopes=DUMMY + 2), 1), ("biased", dict(docs=DUMMY + 3), 1)])
def test_attention_host_refusals(tq, which, kw, code):
    assert _attn(tq, which, **kw) == code
    assert tq.lib().tq_last_error().decode()


def test_workspace_query(tq):
    f = tq.lib().tq_paged_tree_workspace
    assert f(4, 12, 8, 128) == 0 and f(4, 32, 8, 96) == 0 and f(-1, 32, 8, 128) == 0
    assert 0 < f(1, 16, 2, 128) <= f(4096, 16, 2, 128)


def test_bindings_refuse_host_tensors_and_wrong_shapes(tq):
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="same CUDA device"):
        tq.tq_plan_step(i, i, i, torch.zeros(2, 3, dtype=torch.int32), i, i, 16, 4)
    with pytest.raises(ValueError, match="max_rows"):
        tq.tq_plan_step(i, i, i, torch.zeros(2, 3, dtype=torch.int32), i, i, 16, -4)
    with pytest.raises(ValueError, match="expected"):
        tq.tq_plan_step(i, i, i, i, i, i, 16, 4)
    with pytest.raises(ValueError, match="expected"):
        tq.tq_commit_tree(None, None, i, i, i, i)
    pages = torch.zeros(2, 16, 2, 68, dtype=torch.uint8)
    q, f = torch.zeros(2, 4, 128), torch.zeros(16)
    with pytest.raises(ValueError, match="same CUDA device"):
        tq.tq_commit_tree(pages, pages, torch.zeros(2, 3, dtype=torch.int32), i, torch.zeros(2, 3, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="same CUDA device"):
        tq.tq_paged_tree(q, i, i, torch.zeros(2, 1, dtype=torch.int32), pages, pages, torch.zeros(2, 3, dtype=torch.int32),
                         torch.ones(128), f, f)
    with pytest.raises(ValueError, match="words"):
        tq.tq_paged_tree(q, i, i, i, pages, pages, torch.zeros(2, 3, dtype=torch.int32), torch.ones(128), f, f)
    with pytest.raises(ValueError, match="do not match head_dim"):
        tq.tq_paged_prefill_biased(q, i, i, pages[..., :36], pages, torch.zeros(2, 3, dtype=torch.int32),
                                   torch.ones(128), f, f)
    with pytest.raises(ValueError, match="out must be"):
        tq.tq_paged_prefill_biased(q, i, i, pages, pages, torch.zeros(2, 3, dtype=torch.int32), torch.ones(128), f, f,
                                   out=torch.zeros(2, 4, 128, dtype=torch.int32))

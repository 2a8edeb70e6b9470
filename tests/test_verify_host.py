"""Verification of drafted tokens: the oracle's pins, and the refusals that the host makes before
anything is enqueued."""

import numpy as np
import pytest
import torch

from oracle import verify_oracle as vo

DUMMY = 1 << 20


@pytest.fixture(scope="module")
def tq():
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


# ---------------------------------------------------------------- pins

def test_draw_is_the_inverse_of_the_running_sum():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25])
    assert [vo.draw(w, u)[0] for u in (0.0, 0.2, 0.25, 0.5, 0.75, 0.999, 1.0)] == [1, 1, 3, 3, 4, 4, 4]


def _first_token(rng, p, q, kids, count):
    """Shares of the first token behind the root, over many drafts of `kids` children each."""
    seen = np.zeros(len(p))
    logits = np.tile(np.log(p), (kids + 1, 1))
    for _ in range(count):
        tokens = np.concatenate([[0], rng.choice(len(p), kids, p=q)])
        path, lens, nxt, _ = vo.verify(logits, [0, kids + 1], tokens, rng.random(kids + 1), 8, parents=[0] * (kids + 1),
                                       draft=np.tile(q, (kids + 1, 1)), u_accept=rng.random(kids + 1))
        seen[tokens[path[0, 1]] if lens[0] > 1 else nxt[0]] += 1
    return seen / count


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_tokens_follow_the_targets_distribution(kids):
    # whatever the drafter's: 20000 drafts, five standard deviations
    p, q = np.array([0.5, 0.2, 0.2, 0.1]), np.array([0.1, 0.6, 0.2, 0.1])
    got = _first_token(np.random.default_rng(kids), p, q, kids, 20000)
    assert np.all(np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / 20000))


def test_a_drafter_that_equals_the_target_is_always_kept():
    rng = np.random.default_rng(5)
    p = vo.softmax(rng.standard_normal(9), 1.0)
    for _ in range(50):
        tokens = np.concatenate([[0], rng.choice(9, 3, p=p)])
        path, lens, _, _ = vo.verify(np.tile(np.log(p), (4, 1)), [0, 4], tokens, rng.random(4), 8,
                                     draft=np.tile(p, (4, 1)) * (1 - 1e-12), u_accept=rng.random(4))
        assert lens[0] == 4 and list(path[0, :4]) == [0, 1, 2, 3]


def test_walks():
    logits = np.full((4, 5), -1e9)
    logits[0, 3] = logits[1, 2] = logits[2, 2] = logits[3, 4] = 0.0
    u = np.full(4, 0.5)
    # node 0 -> token 3 is node 2 (its second child), node 2 -> token 2 has no child
    path, lens, nxt, _ = vo.verify(logits, [0, 4], [9, 1, 3, 1], u, 3, parents=[0, 0, 0, 1])
    assert list(path[0]) == [0, 2, -1] and lens[0] == 2 and nxt[0] == 2
    # a walk ends at max_path
    path, lens, nxt, _ = vo.verify(logits, [0, 4], [9, 1, 3, 1], u, 1, parents=[0, 0, 0, 1])
    assert list(path[0]) == [0] and nxt[0] == 3
    # no rows; greedy ties go to the lower index; a row without a distribution
    ties = np.zeros((2, 4))
    ties[1] = -np.inf
    _, lens, nxt, _ = vo.verify(ties, [0, 0, 1, 2], [0, 0], u, 2, temperature=[1.0, 0.0, 1.0])
    assert list(lens) == [0, 1, 1] and list(nxt) == [-1, 0, -1]


# ---------------------------------------------------------------- refusals

def _verify(tq, **kw):
    a = dict(x=DUMMY, xt=1, xs=64, r=6, v=64, q=DUMMY, qt=0, qs=64, start=DUMMY, s=2, tok=DUMMY, up=DUMMY, temp=DUMMY,
             ua=DUMMY, us=DUMMY, path=DUMMY, mp=3, lens=DUMMY, nxt=DUMMY, ws=DUMMY, wb=1 << 30)
    a.update(kw)
    return tq.lib().tq_verify_tree(*a.values(), None, None)


@pytest.mark.parametrize("kw", [
    dict(r=-1), dict(v=0), dict(v=(1 << 30) + 1, xs=1 << 31, qs=1 << 31), dict(s=-1), dict(mp=0), dict(xt=3), dict(qt=-1), dict(x=None), dict(start=None), dict(tok=None),
    dict(us=None), dict(ua=None), dict(path=None), dict(lens=None), dict(nxt=None), dict(xs=63), dict(qs=63),
    dict(x=DUMMY + 1), dict(q=DUMMY + 2), dict(start=DUMMY + 2), dict(up=DUMMY + 1), dict(temp=DUMMY + 3),
    dict(ua=DUMMY + 2), dict(path=DUMMY + 2), dict(wb=1000), dict(ws=None), dict(ws=DUMMY + 16)])
def test_verify_host_refusals(tq, kw):
    assert _verify(tq, **kw) == tq.TQ_ERR_INVALID_ARG
    assert tq.lib().tq_last_error().decode().startswith("tq_verify_tree")


def test_workspace_query(tq):
    f = tq.tq_verify_tree_workspace
    assert f(1, (1 << 30) + 1, 1) == 0 and f(-1, 8, 1) == 0 and f(1, 0, 1) == 0 and f(1, 8, -1) == 0
    assert 256 <= f(0, 1, 0) <= f(1, 8, 1) <= f(64, 131072, 8)


def test_bindings_refuse(tq):
    x, i, f = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError, match="same CUDA device"):
        tq.tq_verify_tree(x, torch.zeros(2, dtype=torch.int32), i, f, 3)
    with pytest.raises(ValueError, match="expected"):
        tq.tq_verify_tree(x[0], torch.zeros(2, dtype=torch.int32), i, f, 3)

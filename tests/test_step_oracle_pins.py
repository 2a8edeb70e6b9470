"""Pins of the serving-step oracle: worked examples by hand, and agreement with the prefill
oracle where the visible set is the causal one."""

import numpy as np
import pytest

from oracle import step_oracle as so
from oracle import tq_oracle as o


def test_plan_worked_example():
    # bs 4: seq 0 has 3 tokens in block 7 and gets 3 (one new block); seq 1 is finished with
    # blocks 2, 5; seq 2 is new with 5 tokens (two blocks); ring of 9, head 8 -> wraps
    table = np.array([[7, 0, 0], [2, 5, 0], [0, 0, 0]])
    ring = np.array([1, 3, 4, -9, -9, -9, -9, -9, 6])
    p = so.plan_step([3, 8, 0], [3, -1, 5], [1, 2, 0], table, ring, [8, 4], 4, 10)
    assert p["table"].tolist() == [[7, 6, 0], [2, 5, 0], [1, 3, 0]]
    assert p["slots"].tolist() == [31, 24, 25, 4, 5, 6, 7, 12, -1, -1]
    assert p["q_seq"].tolist() == [0, 0, 0, 2, 2, 2, 2, 2, -1, -1]
    assert p["q_len"].tolist() == [4, 5, 6, 1, 2, 3, 4, 5, 0, 0]
    assert p["row_start"].tolist() == [0, 3, 3, 8]
    assert p["seq_lens"].tolist() == [6, 0, 5] and p["seq_blocks"].tolist() == [2, 0, 2]
    assert p["free_state"].tolist() == [2, 3]
    assert p["ring"][[2, 3, 4]].tolist() == [4, 2, 5]


@pytest.mark.parametrize("case,kind", [(dict(lens=[5]), "arg"), (dict(new=[9]), "arg"), (dict(state=[0, 0]), "blocks"),
                                       (dict(rows=1), "arg"), (dict(state=[3, 1]), "arg"), (dict(lens=[-1]), "arg")])
def test_plan_refusals(case, kind):
    with pytest.raises(so.PlanError) as e:
        so.plan_step(case.get("lens", [4]), case.get("new", [2]), [1], np.zeros((1, 3), int), np.array([1, 2, 0]),
                     case.get("state", [0, 2]), 4, case.get("rows", 8))
    assert e.value.kind == kind


def test_commit_worked_example():
    pages = np.arange(4 * 2, dtype=np.uint8).reshape(4, 2, 1, 1)
    table = np.array([[2, 0, 3]])
    # context of one token: tokens 1.. hold nodes 0..; keep nodes 1, 3, 4
    out, lens = so.commit_tree(pages, table, [1], np.array([[1, 3, 4]]), [3])
    flat = lambda p: [int(p[table[0, t // 2], t % 2, 0, 0]) for t in range(6)]  # noqa: E731
    assert flat(pages) == [4, 5, 0, 1, 6, 7]
    assert flat(out) == [4, 0, 6, 7, 6, 7] and lens.tolist() == [4]
    same, lens = so.commit_tree(pages, table, [1], np.array([[3, 3, 4]]), [2])
    assert np.array_equal(same, pages) and lens.tolist() == [1]


def test_visible_sets():
    see = so.tree_visible([0, -1], [2], np.array([[0b101], [0xFFFF]], dtype=np.uint32), 6)
    assert see.tolist() == [[True, True, True, False, True, False], [False] * 6]
    see = so.biased_visible([0, 0], [2, 5], 6, 1, window=2, prefix_lens=[1], doc_starts=[0, 4])
    assert see.tolist() == [[True, True] + [False] * 4, [False] * 4 + [True, False]]
    see = so.biased_visible([0], [2], 6, 1, window=1, prefix_lens=[4])
    assert see.tolist() == [[True] * 4 + [False] * 2]


def test_attention_is_the_prefill_oracle_on_the_causal_set():
    rng = np.random.default_rng(5)
    d, h, hq, bs, n = 32, 2, 4, 4, 11
    signs = o.splitmix64_signs(d, 42)
    kc, vc = o.codebook_f32(d, 4)[0], o.codebook_f32(d, 2)[0]
    rows = lambda b: o.make_rows(rng.integers(0, 1 << b, size=(4 * bs * h, d)),  # noqa: E731
                                 rng.lognormal(0, 0.5, 4 * bs * h).astype(np.float32), b).reshape(4, bs, h, -1)
    kp, vp = rows(4), rows(2)
    bt = np.array([[3, 1, 0]], dtype=np.int32)
    q = rng.standard_normal((3, hq, d))
    q_seq, q_len = [0, 0, 0], [n, 1, 6]
    see = so.biased_visible(q_seq, q_len, 12, 1)
    got, _ = so.attention(q, q_seq, see, kp, vp, 4, 2, bt, signs, kc, vc)
    want = o.paged_prefill(q, np.array(q_seq), np.array(q_len), kp, vp, 4, 2, bt, signs, kc, vc)
    assert np.allclose(got, want, atol=1e-12)
    # by differences: a cap far above the scores changes them by x^3 / (3 c^2)
    capped, _ = so.attention(q, q_seq, see, kp, vp, 4, 2, bt, signs, kc, vc, softcap=1e4)
    assert np.abs(capped - got).max() < 1e-5

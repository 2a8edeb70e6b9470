"""CPU oracle of the serving-step calls: step planning, commits of accepted rows, and
attention of query rows with a visible set of their own ("vLLM Usage", Slot Mapping: token t
of a sequence sits at block_table[t / bs] * bs + t % bs; "Architecture", Diagnostic vs Serving
Paths: the decode equals attention on reconstructed rows).

Sequential Python over the definitions; attention in fp64 on dense rows, per (row, q head),
with an explicit boolean row of visible tokens.  Pins live in ``tests/test_step_oracle_pins.py``.
"""

from __future__ import annotations

import math

import numpy as np

from oracle import tq_oracle as o


class PlanError(Exception):
    """kind: "blocks" (the ring holds too few) or "arg"."""

    def __init__(self, kind):
        super().__init__(kind)
        self.kind = kind


def plan_step(seq_lens, new_lens, seq_blocks, block_table, free_blocks, free_state, block_size, max_rows):
    """One step, token by token.  Returns a dict of new arrays; raises PlanError (then nothing
    is planned).  A deque stands for the ring: new blocks leave its front, returned ones join
    its back after all new blocks are taken."""
    table, ring = np.array(block_table), np.array(free_blocks)
    nb = len(ring)
    head, count = int(free_state[0]), int(free_state[1])
    if not 0 <= count <= nb or not (0 <= head < nb or (nb == 0 and head == 0)):
        raise PlanError("arg")
    lens, blocks = np.array(seq_lens, dtype=np.int64), np.array(seq_blocks, dtype=np.int64)
    width = table.shape[1]
    total = need_all = back_all = 0
    for s in range(len(lens)):
        if lens[s] < 0 or not 0 <= blocks[s] <= width or lens[s] > blocks[s] * block_size:
            raise PlanError("arg")
        if new_lens[s] < 0:
            back_all += blocks[s]
            continue
        want = -(-(lens[s] + int(new_lens[s])) // block_size)
        if want > width:
            raise PlanError("arg")
        total += int(new_lens[s])
        need_all += max(0, want - blocks[s])
    if total > max_rows:
        raise PlanError("arg")
    if need_all > count:
        raise PlanError("blocks")
    if count + back_all > nb:
        raise PlanError("arg")
    slots, q_seq, q_len, starts = [], [], [], []
    taken = 0
    for s in range(len(lens)):
        starts.append(len(slots))
        for _ in range(max(0, int(new_lens[s]))):
            col = lens[s] // block_size
            if col >= blocks[s]:
                table[s, col] = ring[(head + taken) % nb]
                taken += 1
                blocks[s] += 1
            b = int(table[s, col])
            slots.append(b * block_size + int(lens[s]) % block_size if 0 <= b < nb else -1)
            lens[s] += 1
            q_seq.append(s)
            q_len.append(lens[s])
    back = []
    for s in range(len(lens)):
        if new_lens[s] < 0:
            back += [int(table[s, j]) for j in range(blocks[s])]
            lens[s] = blocks[s] = 0
    for i, b in enumerate(back):
        ring[(head + count + i) % nb] = b
    starts.append(len(slots))
    pad = max_rows - len(slots)
    return dict(slots=np.array(slots + [-1] * pad, dtype=np.int64), q_seq=np.array(q_seq + [-1] * pad, dtype=np.int32),
                q_len=np.array(q_len + [0] * pad, dtype=np.int32), row_start=np.array(starts, dtype=np.int32),
                seq_lens=lens.astype(np.int32), seq_blocks=blocks.astype(np.int32), table=table, ring=ring,
                free_state=np.array([(head + taken) % nb if nb else 0, count - taken + len(back)], dtype=np.int32))


def commit_tree(pages, block_table, ctx_lens, path, path_lens):
    """A copy of pages[NB, bs, H, RB] with the accepted rows moved, one after another, and the
    new lengths.  A sequence whose path is not ascending or leaves its table stays as it is."""
    out = np.array(pages)
    nb, bs = out.shape[:2]
    cap = min(block_table.shape[1] * bs, 2 ** 31 - 1)
    lens = np.array(ctx_lens, dtype=np.int32)
    for s in range(len(lens)):
        ctx, n = int(ctx_lens[s]), int(path_lens[s])
        if not 0 <= ctx <= cap or not 0 <= n <= path.shape[1]:
            continue
        p = [int(x) for x in path[s, :n]]
        if any(x < 0 or ctx + x >= cap for x in p) or any(b <= a for a, b in zip(p, p[1:])):
            continue
        lens[s] = ctx + n
        for j, x in enumerate(p):
            a, b = ctx + x, ctx + j
            ba, bb = int(block_table[s, a // bs]), int(block_table[s, b // bs])
            if 0 <= ba < nb and 0 <= bb < nb:
                out[bb, b % bs] = out[ba, a % bs]
    return out, lens


def tree_visible(q_seq, ctx_lens, mask, cap):
    """Boolean rows [T, cap]: the context, and ctx + j for the set bits j of mask[i] (uint32 words)."""
    see = np.zeros((len(q_seq), cap), dtype=bool)
    for i, s in enumerate(q_seq):
        if not 0 <= s < len(ctx_lens):
            continue
        ctx = min(max(int(ctx_lens[s]), 0), cap)
        see[i, :ctx] = True
        for j in range(32 * mask.shape[1]):
            if (int(mask[i, j // 32]) >> (j % 32)) & 1 and ctx + j < cap:
                see[i, ctx + j] = True
    return see


def biased_visible(q_seq, q_len, cap, num_seqs, window=0, prefix_lens=None, doc_starts=None):
    """Boolean rows [T, cap]: t >= doc and (t < prefix or len - window <= t < len)."""
    see = np.zeros((len(q_seq), cap), dtype=bool)
    for i, s in enumerate(q_seq):
        if not 0 <= s < num_seqs:
            continue
        n = min(max(int(q_len[i]), 0), cap)
        for t in range(cap):
            causal = t < n and (not window or t >= n - window)
            prefix = prefix_lens is not None and t < prefix_lens[s]
            see[i, t] = (causal or prefix) and (doc_starts is None or t >= doc_starts[i])
    return see


def attention(q, q_seq, see, k_pages, v_pages, k_bits, v_bits, block_table, signs, k_centroids32, v_centroids32,
              scale=None, softcap=0.0, slopes=None, q_pos=None):
    """softmax over the visible tokens of f(scale <q, k>) - slope |pos - t| times the values, fp64;
    tokens whose block id is outside the pages are left out; a row that sees none is zero.
    Returns (out[T, Hq, D], reach[T, Hq]: the largest |value| coordinate among the visible)."""
    q = np.asarray(q, dtype=np.float64)
    t_rows, hq, d = q.shape
    nb, bs, h, _ = k_pages.shape
    g = hq // h
    rot = o.rotation_matrix(signs)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, reach = np.zeros_like(q), np.zeros((t_rows, hq))
    for s in sorted({int(x) for x in q_seq if 0 <= x < block_table.shape[0]}):
        mine = [i for i in range(t_rows) if q_seq[i] == s]
        toks = np.nonzero(see[mine].any(0))[0]
        if not len(toks):
            continue
        blk = block_table[s, toks // bs].astype(np.int64)
        ok = (blk >= 0) & (blk < nb)
        toks, blk = toks[ok], blk[ok]
        for head in range(h):
            k = o.dequant_rows(k_pages[blk, toks % bs, head], d, k_bits, rot, k_centroids32)
            v = o.dequant_rows(v_pages[blk, toks % bs, head], d, v_bits, rot, v_centroids32)
            for i in mine:
                vis = see[i, toks]
                if not vis.any():
                    continue
                for c in range(head * g, head * g + g):
                    x = scale * (k[vis] @ q[i, c])
                    if softcap:
                        x = softcap * np.tanh(x / softcap)
                    if slopes is not None:
                        x = x - slopes[c] * np.abs(q_pos[i] - toks[vis])
                    p = np.exp(x - x.max())
                    out[i, c] = (p / p.sum()) @ v[vis]
                    reach[i, c] = np.abs(v[vis]).max()
    return out, reach

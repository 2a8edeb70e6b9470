"""The calls of a drafting engine's step together: plan, append (norms, rotation, packed rows), tree
attention, verification, commit -- each against the oracle on what the step before left, eagerly and
as one captured CUDA graph.

Tolerances are those of the single calls: rows as tests/test_gpu_append.py has them, attention (fp16
outputs) within 2^-10 of the output's norm, verification all of it where the oracle is sure by more
than 2^-18.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import append_oracle as ao  # noqa: E402
from oracle import step_oracle as so  # noqa: E402
from oracle import tq_oracle as o  # noqa: E402
from oracle import verify_oracle as vo  # noqa: E402

pytestmark = pytest.mark.gpu

D, H, HQ, BS, KB, VB, VOCAB, WIDTH = 128, 4, 16, 16, 4, 3, 700, 24
F16 = torch.float16


def _tq():
    import quantized_kv_cache_06_gb300 as tq

    return tq


class Engine:
    """Device state of a few sequences; random projections stand for the model around the calls."""

    def __init__(self, tq, seqs, blocks, seed, max_rows):
        self.tq, self.rng, self.seqs, self.max_rows = tq, np.random.default_rng(seed), seqs, max_rows
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.signs = tq.tq_build_rotation(D, 42, "cuda")
        self.kc, self.vc = tq.tq_codebook(D, KB, "cuda")[0], tq.tq_codebook(D, VB, "cuda")[0]
        self.kp = torch.zeros(blocks, BS, H, tq.tq_row_bytes(D, KB), dtype=torch.uint8, device="cuda")
        self.vp = torch.zeros(blocks, BS, H, tq.tq_row_bytes(D, VB), dtype=torch.uint8, device="cuda")
        self.lens, self.blocks = torch.zeros(seqs, **i32), torch.zeros(seqs, **i32)
        self.table = torch.zeros(seqs, WIDTH, **i32)
        self.ring = torch.arange(blocks, **i32)
        self.free = torch.tensor([0, blocks], **i32)
        self.status = torch.zeros(1, **i32)
        self.rope = tq.tq_build_rope(D, WIDTH * BS, device="cuda")
        self.qw, self.kw = torch.exp(0.2 * rand(D)), torch.exp(0.2 * rand(D))
        self.embed = rand(VOCAB, (HQ + 2 * H) * D).to(F16)
        self.head = rand(HQ * D, VOCAB) / 12
        self.temp = torch.rand(seqs, generator=g, device="cuda") + 0.4
        self.temp[1] = 0.0

    def append(self, tokens, p, positions=None):
        """Queries of the rows, their keys and values written."""
        x = self.embed[tokens.long()]
        q, k, v = x.split([HQ * D, H * D, H * D], 1)
        at = dict(positions=p.q_len, position_offset=-1) if positions is None else dict(positions=positions)
        self.qkv = [y.unflatten(1, (-1, D)) for y in (q, k, v)]
        return self.tq.tq_append_kv(*self.qkv, self.kp, self.vp, p.slots, self.signs, self.kc, self.vc, cos_sin=self.rope,
                                    q_weight=self.qw, k_weight=self.kw, status=self.status, **at)

    def args(self):
        return (self.kp, self.vp, self.table, self.signs, self.kc, self.vc)

    def check_rows(self, q, p, positions):
        """The rows of a step against the oracle: queries, keys, values."""
        slots, pos = p.slots.cpu().numpy(), positions
        live = slots >= 0
        table = self.rope.cpu().numpy()
        want, size = ao.norm_rope(self.qkv[0].double().cpu().numpy()[live], pos[live], table, False, self.qw.cpu().numpy())
        off = np.abs(q.double().cpu().numpy()[live] - want)
        assert np.all(off <= 2.0 ** -11 * np.abs(want) * (1 + 2.0 ** -10) + 2.0 ** -25 + 2.0 ** -20 * size)
        keys = ao.norm_rope(self.qkv[1].double().cpu().numpy()[live], pos[live], table, False, self.kw.cpu().numpy())[0]
        for pages, rows, cents, bits in ((self.kp, keys, self.kc, KB), (self.vp, self.qkv[2].double().cpu().numpy()[live], self.vc, VB)):
            got = pages.view(-1, H, pages.shape[3])[torch.from_numpy(slots[live]).cuda()].cpu().numpy().reshape(-1, pages.shape[3])
            idx, norm, margin = ao.encode(rows.reshape(-1, D), self.signs.cpu().numpy().astype(np.float64), cents.cpu().numpy())
            n = o.index_bytes(D, bits)
            diff = np.abs(o.unpack_indices(got[:, :n], D, bits) - idx)
            assert np.all((diff == 0) | ((diff == 1) & (margin <= 2.0 ** -18)))
            nu = np.ascontiguousarray(got[:, n:]).view("<f4").reshape(-1)
            assert np.all(np.abs(nu - norm) <= 2.0 ** -18 * norm)


def trees(rng, rows):
    """Parents, depths and masks of the rows' trees."""
    parents, depth, masks = [], [], []
    for n in rows:
        see = np.zeros((n, 32), dtype=np.uint64)
        d = np.zeros(n, dtype=np.int64)
        for i in range(n):
            up = -1 if i == 0 else int(rng.integers(max(0, i - 3), i))
            parents.append(up)
            if i:
                see[i] = see[up]
                d[i] = d[up] + 1
            see[i, i] = 1
        depth.append(d)
        masks.append((see << np.arange(32, dtype=np.uint64)).sum(1))
    return (np.array(parents, dtype=np.int32), np.concatenate(depth) if depth else np.zeros(0, int),
            np.concatenate(masks).astype(np.uint32))


def test_drafted_steps():
    tq = _tq()
    e = Engine(tq, 5, 60, 1, 40)
    pad = lambda a, fill: np.concatenate([a, np.full(e.max_rows - len(a), fill, a.dtype)])  # noqa: E731
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    # prompts, then plain sampling: one row a sequence
    rows = [9, 17, 1, 3, 6]
    p = tq.tq_plan_step(e.lens, c(np.array(rows, np.int32)), e.blocks, e.table, e.ring, e.free, BS, e.max_rows, check=True)
    tokens = c(pad(e.rng.integers(0, VOCAB, sum(rows)).astype(np.int32), 0))
    q = e.append(tokens, p)
    assert int(e.status.item()) == 0
    e.check_rows(q, p, p.q_len.cpu().numpy() - 1)
    out = tq.tq_paged_prefill_biased(q, p.q_seq, p.q_len, *e.args())
    last = (p.row_start[1:] - 1).long()
    logits = (out[last].float().flatten(1) @ e.head).to(torch.bfloat16)
    one = torch.arange(6, dtype=torch.int32, device="cuda")
    first = tq.tq_verify_tree(logits, one, torch.zeros(5, dtype=torch.int32, device="cuda"), c(e.rng.random(5).astype(np.float32)), 1,
                              temperature=e.temp, check=True)
    e.lens, e.blocks, e.free, tokens = p.seq_lens, p.seq_blocks, p.free_state, first.next_token
    kept = 0
    for turn in range(6):
        rows = [int(n) for n in e.rng.integers(1, 8, 5)]
        ctx = e.lens
        p = tq.tq_plan_step(ctx, c(np.array(rows, np.int32)), e.blocks, e.table, e.ring, e.free, BS, e.max_rows, check=True)
        parents, depth, mask = trees(e.rng, rows)
        start = np.concatenate([[0], np.cumsum(rows)])
        assert np.array_equal(p.row_start.cpu().numpy(), start)
        drafted = e.rng.integers(0, VOCAB, start[-1]).astype(np.int32)
        drafted[start[:-1]] = tokens.cpu().numpy()
        seq = p.q_seq.cpu().numpy()
        pos = pad(ctx.cpu().numpy()[seq[:start[-1]]] + depth, -1).astype(np.int32)
        q_len = p.q_len.cpu().numpy()
        assert np.all(pos[start[-1]:] == -1) and np.all(q_len[start[-1]:] == 0)

        def attend(drafted):
            q = e.append(c(pad(drafted, 0)), p, c(pos))
            assert int(e.status.item()) == 0
            q = torch.where((p.q_seq >= 0)[:, None, None], q, 0)  # padding rows of q are as they were
            return q, tq.tq_paged_tree(q, p.q_seq, ctx, c(pad(mask, 0).view(np.int32)[:, None]), *e.args(), check=True)

        # a drafter that is often right: what the target would draw at the parents, level by level
        us = e.rng.random(e.max_rows).astype(np.float32)
        temp = e.temp.cpu().numpy()
        for level in range(1, depth.max() + 1):
            _, out = attend(drafted)
            logits = (out.float().flatten(1) @ e.head).to(torch.bfloat16)
            lx = logits.double().cpu().numpy()
            for r in np.nonzero(depth == level)[0]:
                up = start[seq[r]] + parents[r]
                if e.rng.random() < 0.7:
                    t = temp[seq[r]]
                    drafted[r] = vo.best(lx[up]) if t == 0 else vo.draw(vo.softmax(lx[up], t), us[up])[0]
        q, out = attend(drafted)
        e.check_rows(q, p, pos)
        see = so.tree_visible(seq, ctx.cpu().numpy(), pad(mask, 0)[:, None], WIDTH * BS)
        want, _ = so.attention(q.float().cpu().numpy(), seq, see, e.kp.cpu().numpy(), e.vp.cpu().numpy(), KB, VB,
                               e.table.cpu().numpy(), e.signs.cpu().numpy().astype(np.float64), e.kc.cpu().numpy(),
                               e.vc.cpu().numpy())
        got = out.float().cpu().numpy()
        assert np.linalg.norm(got - want) <= 2.0 ** -10 * np.linalg.norm(want)
        logits = (out.float().flatten(1) @ e.head).to(torch.bfloat16)
        v = tq.tq_verify_tree(logits, p.row_start, c(pad(drafted, -1)), c(us), 8, parents=c(pad(parents, -1)), temperature=e.temp,
                              check=True)
        path, lens, nxt, sure = vo.verify(logits.double().cpu().numpy(), start, drafted, us, 8, parents, temp)
        ok = sure > 2.0 ** -18
        assert ok.sum() >= 3
        for a, b in ((v.path, path), (v.path_lens, lens), (v.next_token, nxt)):
            assert np.array_equal(a.cpu().numpy()[ok], b[ok])
        kept += int(v.path_lens.sum())
        before = e.kp.cpu().numpy(), e.vp.cpu().numpy()
        e.lens = tq.tq_commit_tree(e.kp, e.vp, e.table, ctx, v.path, v.path_lens, check=True)
        for old, new in zip(before, (e.kp, e.vp)):
            moved, after = so.commit_tree(old, e.table.cpu().numpy(), ctx.cpu().numpy(), v.path.cpu().numpy(), v.path_lens.cpu().numpy())
            assert np.array_equal(new.cpu().numpy(), moved)
        assert np.array_equal(e.lens.cpu().numpy(), after)
        e.blocks, e.free, tokens = p.seq_blocks, p.free_state, v.next_token
    assert kept > 6 * 5 + 10  # more than the roots alone


@pytest.mark.parametrize("drawn", [False, True])
def test_a_step_captured_and_replayed(drawn):
    # two graphs of the whole step with workspaces of their own, replayed in turn and on two streams
    # at once: the bytes of eager calls from the same state
    tq = _tq()
    seqs, nodes = 6, 5
    r = seqs * nodes

    def fresh(seed):
        e = Engine(tq, seqs, 200, seed, r)
        i32 = dict(dtype=torch.int32, device="cuda")
        e.new = torch.full((seqs,), nodes, **i32)
        e.tokens = torch.zeros(r, **i32)
        e.us, e.ua = torch.zeros(r, device="cuda"), torch.zeros(r, device="cuda")
        e.draft = torch.zeros(r, VOCAB, device="cuda") if drawn else None
        e.ctx = torch.zeros(seqs, **i32)
        e.plan = tq.StepPlan(torch.empty(r, dtype=torch.int64, device="cuda"), torch.empty(r, **i32), torch.empty(r, **i32),
                             torch.empty(seqs + 1, **i32), e.lens, e.blocks, e.free)
        e.mask = torch.tensor([[(1 << (i + 1)) - 1] for i in range(nodes)], **i32).repeat(seqs, 1)
        e.ws = torch.empty(tq.tq_verify_tree_workspace(r, VOCAB, seqs), dtype=torch.uint8, device="cuda")
        e.out = tq.Verified(torch.empty(seqs, nodes, **i32), torch.empty(seqs, **i32), torch.empty(seqs, **i32))
        return e

    def work(e):
        e.ctx.copy_(e.lens)
        tq.tq_plan_step(e.lens, e.new, e.blocks, e.table, e.ring, e.free, BS, r, out=e.plan, status=e.status)
        q = e.append(e.tokens, e.plan)
        out = tq.tq_paged_tree(q, e.plan.q_seq, e.ctx, e.mask, *e.args())
        logits = (out.float().flatten(1) @ e.head).to(torch.bfloat16)
        tq.tq_verify_tree(logits, e.plan.row_start, e.tokens, e.us, nodes, temperature=e.temp, draft_probs=e.draft,
                          u_accept=e.ua if drawn else None, out=e.out, workspace=e.ws)
        tq.tq_commit_tree(e.kp, e.vp, e.table, e.ctx, e.out.path, e.out.path_lens, seq_lens=e.lens)

    g = torch.Generator(device="cuda").manual_seed(4)
    inputs = [(torch.randint(0, VOCAB, (r,), generator=g, device="cuda", dtype=torch.int32), torch.rand(r, generator=g, device="cuda"),
               torch.rand(r, generator=g, device="cuda"), torch.softmax(torch.randn(r, VOCAB, generator=g, device="cuda"), 1))
              for _ in range(4)]

    def feed(e, x):
        e.tokens.copy_(x[0]), e.us.copy_(x[1]), e.ua.copy_(x[2])
        if drawn:
            e.draft.copy_(x[3])

    def state(e):
        return [t.clone() for t in (*e.out, e.lens, e.kp, e.vp, e.table)]

    want = {}
    for seed in (21, 22):
        e = fresh(seed)
        want[seed] = []
        for x in inputs:
            feed(e, x)
            work(e)
            want[seed].append(state(e))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(fresh(3))
    torch.cuda.synchronize()
    engines, graphs = [fresh(21), fresh(22)], []
    for e in engines:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work(e)
        graphs.append(graph)
    for i, x in enumerate(inputs):
        for e in engines:
            feed(e, x)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for e, seed in zip(engines, (21, 22)):
            assert all(torch.equal(a, b) for a, b in zip(state(e), want[seed][i]))

"""The serving-step calls together, as an engine uses them: plan a prompt step, write its rows,
prefill, draft a tree, verify it, commit the accepted nodes, go on with single tokens -- each
against the oracle on the pages the library holds -- eagerly and as one captured CUDA graph.

Tolerances are those of the attention tests (fp16 outputs): the norm of the error within 2^-10 of
the output's.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import step_oracle as so  # noqa: E402
from oracle import tq_oracle as o  # noqa: E402

pytestmark = pytest.mark.gpu

D, H, HQ, BS, KB, VB = 128, 4, 16, 16, 4, 2


def _tq():
    import quantized_kv_cache_06_gb300 as tq

    return tq


class Engine:
    """Device state of a few sequences, and the oracle's copy of the tables."""

    def __init__(self, tq, seqs, width, blocks, seed):
        self.tq, self.rng = tq, np.random.default_rng(seed)
        dev = "cuda"
        i32 = dict(dtype=torch.int32, device=dev)
        self.signs = tq.tq_build_rotation(D, 42, dev)
        self.kc, self.vc = tq.tq_codebook(D, KB, dev)[0], tq.tq_codebook(D, VB, dev)[0]
        self.kp = torch.randint(0, 256, (blocks, BS, H, tq.tq_row_bytes(D, KB)), dtype=torch.uint8, device=dev)
        self.vp = torch.randint(0, 256, (blocks, BS, H, tq.tq_row_bytes(D, VB)), dtype=torch.uint8, device=dev)
        self.lens, self.blocks = torch.zeros(seqs, **i32), torch.zeros(seqs, **i32)
        self.table = torch.zeros(seqs, width, **i32)
        self.ring = torch.from_numpy(self.rng.permutation(blocks).astype(np.int32)).to(dev)
        self.free = torch.tensor([0, blocks], **i32)
        self.status = torch.zeros(1, **i32)
        self.mirror = dict(seq_lens=np.zeros(seqs, int), seq_blocks=np.zeros(seqs, int), table=self.table.cpu().numpy(),
                           ring=self.ring.cpu().numpy(), free_state=np.array([0, blocks]))

    def step(self, new, rows):
        """Plans and writes random rows; returns the plan (checked against the oracle)."""
        m = self.mirror
        want = so.plan_step(m["seq_lens"], new, m["seq_blocks"], m["table"], m["ring"], m["free_state"], BS, rows)
        p = self.tq.tq_plan_step(self.lens, torch.tensor(new, dtype=torch.int32, device="cuda"), self.blocks, self.table,
                                 self.ring, self.free, BS, rows, status=self.status, check=True)
        for name in ("slots", "q_seq", "q_len", "row_start", "seq_lens", "seq_blocks", "free_state"):
            assert np.array_equal(getattr(p, name).cpu().numpy(), want[name]), name
        assert np.array_equal(self.table.cpu().numpy(), want["table"])
        self.mirror = want
        before = self.lens
        self.lens, self.blocks, self.free = p.seq_lens, p.seq_blocks, p.free_state
        for pages, cents in ((self.kp, self.kc), (self.vp, self.vc)):
            raw = torch.from_numpy(self.rng.standard_normal((rows, H, D)).astype(np.float16)).cuda()
            self.tq.tq_write_kv(raw, pages, p.slots, self.signs, cents, status=self.status)
        return p, before

    def check(self, q, out, q_seq, see, **kw):
        ok = q_seq >= 0
        want, _ = so.attention(q.float().cpu().numpy(), q_seq, see, self.kp.cpu().numpy(), self.vp.cpu().numpy(), KB, VB,
                               self.table.cpu().numpy(), self.signs.cpu().numpy().astype(np.float64),
                               self.kc.cpu().numpy(), self.vc.cpu().numpy(), **kw)
        got = out.float().cpu().numpy()
        assert np.all(got[~ok] == 0)
        assert np.linalg.norm(got - want) <= 2.0 ** -10 * np.linalg.norm(want)

    def args(self):
        return (self.kp, self.vp, self.table, self.signs, self.kc, self.vc)

    def queries(self, rows):
        return torch.from_numpy(self.rng.standard_normal((rows, HQ, D)).astype(np.float16)).cuda()


def test_steps_of_an_engine():
    tq = _tq()
    e = Engine(tq, 5, 12, 50, 3)
    cap = 12 * BS
    # a prompt step: four sequences, ragged, with padding rows
    p, _ = e.step([37, 1, 100, 16, 0], 160)
    q = e.queries(160)
    q_seq, q_len = p.q_seq.cpu().numpy(), p.q_len.cpu().numpy()
    out = tq.tq_paged_prefill_biased(q, p.q_seq, p.q_len, *e.args(), window=50, status=e.status, check=True)
    e.check(q, out, q_seq, so.biased_visible(q_seq, q_len, cap, 5, window=50))
    for _ in range(3):  # drafted trees, verified and committed
        nodes = [4, 7, 3, 8, 0]
        p, ctx = e.step(nodes, 24)
        see = [np.zeros((n, 32), dtype=np.uint64) for n in nodes]
        for s in see:
            for i in range(len(s)):
                if i:
                    s[i] = s[e.rng.integers(0, i)]
                s[i, i] = 1
        mask = np.concatenate([(s << np.arange(32, dtype=np.uint64)).sum(1) for s in see]).astype(np.uint32)
        mask = np.concatenate([mask, np.zeros(24 - len(mask), np.uint32)])[:, None]
        q = e.queries(24)
        q_seq = p.q_seq.cpu().numpy()
        out = tq.tq_paged_tree(q, p.q_seq, ctx, torch.from_numpy(mask.view(np.int32)).cuda(), *e.args(), softcap=20.0,
                               status=e.status, check=True)
        e.check(q, out, q_seq, so.tree_visible(q_seq, ctx.cpu().numpy(), mask, cap), softcap=20.0)
        path = np.zeros((5, 8), dtype=np.int32)
        count = np.zeros(5, dtype=np.int32)
        for s, n in enumerate(nodes):  # a random root-to-node chain is ascending
            if n:
                chain = np.nonzero(see[s][e.rng.integers(0, n)])[0]
                path[s, :len(chain)], count[s] = chain, len(chain)
        k0, v0 = e.kp.cpu().numpy(), e.vp.cpu().numpy()
        lens = tq.tq_commit_tree(e.kp, e.vp, e.table, ctx, torch.from_numpy(path).cuda(), torch.from_numpy(count).cuda(),
                                 status=e.status, check=True)
        for before, after in ((k0, e.kp), (v0, e.vp)):
            want, want_lens = so.commit_tree(before, e.table.cpu().numpy(), ctx.cpu().numpy(), path, count)
            assert np.array_equal(after.cpu().numpy(), want)
        assert np.array_equal(lens.cpu().numpy(), want_lens)
        e.lens = lens
        e.mirror["seq_lens"] = want_lens
    # a sequence ends, another starts, single tokens with a distance bias; the committed rows are
    # the ones the plain decode sees too
    p, _ = e.step([1, 1, -1, 1, 20], 32)
    q = e.queries(32)
    q_seq, q_len = p.q_seq.cpu().numpy(), p.q_len.cpu().numpy()
    slopes = torch.tensor([2.0 ** (-8 * (i + 1) / HQ) for i in range(HQ)], device="cuda")
    out = tq.tq_paged_prefill_biased(q, p.q_seq, p.q_len, *e.args(), alibi_slopes=slopes, status=e.status, check=True)
    e.check(q, out, q_seq, so.biased_visible(q_seq, q_len, cap, 5), slopes=slopes.cpu().numpy().astype(np.float64),
            q_pos=q_len - 1)
    n = 23
    plain = tq.tq_paged_prefill(q[:n], p.q_seq[:n], p.q_len[:n], *e.args(), status=e.status, check=True)
    out = tq.tq_paged_prefill_biased(q[:n], p.q_seq[:n], p.q_len[:n], *e.args())
    assert torch.all((plain.float() - out.float()).abs() <= 2e-3 + 2e-3 * plain.float().abs())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_a_step_captured_and_replayed(dtype):
    # plan (state in place), two writes, tree attention and commit in one graph; replays on new
    # inputs give the bytes of eager calls from the same state
    tq = _tq()
    seqs, nodes, width, blocks = 6, 5, 40, 300
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(5)

    def fresh():
        e = Engine(tq, seqs, width, blocks, 11)
        i32 = dict(dtype=torch.int32, device=dev)
        e.new = torch.full((seqs,), nodes, **i32)
        e.raw = torch.zeros(2, seqs * nodes, H, D, dtype=torch.float16, device=dev)
        e.q = torch.zeros(seqs * nodes, HQ, D, dtype=dtype, device=dev)
        chain = torch.tensor([[(1 << (i + 1)) - 1] for i in range(nodes)], **i32)
        e.mask = chain.repeat(seqs, 1)
        e.path = torch.tensor([[0, 1, 3]] * seqs, **i32)
        e.count = torch.tensor([3, 2, 1, 0, 3, 2], **i32)
        r = seqs * nodes
        e.out = torch.empty(r, HQ, D, dtype=dtype, device=dev)
        e.ctx = torch.zeros(seqs, **i32)
        e.plan = tq.StepPlan(torch.empty(r, dtype=torch.int64, device=dev), torch.empty(r, **i32), torch.empty(r, **i32),
                             torch.empty(seqs + 1, **i32), e.lens, e.blocks, e.free)
        e.ws = torch.empty(tq.tq_paged_tree_workspace(r, HQ, H, D), dtype=torch.uint8, device=dev)
        e.kp.zero_(), e.vp.zero_()
        return e

    def work(e):
        e.ctx.copy_(e.lens)
        tq.tq_plan_step(e.lens, e.new, e.blocks, e.table, e.ring, e.free, BS, seqs * nodes, out=e.plan, status=e.status)
        tq.tq_write_kv(e.raw[0], e.kp, e.plan.slots, e.signs, e.kc, status=e.status, check=False)
        tq.tq_write_kv(e.raw[1], e.vp, e.plan.slots, e.signs, e.vc, status=e.status, check=False)
        tq.tq_paged_tree(e.q, e.plan.q_seq, e.ctx, e.mask, e.kp, e.vp, e.table, e.signs, e.kc, e.vc, out=e.out,
                         workspace=e.ws, status=e.status)
        tq.tq_commit_tree(e.kp, e.vp, e.table, e.ctx, e.path, e.count, seq_lens=e.lens, status=e.status)

    inputs = [(torch.randn(2, seqs * nodes, H, D, generator=g, device=dev).half(),
               torch.randn(seqs * nodes, HQ, D, generator=g, device=dev).to(dtype)) for _ in range(4)]
    eager, graphed = fresh(), fresh()
    want = []
    for raw, q in inputs:
        eager.raw.copy_(raw), eager.q.copy_(q)
        work(eager)
        want.append(eager.out.clone())
    warm = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(graphed)
    for (raw, q), w in zip(inputs, want):
        graphed.raw.copy_(raw), graphed.q.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(graphed.out, w)
    assert torch.equal(graphed.lens, eager.lens) and torch.equal(graphed.kp, eager.kp)
    assert torch.equal(graphed.table, eager.table) and int(graphed.status.item()) == 0


def test_a_wait_that_runs_out_is_reported():
    # every bounded wait of the tensor-core attention gives up at once; the next call is right
    tq = _tq()
    e = Engine(tq, 2, 30, 60, 9)
    p, _ = e.step([400, 33], 433)
    rows = slice(393, 433)
    q = e.queries(40)
    args = (q, p.q_seq[rows].contiguous(), p.q_len[rows].contiguous(), *e.args())
    want = tq.tq_paged_prefill_biased(*args, status=e.status, check=True)
    old = tq.tq_set_wait_limit(0)
    try:
        with pytest.raises(tq.TQError) as err:
            tq.tq_paged_prefill_biased(*args, status=e.status, check=True)
        assert err.value.status == tq.TQ_ERR_TIMEOUT
    finally:
        tq.tq_set_wait_limit(-1)
    assert old > 0
    assert torch.equal(want, tq.tq_paged_prefill_biased(*args, status=e.status, check=True))
    assert math.isfinite(float(want.float().abs().max()))

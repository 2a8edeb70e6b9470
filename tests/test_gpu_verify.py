"""tq_verify_tree against the definition in 64 bits.

What a decision may be off by.  A weight 2^y has the rounding of y, half an ulp: below 2^-21 for |y| <
32 (weights beyond that carry less than 2^-32 of a row each), times ln 2, and ex2's own 2^-22; a piece's
sum adds up to 40 roundings of 2^-24 of what is summed so far.  So a running sum over the whole is off by
less than 2^-18 of the whole, and so is p.  r = max(a p - b q, 0) is off by 2^-18 a p.  The oracle says in
these units how near the nearest other outcome was (`sure`); where that is more than 2^-18 the outcome
has to be the oracle's, all of it, and as many sequences as the inputs let expect have to be such.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import verify_oracle as vo  # noqa: E402

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NEAR = 2.0 ** -18


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


class Drafts:
    """Sequences of drafted nodes: logits, tokens that are often right, random numbers."""

    def __init__(self, rows, vocab, dtype, kind="chain", draft=None, seed=0, spread=2.0, temperature=True, pad=0, kids=3):
        rng = np.random.default_rng(seed)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        t, self.vocab = int(self.start[-1]), vocab
        x = rng.standard_normal((t, vocab)) * spread
        self.store = torch.zeros(t, vocab + pad, dtype=dtype, device="cuda")
        self.store[:, :vocab] = torch.from_numpy(x.astype(np.float32)).cuda()
        self.logits = self.store[:, :vocab]
        lx = self.logits.double().cpu().numpy()
        self.temp = rng.uniform(0.5, 1.5, len(rows)).astype(np.float32) if temperature else None
        self.parents = None
        if kind == "tree":
            self.parents = np.concatenate([[-1 if i == 0 else rng.integers(max(0, i - kids), i) for i in range(n)]
                                           for n in rows] or [[]]).astype(np.int32)
        self.ua, self.us = rng.random(t).astype(np.float32), rng.random(t).astype(np.float32)
        self.tokens = np.zeros(t, dtype=np.int32)
        self.draft = None
        if draft is not None:
            noisy = lx + 0.5 * rng.standard_normal(lx.shape)
            q = np.exp(noisy - noisy.max(1, keepdims=True))
            self.draft = torch.from_numpy((q / q.sum(1, keepdims=True)).astype(np.float32)).cuda().to(draft)
        for s, n in enumerate(rows):
            r0 = self.start[s]
            for i in range(1, n):
                up = i - 1 if self.parents is None else int(self.parents[r0 + i])
                if draft is not None:
                    q = self.draft[r0 + up].double().cpu().numpy()
                    self.tokens[r0 + i] = rng.choice(vocab, p=q / q.sum())
                else:
                    temp = 1.0 if self.temp is None else self.temp[s]
                    y = vo.draw(vo.softmax(lx[r0 + up], temp), self.us[r0 + up])[0] if rng.random() < 0.6 else rng.integers(vocab)
                    self.tokens[r0 + i] = y

    def call(self, tq, max_path, **kw):
        c = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        args = dict(parents=c(self.parents), temperature=c(self.temp), draft_probs=self.draft,
                    u_accept=c(self.ua) if self.draft is not None else None)
        args.update(kw)
        return tq.tq_verify_tree(self.logits, c(self.start), c(self.tokens), c(self.us), max_path, **args)

    def sure_at_least(self):
        """Sequences that are sure at least: a row's number lies within 2^-18 of a token's border with
        probability sum min(p, 2^-17) at most (five times that where refusals scale the rest up); the
        mean over the sequences' rows, less four deviations and one."""
        lx, some = self.logits.double().cpu().numpy(), []
        for s in range(len(self.start) - 1):
            temp = 1.0 if self.temp is None else float(self.temp[s])
            p = 0.0
            for r in range(max(0, self.start[s]), self.start[s + 1]):
                w = vo.softmax(lx[r], temp) if 2.0 ** -100 <= temp <= 2.0 ** 100 else None
                p += 0.0 if w is None else np.minimum(w, 2 * NEAR).sum() * (1 if self.draft is None else 5)
            some.append(min(1.0, p))
        some = np.array(some)
        return (1 - some).sum() - 4 * np.sqrt((some * (1 - some)).sum()) - 1

    def want(self, max_path):
        d = None if self.draft is None else self.draft.double().cpu().numpy()
        return vo.verify(self.logits.double().cpu().numpy(), self.start, self.tokens, self.us, max_path, self.parents,
                         self.temp, d, self.ua)


def same(d, got, want):
    path, lens, nxt, sure = want
    ok = sure > NEAR
    assert ok.sum() >= d.sure_at_least()
    for g, w in ((got.path, path), (got.path_lens, lens), (got.next_token, nxt)):
        assert np.array_equal(g.cpu().numpy()[ok], w[ok])


VOCABS = [1, 7, 1000, 1017, 1024, 1025, 5003, 33000]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_fixed_drafts(tq, dtype, vocab, kind):
    d = Drafts([5, 1, 0, 9, 40, 2, 3], vocab, dtype, kind, seed=vocab)
    same(d, d.call(tq, 40, check=True), d.want(40))
    same(d, d.call(tq, 3), d.want(3))


@pytest.mark.parametrize("dtype,draft", [(F32, F32), (F16, F32), (BF16, F32), (BF16, BF16), (F32, F16), (F16, BF16)])
@pytest.mark.parametrize("vocab", [1, 7, 1017, 1025, 5003, 33000])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_drawn_drafts(tq, dtype, draft, vocab, kind):
    d = Drafts([5, 1, 0, 9, 12, 2, 3, 7], vocab, dtype, kind, draft, seed=vocab + 1)
    same(d, d.call(tq, 12, check=True), d.want(12))
    same(d, d.call(tq, 2), d.want(2))


@pytest.mark.parametrize("draft", [None, F32])
def test_large_batches_and_vocabularies(tq, draft):
    d = Drafts([4] * 12, 140001, BF16, "tree", draft, seed=3, spread=3.0)
    same(d, d.call(tq, 6, check=True), d.want(6))
    d = Drafts([2] * 300, 2500, F16, "chain", draft, seed=4)
    same(d, d.call(tq, 2, check=True), d.want(2))


@pytest.mark.parametrize("pad", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_rows_at_any_address(tq, dtype, pad):
    d = Drafts([3] * 6, 2049, dtype, "chain", F32, pad=pad, seed=9)
    assert d.logits.stride(0) == 2049 + pad
    same(d, d.call(tq, 3, check=True), d.want(3))
    # neighbours of the rows are never part of them
    d.store[:, 2049:] = 100.0
    same(d, d.call(tq, 3), d.want(3))


@pytest.mark.parametrize("draft", [None, F32])
def test_masked_logits(tq, draft):
    d = Drafts([4] * 40, 3000, F32, "chain", draft, seed=5)
    lowest = torch.finfo(F32).min
    hide = torch.rand(d.logits.shape, device="cuda")
    d.logits[hide < 0.3] = -float("inf")
    d.logits[(hide > 0.3) & (hide < 0.5)] = float("nan")
    d.logits[(hide > 0.5) & (hide < 0.6)] = lowest
    d.logits[0::4, 1024:] = -float("inf")  # all tokens in the first piece
    d.logits[1::4, :2900] = lowest
    got = d.call(tq, 4, check=True)
    same(d, got, d.want(4))
    after = got.next_token.cpu().numpy()
    rows = d.start[:-1] + got.path_lens.cpu().numpy() - 1
    last = got.path.cpu().numpy()[np.arange(40), got.path_lens.cpu().numpy() - 1]
    rows = d.start[:-1] + last
    assert torch.all(d.logits[torch.from_numpy(rows).cuda().long(), torch.from_numpy(after).cuda().long()] > lowest)


def test_rows_of_the_lowest_value_alone(tq):
    # a row whose every logit is the type's lowest is uniform
    for dtype in (F32, F16, BF16):
        x = torch.full((4, 2000), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        u = torch.tensor([0.0, 0.25, 0.75, 0.99999994], device="cuda")
        r = tq.tq_verify_tree(x, torch.arange(5, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"),
                              u, 1, check=True)
        assert r.next_token.tolist() == [0, 500, 1500, 1999]


@pytest.mark.parametrize("draft", [None, F32])
@pytest.mark.parametrize("worst", ["-inf", "nan", "inf"])
def test_rows_without_a_distribution(tq, draft, worst):
    d = Drafts([3] * 6, 1500, BF16, "chain", draft, seed=8)
    if worst == "inf":
        d.logits[4, 77] = float("inf")
    else:
        d.logits[4] = float(worst)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = d.call(tq, 3, status=status)
    assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
    want = d.want(3)
    same(d, got, want)
    assert want[2][1] == -1 or want[1][1] == 1  # the walk of sequence 1 ends at its row 1, or before it


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("draft", [None, F32])
def test_greedy(tq, dtype, draft):
    d = Drafts([6] * 20, 4000, dtype, "tree", draft, seed=11)
    d.logits.copy_(d.logits.float().mul(2).round().clamp(max=5).to(dtype))  # many ties
    d.temp = np.where(np.arange(20) % 3 == 0, d.temp, 0.0).astype(np.float32)
    best = np.argmax(d.logits.double().cpu().numpy(), axis=1)
    for s in range(20):
        r0 = d.start[s]
        for i in range(1, 6):
            if (s + i) % 3:
                d.tokens[r0 + i] = best[r0 + d.parents[r0 + i]]
    want = d.want(6)
    got = d.call(tq, 6, check=True)
    greedy = d.temp == 0
    for g, w in ((got.path, want[0]), (got.path_lens, want[1]), (got.next_token, want[2])):
        assert np.array_equal(g.cpu().numpy()[greedy], w[greedy])
    same(d, got, want)
    assert want[1][greedy].max() > 2


def test_extreme_temperatures(tq):
    d = Drafts([1] * 8, 2000, F32, seed=12)
    d.temp = np.array([2.0 ** -100, 1e-20, 1e-4, 0.05, 50.0, 1e10, 2.0 ** 100, 0.0], dtype=np.float32)
    same(d, d.call(tq, 1, check=True), d.want(1))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-1.0, float("nan"), float("inf"), 2.0 ** 101, 1e-38):
        d.temp[5] = bad
        got = d.call(tq, 1, status=status)
        assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
        same(d, got, d.want(1))  # the oracle takes it as 0 too


def test_numbers_at_the_ends(tq):
    p = torch.tensor([[-float("inf"), 0.0, 0.0, -float("inf"), 0.0, -float("inf")]], device="cuda").repeat(6, 1)
    u = torch.tensor([0.0, 0.5, 0.99999994, 1.0, float("nan"), -3.0], device="cuda")
    r = tq.tq_verify_tree(p, torch.arange(7, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda"), u, 1)
    assert r.next_token.tolist() == [1, 2, 4, 4, 1, 1]


def test_a_drafter_equal_to_the_target(tq):
    # every drafted token kept for u below 1 by more than the rounding of p
    d = Drafts([6] * 10, 6000, F32, "chain", F32, seed=13, temperature=False)
    d.draft = torch.softmax(d.logits.double(), 1).float()
    d.ua = d.ua * (1 - 2.0 ** -12)
    got = d.call(tq, 6, check=True)
    assert torch.all(got.path_lens == 6)
    # refused all the same (u 1): something is drawn, a token of the vocabulary
    d.ua = np.full_like(d.ua, 1.0)
    got = d.call(tq, 6, check=True)
    assert torch.all((got.next_token >= 0) & (got.next_token < 6000))


def test_a_drafter_above_the_target_everywhere(tq):
    # max(p - q, 0) is empty: the distribution stays, and the next child is tried against it
    d = Drafts([4] * 10, 500, F32, "tree", F32, seed=14, kids=4)
    d.draft = torch.full_like(d.draft, 2.0)
    same(d, d.call(tq, 4, check=True), d.want(4))
    d.draft = torch.where(d.draft > 0, torch.tensor(float("nan"), device="cuda"), d.draft)
    d.draft[:, ::2] = -1.0
    same(d, d.call(tq, 4, check=True), d.want(4))


def test_several_children_refused(tq):
    # eight children of the root, drawn from a drafter far from the target
    rows = [9] * 30
    d = Drafts(rows, 300, F32, "tree", F32, seed=15, spread=1.0)
    d.parents = np.tile(np.array([-1] + [0] * 8, dtype=np.int32), 30)
    rng = np.random.default_rng(2)
    q = rng.dirichlet(np.full(300, 0.3), 270)
    d.draft = torch.from_numpy(q.astype(np.float32)).cuda()
    for s in range(30):
        r = d.start[s]
        d.tokens[r + 1:r + 9] = rng.choice(300, 8, p=q[r] / q[r].sum())
    want = d.want(9)
    same(d, d.call(tq, 9, check=True), want)
    assert (want[1] == 1).sum() >= 1 and (want[1] == 2).sum() >= 3


@pytest.mark.parametrize("draft", [None, F32])
def test_tokens_and_parents_out_of_range(tq, draft):
    d = Drafts([6] * 8, 900, F16, "tree", draft, seed=16)
    d.tokens[1::6] = [-1, 900, 2 ** 31 - 1, -2 ** 31, 901, -5, 900, 1000]
    same(d, d.call(tq, 6, check=True), d.want(6))
    d.parents[2::6] = [2, 5, -1, 100, -2 ** 31, 2 ** 31 - 1, 3, 2]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = d.call(tq, 6, status=status)
    assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
    same(d, got, d.want(6))


def test_rows_behind_the_last_and_bad_row_starts(tq):
    d = Drafts([4, 0, 3], 700, F32, seed=17)
    want = d.want(4)
    pad = torch.full((5, 700), float("nan"), device="cuda")
    d.logits = torch.cat([d.logits, pad])
    d.tokens, d.us = np.concatenate([d.tokens, np.full(5, -7, np.int32)]), np.concatenate([d.us, np.full(5, np.nan, np.float32)])
    same(d, d.call(tq, 4, check=True), want)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([0, 4, 4, 13], [-1, 4, 4, 7], [0, 4, 2, 7], [0, 2 ** 31 - 1, 4, 7]):
        start = d.start
        d.start = np.array(bad, dtype=np.int32)
        got = d.call(tq, 4, status=status)
        assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
        for s in range(3):
            if not (0 <= bad[s] <= bad[s + 1] <= 12):
                assert got.path_lens[s] == 0 and got.next_token[s] == -1 and torch.all(got.path[s] == -1)
        d.start = start
    none = tq.tq_verify_tree(d.logits, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.from_numpy(d.tokens).cuda(),
                             torch.from_numpy(d.us).cuda(), 2)
    assert none.path.shape == (0, 2)
    empty = tq.tq_verify_tree(d.logits[:0], torch.zeros(3, dtype=torch.int32, device="cuda"),
                              torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda"), 2, check=True)
    assert empty.path_lens.tolist() == [0, 0] and empty.next_token.tolist() == [-1, -1] and torch.all(empty.path == -1)


@pytest.mark.parametrize("draft", [None, BF16])
def test_same_bits_on_another_stream_and_in_a_graph(tq, draft):
    d = Drafts([5] * 16, 40000, BF16, "tree", draft, seed=18)
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    start, tokens, us, ua, up, temp = c(d.start), c(d.tokens), c(d.us), c(d.ua), c(d.parents), c(d.temp)
    out = tq.Verified(torch.empty(16, 5, dtype=torch.int32, device="cuda"), torch.empty(16, dtype=torch.int32, device="cuda"),
                      torch.empty(16, dtype=torch.int32, device="cuda"))
    ws = torch.empty(tq.tq_verify_tree_workspace(80, 40000, 16), dtype=torch.uint8, device="cuda")

    def work():
        tq.tq_verify_tree(d.logits, start, tokens, us, 5, parents=up, temperature=temp, draft_probs=d.draft,
                          u_accept=ua if draft else None, out=out, workspace=ws)

    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    ws.fill_(255)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    base = d.logits.clone()
    for turn in range(3):
        d.logits.copy_(base.roll(turn, 1))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, got))


def test_refusals_of_the_binding(tq):
    x = torch.zeros(4, 8, device="cuda")
    i, f, start = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda"), \
        torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=x.long()), dict(logits=x.t()), dict(row_start=start.long()), dict(tokens=i[:3]), dict(u_sample=f.double()),
                dict(max_path=0), dict(draft_probs=x), dict(u_accept=f), dict(draft_probs=x[:, :7], u_accept=f),
                dict(temperature=f), dict(parents=i.float()), dict(tokens=i.cpu()), dict(status=f)):
        args = dict(logits=x, row_start=start, tokens=i, u_sample=f, max_path=3)
        args.update(bad)
        with pytest.raises(ValueError):
            tq.tq_verify_tree(**args)


def test_long_sequences(tq):
    # more nodes than are kept in shared memory, in chains and trees, with and without draft probabilities
    for kind, draft in (("chain", None), ("tree", None), ("chain", F32), ("tree", BF16)):
        d = Drafts([300, 700, 3], 400, F32, kind, draft, seed=30, kids=40)
        if draft is not None and kind == "chain":  # long walks
            d.draft = torch.softmax(d.logits.double() / torch.tensor(np.repeat(d.temp, [300, 700, 3]))[:, None].cuda(), 1).float()
            d.ua = d.ua * np.float32(0.999)
        same(d, d.call(tq, 700, check=True), d.want(700))


def test_more_pieces_than_are_held(tq):
    # a vocabulary of more pieces than shared memory has room for
    d = Drafts([2, 3], 300001, BF16, "chain", F32, seed=31, spread=3.0)
    same(d, d.call(tq, 3, check=True), d.want(3))
    d.draft = None
    same(d, d.call(tq, 3, check=True), d.want(3))


def test_rows_beyond_32_bit_offsets(tq):
    d = Drafts([2, 1], 1200, BF16, "chain", F32, seed=32)
    want = d.call(tq, 2, check=True)
    far = torch.empty(3, (1 << 31) + 64, dtype=BF16, device="cuda")[:, 8:1208]
    far.copy_(d.logits)
    d.logits = far
    got = d.call(tq, 2, check=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

"""tq_verify_tree's tokens against 64 bits, at the vocabularies of language models: a drawn token is the
first whose running sum passes u times the whole, and a drafted one is kept when u q(x) < r(x), however
near the number is.

What may be off.  A weight 2^y is off by at most 2^-45 (1 + |y|) of itself and its rounding to 2^-55; the
mean of |y| over a row is below log2 of the vocabulary, 18 here.  So a border is off by less than 19 2^-45
and the vocabulary's 2^18 2^-55 2^-10 (16 standard deviations of independent roundings), of the whole:
below 2^-40.  Numbers nearer than that to a border are left out; by the width of the window there is
hardly one among 10^5, and no more than a few are let pass as such.  A residual distribution of mass Z has
the same bound over Z.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
I32 = torch.int32
TIE = 2.0 ** -40
DEV = "cuda"


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


def language(n, vocab, dtype, seed):
    """Logits of n rows: a broad bulk that holds a third of the mass or more, a few likely tokens, some
    that are never allowed; and temperatures."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(n, vocab, generator=gen, device=DEV).mul_(1.8)
    likely = torch.randint(0, vocab, (n, 8), generator=gen, device=DEV)
    x.scatter_(1, likely, torch.randn(n, 8, generator=gen, device=DEV).mul_(1.5).add_(8.0))
    x[:, vocab - vocab // 50:] = -float("inf")
    return x.to(dtype), torch.rand(n, generator=gen, device=DEV) * 0.6 + 0.6, gen


def weights(logits, temp):
    """exp((x - max x) / temperature) in 64 bits."""
    x = logits.double()
    return torch.exp_((x - x.amax(1, keepdim=True)) / temp.double()[:, None])


def drawn(cum, u):
    """First tokens whose running sums pass u times the whole, and the distance to the nearer border of
    each, relative to the whole."""
    goal = u.double() * cum[:, -1]
    i = torch.searchsorted(cum, goal[:, None], right=True).clamp_(max=cum.shape[1] - 1)
    ends = torch.cat([cum.gather(1, (i - 1).clamp(min=0)) * (i > 0), cum.gather(1, i)], 1)
    return i[:, 0].to(I32), ((ends - goal[:, None]).abs() / cum[:, -1:]).amin(1)


def at_borders(cum, gen, turn):
    """Numbers of 32 bits next to borders: of tokens of the bulk, at ends of pieces of 1024, behind the
    likeliest token; the nearest number and the ones beside it."""
    n, v = cum.shape
    w = torch.diff(cum, prepend=torch.zeros(n, 1, dtype=cum.dtype, device=DEV), dim=1)
    at = torch.randint(0, v, (n,), generator=gen, device=DEV)
    at = torch.where(torch.arange(n, device=DEV) % 3 == 1, at // 1024 * 1024 + 1023, at).clamp(max=v - 1)
    at = torch.where(torch.arange(n, device=DEV) % 3 == 2, w.argmax(1) - turn % 2, at).clamp(min=0)
    u = (cum.gather(1, at[:, None])[:, 0] / cum[:, -1]).float()
    u = torch.nextafter(u, torch.full_like(u, 2.0 * (turn % 3 == 1))) if turn % 3 else u
    return u.clamp(0, 1 - 2.0 ** -24)


def equal(got, want, near, most=0):
    """`most`: numbers that may lie as near as TIE.  (Numbers that were rounded to 32 bits from borders do so
    with probability 2^-15 / u, u above 2^-15: a few in a thousand where the borders are spread over the
    row.)"""
    wrong = (got != want) & (near > TIE)
    assert not wrong.any(), f"{int(wrong.sum())} of {wrong.numel()}, up to {float(near[wrong].max()):.2e} from a border"
    assert int((near <= TIE).sum()) <= most


def start_of(seqs, rows):
    return torch.arange(seqs + 1, dtype=I32, device=DEV) * rows


@pytest.mark.parametrize("dtype,vocab,seqs,turns", [(BF16, 131072, 1024, 100), (BF16, 140001, 600, 60), (F32, 131072, 512, 100),
                                                    (F16, 140001, 30, 100), (F32, 140001, 17, 60), (BF16, 32768, 300, 60),
                                                    (BF16, 300001, 40, 20)])
def test_drawn_tokens(tq, dtype, vocab, seqs, turns):
    logits, temp, gen = language(seqs, vocab, dtype, vocab + seqs)
    cum = weights(logits, temp).cumsum_(1)
    assert float(torch.quantile(cum[:, -1], 0.5)) > 3  # no token holds a row
    start, tokens = start_of(seqs, 1), torch.zeros(seqs, dtype=I32, device=DEV)
    got, want, near = [], [], []
    for turn in range(turns):
        u = torch.rand(seqs, generator=gen, device=DEV)
        got.append(tq.tq_verify_tree(logits, start, tokens, u, 1, temperature=temp).next_token)
        i, d = drawn(cum, u)
        want.append(i), near.append(d)
    equal(torch.cat(got), torch.cat(want), torch.cat(near), most=2)


@pytest.mark.parametrize("dtype,vocab,seqs", [(BF16, 131072, 400), (F16, 131072, 20), (F32, 140001, 300), (BF16, 140001, 33),
                                              (F32, 1000, 2000), (BF16, 1025, 20)])
def test_numbers_next_to_borders(tq, dtype, vocab, seqs):
    logits, temp, gen = language(seqs, vocab, dtype, vocab)
    cum = weights(logits, temp).cumsum_(1)
    start, tokens = start_of(seqs, 1), torch.zeros(seqs, dtype=I32, device=DEV)
    got, want, near = [], [], []
    for turn in range(12):
        u = at_borders(cum, gen, turn)
        got.append(tq.tq_verify_tree(logits, start, tokens, u, 1, temperature=temp, check=True).next_token)
        i, d = drawn(cum, u)
        want.append(i), near.append(d)
    near = torch.cat(near)
    assert (near < 2.0 ** -24).float().mean() > 0.5  # they are near
    equal(torch.cat(got), torch.cat(want), near, most=near.numel() // 100)


@pytest.mark.parametrize("seqs", [5, 200])
def test_walks_over_numbers_next_to_borders(tq, seqs):
    # chains whose drafted tokens are the ones that numbers next to borders draw: every node is walked to
    nodes, vocab = 6, 50001
    logits, temp, gen = language(seqs * nodes, vocab, BF16, seqs)
    temp = temp[::nodes].contiguous()
    cum = weights(logits, temp.repeat_interleave(nodes)).cumsum_(1)
    u = at_borders(cum, gen, 0)
    want, near = drawn(cum, u)
    u = torch.where(near > TIE, u, 0.5)
    want, near = drawn(cum, u)
    assert (near > TIE).all()
    tokens = torch.zeros(seqs * nodes, dtype=I32, device=DEV)
    tokens[1:] = want[:-1]
    start = start_of(seqs, nodes)
    seen = tq.tq_verify_tree(logits, start, tokens, u, nodes, temperature=temp, check=True)
    assert torch.all(seen.path_lens == nodes) and torch.equal(seen.next_token, want[nodes - 1::nodes])
    assert torch.all(seen.path == torch.arange(nodes, dtype=I32, device=DEV))
    # and left at the first that draws another; a path of two
    tokens[3::nodes] = (tokens[3::nodes] + 1) % vocab
    seen = tq.tq_verify_tree(logits, start, tokens, u, nodes, temperature=temp, check=True)
    assert torch.all(seen.path_lens == 3) and torch.equal(seen.next_token, want[2::nodes])
    seen = tq.tq_verify_tree(logits, start, tokens, u, 2, temperature=temp, check=True)
    assert torch.all(seen.path_lens == 2) and torch.equal(seen.next_token, want[1::nodes])


def refused(seqs, kids, vocab, dtype, draft, seed):
    """Roots with `kids` children of one token that the drafter overrates most: all are refused at u
    near 1.  Rows of logits and draft, tokens, parents, and the weights that are left."""
    logits, temp, gen = language(seqs * (kids + 1), vocab, dtype, seed)
    temp = temp[::kids + 1].contiguous()
    near = logits[::kids + 1].float() + 0.7 * torch.randn(seqs, vocab, generator=gen, device=DEV)
    q = torch.zeros(seqs * (kids + 1), vocab, dtype=draft, device=DEV)
    q[::kids + 1] = torch.softmax(near / temp[:, None], 1).to(draft)
    q64 = q[::kids + 1].double()
    w = weights(logits[::kids + 1], temp)
    r = w / w.sum(1, keepdim=True)
    token = (q64 - r).argmax(1)
    z = torch.ones(seqs, dtype=torch.float64, device=DEV)
    for _ in range(kids):
        r = (r - q64).clamp_(min=0)
        z *= r.sum(1)
        r /= r.sum(1, keepdim=True)
    tokens = token.to(I32).repeat_interleave(kids + 1)
    parents = torch.zeros(seqs * (kids + 1), dtype=I32, device=DEV)
    ua = torch.full((seqs * (kids + 1),), 1 - 2.0 ** -24, device=DEV)
    return logits, temp, q, tokens, parents, ua, r.cumsum_(1), z, gen


@pytest.mark.parametrize("dtype,draft,vocab,seqs,kids,turns", [
    (BF16, F32, 131072, 256, 1, 220), (F32, F32, 131072, 96, 1, 60), (BF16, BF16, 140001, 30, 2, 60), (F16, F32, 32768, 200, 3, 40),
    (F32, BF16, 1000, 1500, 2, 20), (BF16, F16, 140001, 3, 1, 60)])
def test_tokens_drawn_from_what_refusals_leave(tq, dtype, draft, vocab, seqs, kids, turns):
    logits, temp, q, tokens, parents, ua, cum, z, gen = refused(seqs, kids, vocab, dtype, draft, seed=vocab + kids)
    start, rows = start_of(seqs, kids + 1), seqs * (kids + 1)
    assert float(z.min()) > 2.0 ** -16
    got, want, near = [], [], []
    for turn in range(turns):
        us = torch.rand(rows, generator=gen, device=DEV)
        if turn % 4 == 3:
            us[::kids + 1] = at_borders(cum, gen, turn // 4)
        seen = tq.tq_verify_tree(logits, start, tokens, us, 4, parents=parents, temperature=temp, draft_probs=q, u_accept=ua)
        assert torch.all(seen.path_lens == 1)
        got.append(seen.next_token)
        i, d = drawn(cum, us[::kids + 1])
        want.append(i), near.append(d * z)
    near = torch.cat(near)
    equal(torch.cat(got), torch.cat(want), near, most=near.numel() // 100)


@pytest.mark.parametrize("dtype,vocab", [(BF16, 131072), (F32, 50001)])
@pytest.mark.parametrize("seqs", [20, 160])
def test_children_kept_or_refused_next_to_the_border(tq, dtype, vocab, seqs):
    # u next to r(x) / q(x), for a first child and for one behind a refused one
    logits, temp, q, tokens, parents, ua, cum, z, gen = refused(seqs, 2, vocab, dtype, F32, seed=vocab + 7)
    w = weights(logits[::3], temp)
    p = w / w.sum(1, keepdim=True)
    q64 = q[::3].double()
    rest = (p - q64).clamp(min=0)
    rest /= rest.sum(1, keepdim=True)
    us = torch.rand(seqs * 3, generator=gen, device=DEV)
    start = start_of(seqs, 3)
    for second in (False, True):
        r = rest if second else p
        ratio = r / q64
        ok = (ratio > 0.05) & (ratio < 0.95)
        x = torch.where(ok, torch.rand(ok.shape, generator=gen, device=DEV), -1.0).argmax(1)
        assert ok.gather(1, x[:, None]).all()
        tok = tokens.clone()
        tok[2 if second else 1::3] = x.to(I32)
        r_x, q_x = (t.gather(1, x[:, None])[:, 0] for t in (r, q64))
        u = (r_x / q_x).float()
        for turn in range(3):
            v = u if turn == 0 else torch.nextafter(u, torch.full_like(u, float(turn - 1)))
            a = ua.clone()
            a[2 if second else 1::3] = v
            kept = v.double() * q_x < r_x
            far = (v.double() * q_x - r_x).abs() / r_x > TIE / z  # (r of a first child: p, and more room than that)
            assert far.float().mean() > 0.9
            seen = tq.tq_verify_tree(logits, start, tok, us, 4, parents=parents, temperature=temp, draft_probs=q, u_accept=a)
            assert torch.equal((seen.path_lens == 2)[far], kept[far])
            node = torch.where(kept, 2 if second else 1, -1)
            assert torch.equal(seen.path[far, 1], node[far].to(I32))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_vocabularies_of_millions(tq, dtype):
    # 20000 pieces a row, 80000 or 160000 vectors; drawn and refused
    seqs, vocab = 4, 20_000_003
    logits, temp, gen = language(seqs, vocab, dtype, 11)
    cum = weights(logits, temp).cumsum_(1)
    start, tokens = start_of(seqs, 1), torch.zeros(seqs, dtype=I32, device=DEV)
    for turn in range(6):
        u = torch.rand(seqs, generator=gen, device=DEV)
        equal(tq.tq_verify_tree(logits, start, tokens, u, 1, temperature=temp, check=True).next_token, *drawn(cum, u))
    logits, temp, q, tokens, parents, ua, cum, z, gen = refused(2, 1, vocab, dtype, BF16, seed=12)
    for turn in range(6):
        us = torch.rand(4, generator=gen, device=DEV)
        seen = tq.tq_verify_tree(logits, start_of(2, 2), tokens, us, 2, parents=parents, temperature=temp, draft_probs=q, u_accept=ua)
        i, d = drawn(cum, us[::2])
        equal(seen.next_token, i, d * z)


def test_a_captured_call_follows_its_inputs(tq):
    # sequences that need more than fp32 in one replay and not in the next
    seqs, vocab = 100, 33001
    logits, temp, gen = language(seqs, vocab, BF16, 5)
    cum = weights(logits, temp).cumsum_(1)
    start, tokens, u = start_of(seqs, 1), torch.zeros(seqs, dtype=I32, device=DEV), torch.zeros(seqs, device=DEV)
    out = tq.Verified(torch.empty(seqs, 1, dtype=I32, device=DEV), torch.empty(seqs, dtype=I32, device=DEV),
                      torch.empty(seqs, dtype=I32, device=DEV))
    ws = torch.full((tq.tq_verify_tree_workspace(seqs, vocab, seqs),), 255, dtype=torch.uint8, device=DEV)

    def work():
        tq.tq_verify_tree(logits, start, tokens, u, 1, temperature=temp, out=out, workspace=ws)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for turn in range(6):
        u.copy_(at_borders(cum, gen, turn) if turn % 2 else torch.rand(seqs, generator=gen, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        equal(out.next_token, *drawn(cum, u), most=1 + turn % 2)


def test_long_walks(tq):
    # more nodes than shared memory holds, every drafted token the one that is drawn
    rows, vocab = [300, 700, 3], 400
    for kind in ("chain", "tree"):
        logits, _, gen = language(sum(rows), vocab, F32, 9)
        start = np.concatenate([[0], np.cumsum(rows)])
        cum = weights(logits, torch.ones(sum(rows), device=DEV)).cumsum_(1)
        u = torch.rand(sum(rows), generator=gen, device=DEV)
        u[::3] = at_borders(cum, gen, 0)[::3]
        u = torch.where(drawn(cum, u)[1] > TIE, u, 0.5)
        want, near = drawn(cum, u)
        assert (near > TIE).all()
        want = want.cpu().numpy()
        tokens, parents, paths = np.zeros(sum(rows), dtype=np.int32), np.zeros(sum(rows), dtype=np.int32), []
        for r0, n in zip(start, rows):
            # a tree: behind each node of the walk a child that is drawn and one that is not
            up = np.arange(n) - 1 if kind == "chain" else np.where(np.arange(n) % 2, np.arange(n) - 2, np.arange(n) - 1)
            up = np.maximum(up, 0)
            parents[r0:r0 + n] = up
            path = [0]
            for i in range(1, n):
                good = kind == "chain" or i % 2 == 1
                tokens[r0 + i] = (want[r0 + up[i]] + (0 if good else 1)) % vocab
                if good:
                    path.append(i)
            if kind == "tree":
                parents[r0 + 1] = 0
            paths.append(path)
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()  # noqa: E731
        seen = tq.tq_verify_tree(logits, c(start), c(tokens), u, 700, parents=None if kind == "chain" else c(parents), check=True)
        for s, path in enumerate(paths):
            assert int(seen.path_lens[s]) == len(path)
            assert seen.path[s, :len(path)].tolist() == path
            assert int(seen.next_token[s]) == want[start[s] + path[-1]]
        assert len(paths[1]) >= 350


def test_more_sequences_than_clusters(tq):
    # draft probabilities, small vocabularies: clusters take sequences in turn
    seqs, vocab = 2500, 300
    logits, temp, q, tokens, parents, ua, cum, z, gen = refused(seqs, 1, vocab, BF16, F32, seed=3)
    us = torch.rand(seqs * 2, generator=gen, device=DEV)
    seen = tq.tq_verify_tree(logits, start_of(seqs, 2), tokens, us, 2, parents=parents, temperature=temp, draft_probs=q,
                             u_accept=ua, check=True)
    i, d = drawn(cum, us[::2])
    equal(seen.next_token, i, d * z, most=1)

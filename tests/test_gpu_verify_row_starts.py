"""tq_verify_tree with a row_start whose last entry lies below an earlier one: sequences with rows behind the
last entry have none, whatever the workspace holds, and the others are what they are in a good list."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

I32 = torch.int32


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


@pytest.mark.parametrize("many", [0, 100])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("bad", [[0, 4, 12, 7], [0, 4, 4, 2], [0, 4, 4, -1], [0, 4, 2], [3, 9, 12, 0], [0, 2 ** 31 - 1, 5]])
def test_last_entry_below_an_earlier_one(tq, bad, greedy, draft, many):
    # `many`: as many empty sequences in front, so that a call takes its form for many sequences
    bad = [0] * many + bad if many and bad[0] == 0 else bad
    seqs, rows, vocab = len(bad) - 1, 12, 2100
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(rows, vocab, generator=gen, device="cuda") * 3
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=I32)
    args = dict(temperature=torch.full((seqs,), 0.0 if greedy else 0.8, device="cuda"))
    if draft:
        args.update(draft_probs=torch.softmax(x + torch.randn(x.shape, generator=gen, device="cuda"), 1),
                    u_accept=torch.rand(rows, generator=gen, device="cuda"))
    us = torch.rand(rows, generator=gen, device="cuda")

    def call(start):
        ws = torch.full((tq.tq_verify_tree_workspace(rows, vocab, seqs),), 255, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=I32, device="cuda")
        seen = tq.tq_verify_tree(x, torch.tensor(start, dtype=I32, device="cuda"), tokens, us, 5, workspace=ws, status=status,
                                 **args)
        return seen, int(status.item())

    got, status = call(bad)
    assert status == tq.TQ_ERR_INVALID_ARG
    for s in range(seqs):
        if bad[s] >= 0 and bad[s] <= bad[s + 1] <= min(rows, bad[-1]):
            # the same sequence alone in a good list
            good = [bad[s]] * (s + 1) + [bad[s + 1]] * (seqs - s)
            want, _ = call(good)
            assert torch.equal(got.path[s], want.path[s]) and got.path_lens[s] == want.path_lens[s]
            assert got.next_token[s] == want.next_token[s]
        else:
            assert got.path_lens[s] == 0 and got.next_token[s] == -1 and torch.all(got.path[s] == -1)


@pytest.mark.parametrize("draft", [False, True])
def test_rows_that_two_sequences_claim(tq, draft):
    # one draws from them, the other takes largest logits: neither reads the other's numbers
    rows, vocab, start = 12, 1500, [0, 8, 3, 12]
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(rows, vocab, generator=gen, device="cuda") * 3
    best = x.argmax(1).to(I32)
    tokens = torch.roll(best, 1)  # greedy walks go on to the end
    for temps in ([0.7, 0.0, 0.0], [0.0, 0.0, 0.7]):
        args = dict(temperature=torch.tensor(temps, device="cuda"))
        if draft:
            args.update(draft_probs=torch.softmax(x, 1), u_accept=torch.zeros(rows, device="cuda"))
        ws = torch.full((tq.tq_verify_tree_workspace(rows, vocab, 3),), 255, dtype=torch.uint8, device="cuda")
        status = torch.zeros(1, dtype=I32, device="cuda")
        seen = tq.tq_verify_tree(x, torch.tensor(start, dtype=I32, device="cuda"), tokens, torch.rand(rows, generator=gen, device="cuda"),
                                 12, workspace=ws, status=status, **args)
        assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
        assert torch.all((seen.next_token >= -1) & (seen.next_token < vocab)) and seen.path_lens[1] == 0
        lens = seen.path_lens.tolist()
        for s in (0, 2):  # a greedy walk is right as far as it goes
            if temps[s] == 0.0:
                assert seen.path[s, :lens[s]].tolist() == list(range(lens[s]))
                assert seen.next_token[s] in (-1, best[start[s] + lens[s] - 1])

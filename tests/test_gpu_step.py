"""tq_plan_step and tq_commit_tree on the GPU against the sequential oracle: whole numbers and
bytes, so every output has to be equal."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import step_oracle as so  # noqa: E402

pytestmark = pytest.mark.gpu


def _tq():
    import quantized_kv_cache_06_gb300 as tq

    return tq


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def _state(rng, s, bs, width, spare_blocks, finished=0.1, most_new=None, reserve=True):
    lens = rng.integers(0, width * bs + 1, size=s)
    blocks = -(-lens // bs)
    if reserve:  # some sequences hold blocks that an earlier step reserved
        blocks = np.minimum(width, blocks + rng.integers(0, 2, size=s))
    new = np.minimum(rng.integers(0, (most_new or 2 * bs) + 1, size=s), width * bs - lens)
    new[rng.random(s) < finished] = -1
    used = int(blocks.sum())
    nb = used + spare_blocks
    perm = rng.permutation(nb)
    table = rng.integers(-5, 5, size=(s, width))  # entries not in use hold anything
    at = 0
    for i in range(s):
        table[i, :blocks[i]] = perm[at:at + blocks[i]]
        at += blocks[i]
    ring = np.full(nb, -7)
    head = int(rng.integers(0, nb)) if nb else 0
    ring[(head + np.arange(spare_blocks)) % max(nb, 1)] = perm[used:]
    return lens, new, blocks, table, ring, np.array([head, spare_blocks])


def _run(tq, lens, new, blocks, table, ring, state, bs, max_rows, inplace=False, check=False):
    t = [_dev(x) for x in (lens, new, blocks, table, ring, state)]
    out = None
    if inplace:
        e = lambda n, dt=torch.int32: torch.full((n,), 77, dtype=dt, device="cuda")  # noqa: E731
        out = tq.StepPlan(e(max_rows, torch.int64), e(max_rows), e(max_rows), e(len(lens) + 1), t[0], t[2], t[5])
    status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    p = tq.tq_plan_step(*t, bs, max_rows, out=out, status=status, check=check)
    return p, t[3], t[4], int(status.item())


def _equal(p, table, ring, want):
    for name in ("slots", "q_seq", "q_len", "row_start", "seq_lens", "seq_blocks", "free_state"):
        assert np.array_equal(getattr(p, name).cpu().numpy(), want[name]), name
    assert np.array_equal(table.cpu().numpy(), want["table"])
    assert np.array_equal(ring.cpu().numpy(), want["ring"])


@pytest.mark.parametrize("s,bs,width,spare,extra,inplace", [
    (1, 16, 4, 8, 0, False), (1, 1, 7, 20, 3, True), (5, 16, 9, 64, 1, True), (64, 16, 40, 900, 11, False),
    (33, 3, 50, 400, 0, True), (1023, 8, 6, 6000, 7, True), (1024, 16, 4, 4000, 0, False),
    (1025, 4, 5, 5000, 900, True), (3000, 2, 7, 12000, 5, False)])
def test_plan_matches_the_oracle(s, bs, width, spare, extra, inplace):
    tq = _tq()
    rng = np.random.default_rng(s * 1000 + bs)
    st = _state(rng, s, bs, width, spare)
    rows = int(np.maximum(st[1], 0).sum()) + extra
    want = so.plan_step(*st, bs, rows)
    p, table, ring, code = _run(tq, *st, bs, rows, inplace)
    assert code == tq.TQ_OK
    _equal(p, table, ring, want)


def test_plan_long_prompt_over_a_cluster():
    tq = _tq()
    rng = np.random.default_rng(9)
    bs, width = 16, 8192
    lens, new = np.array([5, 0, 100, 131000]), np.array([1, 70001, 0, 72])
    blocks = -(-lens // bs)
    nb = int(blocks.sum()) + 4500
    perm = rng.permutation(nb)
    table = np.zeros((4, width), dtype=np.int64)
    at = 0
    for i in range(4):
        table[i, :blocks[i]] = perm[at:at + blocks[i]]
        at += blocks[i]
    ring = np.zeros(nb, dtype=np.int64)
    head = nb - 100  # the taken blocks wrap around the ring
    ring[(head + np.arange(nb - at)) % nb] = perm[at:]
    st = (lens, new, blocks, table, ring, np.array([head, nb - at]))
    rows = int(new.sum())
    p, t, r, code = _run(tq, *st, bs, rows)
    assert code == tq.TQ_OK
    _equal(p, t, r, so.plan_step(*st, bs, rows))


def test_plan_without_sequences_or_rows():
    tq = _tq()
    z = np.zeros(0, dtype=np.int64)
    p, _, _, code = _run(tq, z, z, z, np.zeros((0, 3), dtype=np.int64), np.arange(4), np.array([1, 2]), 16, 5)
    assert code == tq.TQ_OK and p.slots.tolist() == [-1] * 5 and p.row_start.tolist() == [0]
    assert p.free_state.tolist() == [1, 2]
    one = np.array([20])
    p, _, _, code = _run(tq, one, np.array([0]), np.array([2]), np.array([[3, 1]]), np.arange(4), np.array([1, 2]), 16, 0)
    assert code == tq.TQ_OK and p.row_start.tolist() == [0, 0] and p.seq_lens.tolist() == [20]


@pytest.mark.parametrize("change,code", [
    (dict(lens=[40, 3]), "TQ_ERR_INVALID_ARG"), (dict(lens=[-1, 3]), "TQ_ERR_INVALID_ARG"),
    (dict(new=[40, 1]), "TQ_ERR_INVALID_ARG"), (dict(state=[0, 1]), "TQ_ERR_OUT_OF_BLOCKS"),
    (dict(state=[6, 2]), "TQ_ERR_INVALID_ARG"), (dict(state=[0, 7]), "TQ_ERR_INVALID_ARG"),
    (dict(state=[-1, 2]), "TQ_ERR_INVALID_ARG"), (dict(rows=20), "TQ_ERR_INVALID_ARG"),
    (dict(blocks=[4, 1]), "TQ_ERR_INVALID_ARG"), (dict(state=[0, 6], new=[1, -1]), "TQ_ERR_INVALID_ARG")])
def test_plan_refusals_change_nothing(change, code):
    tq = _tq()
    st = dict(lens=[30, 3], new=[3, 30], blocks=[2, 1], state=[0, 4], rows=40)
    st.update(change)
    table, ring = np.array([[0, 1, -1], [2, -1, -1]]), np.array([3, 4, 5, 5, 5, 5])
    p, t, r, got = _run(tq, np.array(st["lens"]), np.array(st["new"]), np.array(st["blocks"]), table, ring,
                        np.array(st["state"]), 16, st["rows"])
    assert got == getattr(tq, code)
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), ring)
    assert p.seq_lens.tolist() == st["lens"] and p.seq_blocks.tolist() == st["blocks"]
    assert p.free_state.tolist() == st["state"]
    assert p.slots.tolist() == [-1] * st["rows"] and p.q_seq.tolist() == [-1] * st["rows"]
    with pytest.raises(tq.TQError):
        _run(tq, np.array(st["lens"]), np.array(st["new"]), np.array(st["blocks"]), table, ring, np.array(st["state"]),
             16, st["rows"], check=True)


def test_plan_refuses_a_ring_that_meets_its_returned_blocks():
    # six blocks, all said to be free, one of them in use and returned
    tq = _tq()
    table, ring = np.array([[0, 1, -1], [2, -1, -1]]), np.arange(6)
    args = np.array([30, 3]), np.array([3, -1]), np.array([2, 1])
    p, t, r, code = _run(tq, *args, table, ring, np.array([0, 6]), 16, 3)
    assert code == tq.TQ_ERR_INVALID_ARG and p.free_state.tolist() == [0, 6]
    assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), ring)
    # the same with one less: the ring is full afterwards but for the block taken
    p, t, r, code = _run(tq, *args, table, ring, np.array([0, 5]), 16, 3)
    assert code == tq.TQ_OK and p.free_state.tolist() == [1, 5]
    assert t.tolist()[0] == [0, 1, 0] and r.tolist() == [0, 1, 2, 3, 4, 2]


def test_plan_reports_bad_block_ids():
    tq = _tq()
    # the partly filled block of sequence 0 and a ring entry lie outside the pages
    p, t, _, code = _run(tq, np.array([5, 0]), np.array([2, 3]), np.array([1, 0]), np.array([[9], [0]]),
                         np.array([-3, 1, 2]), np.array([0, 3]), 16, 5)
    assert code == tq.TQ_ERR_BLOCK_OUT_OF_RANGE
    assert p.slots.tolist() == [-1] * 5 and t.tolist() == [[9], [-3]]


# ---------------------------------------------------------------- commit

def _commit_case(rng, s, bs, h, rbs, nodes, most_path, ctx_max):
    ctx = rng.integers(0, ctx_max + 1, size=s)
    blocks = -(-(ctx + nodes) // bs)
    width, nb = int(blocks.max()), int(blocks.sum()) + 2
    perm = rng.permutation(nb)
    table = np.zeros((s, width), dtype=np.int64)
    at = 0
    for i in range(s):
        table[i, :blocks[i]] = perm[at:at + blocks[i]]
        at += blocks[i]
    path = np.stack([np.sort(rng.permutation(nodes)[:most_path]) for _ in range(s)])
    count = rng.integers(0, most_path + 1, size=s)
    pages = [rng.integers(0, 256, size=(nb, bs, h, rb), dtype=np.uint8) for rb in rbs]
    return ctx, table, path, count, pages


@pytest.mark.parametrize("s,bs,h,rbs,nodes,path,ctx", [
    (1, 16, 8, (68, 68), 8, 8, 40), (7, 16, 8, (68, 36), 16, 4, 100), (3, 16, 2, (68, 36), 64, 12, 5),
    (5, 1, 1, (8, 14), 5, 3, 3), (4, 5, 3, (10, 10), 33, 33, 9), (2, 8, 5, (13, 7), 20, 20, 30),
    (2, 16, 4, (72, 56), 200, 150, 500), (300, 4, 1, (132, 132), 3, 1, 6)])
def test_commit_matches_the_oracle(s, bs, h, rbs, nodes, path, ctx):
    tq = _tq()
    rng = np.random.default_rng(s + nodes + path)
    ctx, table, path, count, pages = _commit_case(rng, s, bs, h, rbs, nodes, path, ctx)
    dev = [torch.from_numpy(p).cuda() for p in pages]
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    lens = tq.tq_commit_tree(dev[0], dev[1], _dev(table), _dev(ctx), _dev(path), _dev(count), status=status, check=True)
    for got, p in zip(dev, pages):
        want, want_lens = so.commit_tree(p, table, ctx, path, count)
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(lens.cpu().numpy(), want_lens)


def test_commit_one_component_in_place_lengths_and_whole_path():
    tq = _tq()
    rng = np.random.default_rng(4)
    ctx, table, path, count, pages = _commit_case(rng, 4, 16, 8, (84,), 32, 9, 60)
    count[:] = 9
    k = torch.from_numpy(pages[0]).cuda()
    lens = _dev(ctx)
    assert tq.tq_commit_tree(None, k, _dev(table), lens, _dev(path), _dev(count), seq_lens=lens) is lens
    want, want_lens = so.commit_tree(pages[0], table, ctx, path, count)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(lens.cpu().numpy(), want_lens)


@pytest.mark.parametrize("h,rbs", [(16, (132, 132)), (5, (133, 259)), (64, (164, 164))])
def test_commit_of_wide_tokens_with_lengths_in_place(h, rbs):
    # more 16-byte (or 1-byte) columns than a CTA has threads
    tq = _tq()
    rng = np.random.default_rng(h)
    ctx, table, path, count, pages = _commit_case(rng, 40, 4, h, rbs, 9, 6, 20)
    dev = [torch.from_numpy(p).cuda() for p in pages]
    lens = _dev(ctx)
    assert tq.tq_commit_tree(dev[0], dev[1], _dev(table), lens, _dev(path), _dev(count), seq_lens=lens) is lens
    for got, p in zip(dev, pages):
        want, want_lens = so.commit_tree(p, table, ctx, path, count)
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(lens.cpu().numpy(), want_lens)


def test_commit_bad_paths_move_nothing():
    tq = _tq()
    rng = np.random.default_rng(6)
    ctx, table, path, count, pages = _commit_case(rng, 6, 8, 2, (68, 68), 16, 5, 30)
    count[:] = 3
    path[0, 1] = path[0, 0]      # not ascending
    path[1, 2] = 10 ** 6         # beyond the table
    count[2] = 6                 # longer than max_path
    count[3] = -1
    path[4, 0] = -2
    dev = [torch.from_numpy(p).cuda() for p in pages]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = tq.tq_commit_tree(dev[0], dev[1], _dev(table), _dev(ctx), _dev(path), _dev(count), status=status)
    assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
    for got, p in zip(dev, pages):
        want, want_lens = so.commit_tree(p, table, ctx, path, count)
        assert np.array_equal(got.cpu().numpy(), want)
    assert np.array_equal(lens.cpu().numpy(), want_lens) and np.array_equal(want_lens[:5], ctx[:5])


def test_commit_bad_block_ids_are_reported():
    tq = _tq()
    rng = np.random.default_rng(8)
    ctx, table, path, count, pages = _commit_case(rng, 2, 4, 2, (68, 68), 12, 6, 0)
    count[:] = 6
    table[1, -1] = 10 ** 5
    path[:] = [1, 3, 5, 7, 8, 11]
    dev = [torch.from_numpy(p).cuda() for p in pages]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_commit_tree(dev[0], dev[1], _dev(table), _dev(ctx), _dev(path), _dev(count), status=status)
    assert int(status.item()) == tq.TQ_ERR_BLOCK_OUT_OF_RANGE
    for got, p in zip(dev, pages):
        assert np.array_equal(got.cpu().numpy(), so.commit_tree(p, table, ctx, path, count)[0])

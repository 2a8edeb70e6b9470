"""tq_paged_tree and tq_paged_prefill_biased on the GPU against the fp64 oracle.

Tolerances.  With a score error dx (natural units) and values bounded by V over the visible
tokens, |out - exact| <= 2 V dx (weights move by at most e^(2 dx)) plus the roundings of the
weights, the values and the output.
  fp32 output: everything in fp32.  A score is D products summed in order, dx <= (D + 24) u S
    with u = 2^-24 and S the largest |scale nu <q, c>| bound, scale |q| nu |c|; the sums over n
    tokens round n times.  The tests' S stays below 40 and n below 2^13; errors of the sums are
    independent, so sqrt(n) u is taken for them.
  fp16 / bf16 output: centroids, weights and (bf16) queries rounded once to fp16, half a step
    2^-11 each.  dx: D independent errors, 6 standard deviations of 2^-11 / sqrt(3) on terms of
    root sum of squares S / sqrt(D) times 2 (rotated coordinates are near Gaussian): at S = 40,
    D = 64: 6 * 2.8e-4 * 10 = 1.7e-2.  Weights and values: 2 * 2^-11 V.  Output: half a step.
The norm of the whole error is held to what independent roundings leave: fp32 1e-5, fp16
2 * 2^-11, bf16 2^-8 of the norm of the output.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import step_oracle as so  # noqa: E402
from oracle import tq_oracle as o  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
NORM = {"fp32": 1e-5, "fp16": 2 * 2.0 ** -11, "bf16": 2.0 ** -8}


def _tq():
    import quantized_kv_cache_06_gb300 as tq

    return tq


class Cache:
    """Random packed rows behind a permuted block table; rows of no token are random bytes."""

    def __init__(self, rng, lens, d, h, kb, vb, bs=16, norm=1.0, spare=2):
        self.d, self.h, self.kb, self.vb, self.bs = d, h, kb, vb, bs
        blocks = [-(-int(n) // bs) for n in lens]
        self.nb = sum(blocks) + spare
        self.width = max(max(blocks), 1)
        perm = rng.permutation(self.nb)
        self.bt = np.zeros((len(lens), self.width), dtype=np.int32)
        at = 0
        for i, b in enumerate(blocks):
            self.bt[i, :b] = perm[at:at + b]
            at += b
        self.signs = o.splitmix64_signs(d, 42)
        self.kc, self.vc = o.codebook_f32(d, kb)[0], o.codebook_f32(d, vb)[0]
        self.pages = []
        for bits in (kb, vb):
            pg = rng.integers(0, 256, size=(self.nb, bs, h, o.row_bytes(d, bits)), dtype=np.uint8)
            for i, n in enumerate(lens):
                t = np.arange(int(n))
                idx = rng.integers(0, 1 << bits, size=(int(n) * h, d))
                nu = (norm * math.sqrt(d) * rng.lognormal(0.0, 0.3, size=int(n) * h)).astype(np.float32)
                pg[self.bt[i, t // bs], t % bs] = o.make_rows(idx, nu, bits).reshape(int(n), h, -1)
            self.pages.append(pg)

    @property
    def cap(self):
        return self.width * self.bs

    def dev(self):
        f = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)  # noqa: E731
        return dict(k_pages=f(self.pages[0], torch.uint8), v_pages=f(self.pages[1], torch.uint8),
                    block_table=f(self.bt, torch.int32), signs=f(self.signs, torch.float32),
                    k_centroids=f(self.kc, torch.float32), v_centroids=f(self.vc, torch.float32))

    def oracle(self, q, q_seq, see, **kw):
        return so.attention(q, q_seq, see, *self.pages, self.kb, self.vb, self.bt, self.signs, self.kc, self.vc, **kw)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()


def _close(got, want, reach, dtype, d):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    if dtype == "fp32":
        dx = (d + 24) * 2.0 ** -24 * 40 + 90 * 2.0 ** -24
        tol = 2 * dx * reach[..., None]
    else:
        dx = 6 * 2.0 ** -11 / math.sqrt(3) * 40 / math.sqrt(d) * 2
        tol = (dx + 2 * 2.0 ** -11) * reach[..., None] + HALF_STEP[dtype] * np.abs(want)
    err = np.abs(got - want)
    assert np.all(err <= tol + 1e-12), float((err - tol).max())
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= NORM[dtype] * norm + 1e-12, np.linalg.norm(got - want) / norm


def _tree(rng, counts, words=None):
    """Random trees: mask words of the ancestors and the node itself."""
    words = words or -(-max(list(counts) + [1]) // 32)
    out = []
    for n in counts:
        see = np.zeros((n, 32 * words), dtype=np.uint64)
        for i in range(n):
            if i and rng.random() < 0.9:
                see[i] = see[rng.integers(0, i)]
            see[i, i] = 1
        out.append((see.reshape(n, words, 32) << np.arange(32, dtype=np.uint64)).sum(2))
    return np.concatenate(out).astype(np.uint32)


def _run_tree(tq, c, q, dtype, q_seq, ctx, mask, **kw):
    qd = torch.from_numpy(q).cuda().to(DT[dtype])
    status = torch.full((1,), 55, dtype=torch.int32, device="cuda")
    out = tq.tq_paged_tree(qd, _i32(q_seq), _i32(ctx), _i32(mask.view(np.int32)), **c.dev(), status=status, **kw)
    torch.cuda.synchronize()
    return out, qd.float().cpu().numpy(), int(status.item())


TREE_CASES = [
    # d, kb, vb, hq, h, bs, contexts, nodes
    (128, 4, 4, 16, 2, 16, [64], [8]),
    (128, 4, 4, 32, 8, 16, [100, 0, 1, 300], [7, 5, 1, 33]),
    (128, 4, 2, 16, 4, 16, [127, 128, 129], [1, 2, 3]),
    (128, 2, 4, 8, 1, 8, [500], [40]),
    (128, 3, 3, 8, 8, 32, [140, 17], [64, 9]),
    (128, 5, 5, 8, 4, 64, [200, 33], [17, 2]),
    (128, 3, 5, 12, 3, 1, [37, 130], [4, 12]),
    (128, 2, 2, 20, 5, 24, [90, 260], [3, 30]),
    (64, 4, 4, 16, 2, 16, [64, 255], [8, 20]),
    (64, 2, 3, 32, 4, 16, [300], [65]),
    (64, 3, 2, 4, 4, 128, [129, 400], [2, 1]),
    (64, 5, 4, 8, 4, 256, [10, 600], [11, 5]),
    (256, 4, 4, 8, 1, 16, [130, 31], [9, 70]),
    (256, 5, 5, 32, 8, 16, [77], [3]),
    (256, 3, 2, 8, 4, 5, [200, 1], [6, 1]),
    (256, 4, 5, 8, 4, 16, [300, 20], [40, 2]),
    (256, 4, 3, 4, 4, 16, [300, 20], [40, 2]),
    (256, 5, 4, 8, 4, 16, [300, 20], [4, 2]),
    (128, 4, 5, 16, 4, 16, [700], [20]),
    (64, 5, 5, 16, 4, 16, [700], [20]),
    (32, 4, 3, 8, 2, 16, [70], [12]),
    (16, 3, 5, 8, 2, 16, [70, 3], [12, 1]),
]


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("case", TREE_CASES, ids=lambda c: "d%d_k%dv%d_%dx%d_bs%d" % c[:6])
def test_tree_matches_the_oracle(case, dtype):
    tq = _tq()
    d, kb, vb, hq, h, bs, ctx, nodes = case
    rng = np.random.default_rng(d + 10 * kb + vb + bs + hq)
    c = Cache(rng, np.add(ctx, nodes), d, h, kb, vb, bs)
    q_seq = np.repeat(np.arange(len(ctx)), nodes)
    mask = _tree(rng, nodes)
    q = rng.standard_normal((len(q_seq), hq, d)).astype(np.float32)
    out, qr, code = _run_tree(tq, c, q, dtype, q_seq, ctx, mask)
    assert code == tq.TQ_OK
    want, reach = c.oracle(qr, q_seq, so.tree_visible(q_seq, ctx, mask, c.cap))
    _close(out, want, reach, dtype, d)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tree_softcap_scale_and_empty_rows(d, dtype):
    tq = _tq()
    rng = np.random.default_rng(d)
    ctx, nodes = [0, 150, 0], [6, 3, 2]
    c = Cache(rng, np.add(ctx, nodes), d, 4, 4, 4)
    q_seq = np.repeat(np.arange(3), nodes)
    mask = _tree(rng, nodes, words=3)
    mask[[2, 9]] = 0  # rows that see nothing (context of length 0)
    q = rng.standard_normal((11, 16, d)).astype(np.float32)
    out, qr, code = _run_tree(tq, c, q, dtype, q_seq, ctx, mask, scale=0.11, softcap=3.0)
    assert code == tq.TQ_OK
    assert torch.all(out[[2, 9]] == 0)
    want, reach = c.oracle(qr, q_seq, so.tree_visible(q_seq, ctx, mask, c.cap), scale=0.11, softcap=3.0)
    _close(out, want, reach, dtype, d)


def _random_view(rng, lens, rows):
    q_seq, q_len = [], []
    for s, (n, r) in enumerate(zip(lens, rows)):
        q_seq += [s] * r
        q_len += list(range(n - r + 1, n + 1))
    return np.array(q_seq), np.array(q_len)


BIASED = [dict(), dict(window=1), dict(window=70), dict(alibi=True), dict(softcap=2.0), dict(prefix=[0, 40, 200, 1]),
          dict(docs=True), dict(window=33, prefix=[5, 0, 300, 1]), dict(docs=True, prefix=[150, 20, 90, 1]),
          dict(window=130, alibi=True, softcap=4.0, docs=True, prefix=[9, 3, 140, 1])]


@pytest.mark.parametrize("kind", range(len(BIASED)))
@pytest.mark.parametrize("shape", [(128, 4, 4, 16, 4, 16, "bf16"), (128, 4, 2, 8, 1, 16, "fp16"),
                                   (64, 3, 3, 8, 8, 16, "fp16"), (256, 5, 5, 16, 4, 32, "bf16"),
                                   (64, 2, 4, 8, 2, 8, "fp32"), (16, 2, 2, 4, 2, 16, "fp16")],
                         ids=lambda s: "d%d_k%dv%d_%dx%d_bs%d_%s" % s)
def test_biased_matches_the_oracle(shape, kind):
    tq = _tq()
    d, kb, vb, hq, h, bs, dtype = shape
    b = BIASED[kind]
    rng = np.random.default_rng(kind * 100 + d + kb)
    lens, rows = [300, 64, 513, 1], [20, 64, 3, 1]
    c = Cache(rng, lens, d, h, kb, vb, bs)
    q_seq, q_len = _random_view(rng, lens, rows)
    docs = np.array([int(rng.integers(0, n)) for n in q_len]) if b.get("docs") else None
    slopes = np.array([2.0 ** (-8 * (i + 1) / hq) for i in range(hq)], dtype=np.float32) if b.get("alibi") else None
    q = rng.standard_normal((len(q_seq), hq, d)).astype(np.float32)
    qd = torch.from_numpy(q).cuda().to(DT[dtype])
    status = torch.full((1,), 55, dtype=torch.int32, device="cuda")
    out = tq.tq_paged_prefill_biased(qd, _i32(q_seq), _i32(q_len), **c.dev(), softcap=b.get("softcap", 0.0),
                                     window=b.get("window", 0), prefix_lens=_i32(b["prefix"]) if "prefix" in b else None,
                                     doc_starts=None if docs is None else _i32(docs),
                                     alibi_slopes=None if slopes is None else torch.from_numpy(slopes).cuda(),
                                     status=status)
    assert int(status.item()) == tq.TQ_OK
    see = so.biased_visible(q_seq, q_len, c.cap, len(lens), b.get("window", 0), b.get("prefix"), docs)
    want, reach = c.oracle(qd.float().cpu().numpy(), q_seq, see, softcap=b.get("softcap", 0.0), slopes=slopes,
                           q_pos=q_len - 1)
    _close(out, want, reach, dtype, d)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 31])
def test_decode_batches_and_padding_rows(dtype, rows):
    # many sequences with a few rows each, rows out of order, padding rows between and behind
    tq = _tq()
    rng = np.random.default_rng(rows)
    lens = [int(x) for x in rng.integers(1, 400, size=9)]
    c = Cache(rng, lens, 128, 4, 4, 4)
    q_seq = np.concatenate([rng.permutation(9).repeat(rows), [-1] * 5])
    q_seq = np.insert(q_seq, [3, 3, 7], -1)
    q_len = np.array([int(rng.integers(0, lens[s] + 1)) if s >= 0 else 0 for s in q_seq])
    q = rng.standard_normal((len(q_seq), 16, 128)).astype(np.float32)
    qd = torch.from_numpy(q).cuda().to(DT[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = tq.tq_paged_prefill_biased(qd, _i32(q_seq), _i32(q_len), **c.dev(), status=status, check=True)
    assert torch.all(out[torch.from_numpy(q_seq < 0).cuda()] == 0)
    see = so.biased_visible(q_seq, q_len, c.cap, 9)
    want, reach = c.oracle(qd.float().cpu().numpy(), q_seq, see)
    _close(out, want, reach, dtype, 128)


@pytest.mark.parametrize("slope", [0.3, 0.65, 0.7, 1.0, 4.0])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 256])
def test_a_distance_bias_that_moves_every_maximum(d, dtype, slope):
    # weights of one tile against the maximum of the one before: 2^55 to beyond the largest float
    tq = _tq()
    rng = np.random.default_rng(int(100 * slope) + d)
    lens = [700, 900]
    c = Cache(rng, lens, d, 2, 4, 4)
    q_seq, q_len = np.array([0, 1, 1]), np.array([700, 900, 513])
    q = rng.standard_normal((3, 4, d)).astype(np.float32)
    qd = torch.from_numpy(q).cuda().to(DT[dtype])
    slopes = np.array([slope, slope / 2, slope, 1.5 * slope])
    out = tq.tq_paged_prefill_biased(qd, _i32(q_seq), _i32(q_len), **c.dev(), check=True,
                                     alibi_slopes=torch.from_numpy(slopes).float().cuda())
    see = so.biased_visible(q_seq, q_len, c.cap, 2)
    want, reach = c.oracle(qd.float().cpu().numpy(), q_seq, see, slopes=slopes.astype(np.float32).astype(np.float64),
                           q_pos=q_len - 1)
    # (what has weight lies near the row: its bias, at most 30, is off by as many 2^-24)
    _close(out, want, reach * (2 if dtype == "fp32" else 1), dtype, d)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_long_sequence_among_single_tokens(d, dtype):
    # few rows a sequence on average, so narrow windows; one sequence fills several of them
    tq = _tq()
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(1, 300, size=11)] + [350]
    c = Cache(rng, lens, d, 2, 4, 3)
    q_seq = np.concatenate([np.arange(11), np.full(50, 11)])
    q_len = np.concatenate([lens[:11], np.arange(301, 351)])
    q = rng.standard_normal((len(q_seq), 8, d)).astype(np.float32)
    qd = torch.from_numpy(q).cuda().to(DT[dtype])
    out = tq.tq_paged_prefill_biased(qd, _i32(q_seq), _i32(q_len), **c.dev(), window=170, check=True)
    want, reach = c.oracle(qd.float().cpu().numpy(), q_seq, so.biased_visible(q_seq, q_len, c.cap, 12, window=170))
    _close(out, want, reach, dtype, d)


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_agrees_with_the_prefill_without_modifiers(dtype):
    tq = _tq()
    rng = np.random.default_rng(12)
    lens, rows = [700, 90], [33, 5]
    c = Cache(rng, lens, 128, 8, 4, 4)
    q_seq, q_len = _random_view(rng, lens, rows)
    q = torch.from_numpy(rng.standard_normal((38, 32, 128)).astype(np.float32)).cuda().to(DT[dtype])
    dv = c.dev()
    a = tq.tq_paged_prefill_biased(q, _i32(q_seq), _i32(q_len), **dv, out_dtype=torch.float32)
    b = tq.tq_paged_prefill(q, _i32(q_seq), _i32(q_len), **dv, out_dtype=torch.float32)
    err = (a - b).abs()
    assert torch.all(err <= 2e-3 + 2e-3 * b.abs())  # the prefill's own tolerance


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_bad_rows_lengths_and_blocks(dtype):
    tq = _tq()
    rng = np.random.default_rng(3)
    c = Cache(rng, [100, 50], 128, 2, 4, 4)
    q = rng.standard_normal((4, 8, 128)).astype(np.float32)
    # a sequence outside the table; a node beyond the table row
    mask = np.array([[1], [1], [1 << 31], [3]], dtype=np.uint32)
    q_seq = np.array([0, 7, 0, 1])
    ctx = [99, 48]
    out, qr, code = _run_tree(tq, c, q, dtype, q_seq, ctx, mask)
    assert code == tq.TQ_ERR_INVALID_ARG and torch.all(out[1] == 0)
    see = so.tree_visible(q_seq, ctx, mask, c.cap)
    want, reach = c.oracle(qr, q_seq, see)
    _close(out, want, reach, dtype, 128)
    # a block id outside the pages: its tokens are left out
    c.bt[0, 2] = c.nb + 3
    c.bt[1, 1] = -1
    mask[2] = 1
    out, qr, code = _run_tree(tq, c, q, dtype, [0, 0, 0, 1], ctx, mask)
    assert code == tq.TQ_ERR_BLOCK_OUT_OF_RANGE
    want, reach = c.oracle(qr, [0, 0, 0, 1], so.tree_visible([0, 0, 0, 1], ctx, mask, c.cap))
    _close(out, want, reach, dtype, 128)
    # contexts and lengths beyond the table row are clamped
    c = Cache(rng, [96, 48], 128, 2, 4, 4)
    out, qr, code = _run_tree(tq, c, q, dtype, [0, 0, 1, 1], [10 ** 6, -4], np.array([[0]] * 3 + [[3]], dtype=np.uint32))
    assert code == tq.TQ_ERR_INVALID_ARG
    see = so.tree_visible([0, 0, 1, 1], [c.cap, 0], np.array([[0]] * 3 + [[3]], dtype=np.uint32), c.cap)
    want, reach = c.oracle(qr, [0, 0, 1, 1], see)
    _close(out, want, reach, dtype, 128)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_infinite_and_nan_norms_in_masked_places(d, dtype):
    tq = _tq()
    rng = np.random.default_rng(d + 1)
    ctx, nodes = [140], [9]
    c = Cache(rng, [149], d, 2, 4, 4)
    q_seq, mask = np.zeros(9, dtype=int), _tree(rng, nodes)
    see = so.tree_visible(q_seq, ctx, mask, c.cap)
    for t, bad in zip([x for x in range(140, 149) if not see[:4, x].any()], [np.nan, np.inf, -np.inf, np.nan, np.inf]):
        raw = np.frombuffer(np.float32(bad).tobytes(), dtype=np.uint8)
        for pg in c.pages:
            pg[c.bt[0, t // 16], t % 16, :, -4:] = raw
    q = rng.standard_normal((4, 8, d)).astype(np.float32)
    out, qr, code = _run_tree(tq, c, q, dtype, q_seq[:4], ctx, mask[:4])
    assert code == tq.TQ_OK
    want, reach = c.oracle(qr, q_seq[:4], see[:4])
    _close(out, want, reach, dtype, d)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_very_large_and_small_norms(dtype):
    # value norms of 1e-3 and 3e5 in one row's set, key norms that make one token win: the
    # output is near that token's value; every weight counts relative to the largest product
    tq = _tq()
    rng = np.random.default_rng(17)
    c = Cache(rng, [300], 128, 2, 4, 4, norm=0.5)
    for t, nu in ((5, 3e5), (130, 2e5), (7, 1e-3), (250, 1e4)):
        c.pages[1][c.bt[0, t // 16], t % 16, :, -4:] = np.frombuffer(np.float32(nu).tobytes(), dtype=np.uint8)
    q = rng.standard_normal((3, 8, 128)).astype(np.float32)
    q_seq, q_len = np.zeros(3, dtype=int), np.array([299, 300, 100])
    qd = torch.from_numpy(q).cuda().to(DT[dtype])
    out = tq.tq_paged_prefill_biased(qd, _i32(q_seq), _i32(q_len), **c.dev(), out_dtype=torch.float32)
    want, reach = c.oracle(qd.float().cpu().numpy(), q_seq, so.biased_visible(q_seq, q_len, c.cap, 1))
    got = out.cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)
    out = tq.tq_paged_prefill_biased(qd, _i32(q_seq), _i32(q_len), **c.dev(), out_dtype=torch.bfloat16)
    got = out.float().cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want)


def test_repeated_calls_and_streams_give_the_same_bytes():
    tq = _tq()
    rng = np.random.default_rng(21)
    lens, rows = [3000, 41, 900], [17, 9, 40]
    c = Cache(rng, lens, 128, 8, 4, 4)
    q_seq, q_len = _random_view(rng, lens, rows)
    q = torch.from_numpy(rng.standard_normal((66, 32, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
    dv, s, n = c.dev(), _i32(q_seq), _i32(q_len)
    first = tq.tq_paged_prefill_biased(q, s, n, **dv)
    for _ in range(3):
        assert torch.equal(first, tq.tq_paged_prefill_biased(q, s, n, **dv))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got.append(tq.tq_paged_prefill_biased(q, s, n, **dv))
    torch.cuda.synchronize()
    assert all(torch.equal(first, g) for g in got)


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
def test_pages_beyond_32_bit_offsets(dtype):
    # 40 million tokens of one head (2.7 GB a component); the rows lie at both ends
    tq = _tq()
    rng = np.random.default_rng(23)
    c = Cache(rng, [200], 128, 1, 4, 4)
    nb = 4_100_000 if dtype == "fp16" else 2_600_000
    shift = nb - c.nb
    half = c.width // 2
    dv = c.dev()
    big = []
    for name in ("k_pages", "v_pages"):
        pg = torch.zeros(nb, 16, 1, dv[name].shape[3], dtype=torch.uint8, device="cuda")
        pg[:c.nb] = dv[name]
        pg[shift:] = dv[name]
        big.append(pg)
    table = dv["block_table"].clone()
    table[:, half:] += shift
    dv.update(k_pages=big[0], v_pages=big[1], block_table=table)
    q = torch.from_numpy(rng.standard_normal((2, 4, 128)).astype(np.float32)).cuda().to(DT[dtype])
    q_seq, q_len = np.zeros(2, dtype=int), np.array([199, 200])
    out = tq.tq_paged_prefill_biased(q, _i32(q_seq), _i32(q_len), **dv)
    want, reach = c.oracle(q.float().cpu().numpy(), q_seq, so.biased_visible(q_seq, q_len, c.cap, 1))
    _close(out, want, reach, dtype, 128)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_codebooks_that_are_not_odd(dtype):
    # the calls take any ascending centroids; the library's own are odd, which the values' expansion uses
    tq = _tq()
    rng = np.random.default_rng(31)
    c = Cache(rng, [200], 128, 4, 4, 4)
    c.vc = np.sort(c.vc + rng.uniform(0.0, 0.01, 16).astype(np.float32)).astype(np.float32)
    c.kc = np.sort(c.kc + rng.uniform(0.0, 0.01, 16).astype(np.float32)).astype(np.float32)
    q = torch.from_numpy(rng.standard_normal((5, 8, 128)).astype(np.float32)).cuda().to(DT[dtype])
    q_seq, q_len = np.zeros(5, dtype=int), np.array([200, 3, 130, 77, 199])
    out = tq.tq_paged_prefill_biased(q, _i32(q_seq), _i32(q_len), **c.dev())
    want, reach = c.oracle(q.float().cpu().numpy(), q_seq, so.biased_visible(q_seq, q_len, c.cap, 1))
    _close(out, want, reach, dtype, 128)


def test_no_rows():
    tq = _tq()
    c = Cache(np.random.default_rng(1), [5], 128, 2, 4, 4)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    out = tq.tq_paged_prefill_biased(torch.empty(0, 8, 128, device="cuda", dtype=torch.float16), e, e, **c.dev(),
                                     status=torch.ones(1, dtype=torch.int32, device="cuda"), check=True)
    assert out.shape == (0, 8, 128)

"""Attention views at the ends of their ranges: weights next to the largest fp16, caps and queries
and norms of any size, blocks that no row sees, lengths beyond the table."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import views as w  # noqa: E402
from oracle import step_oracle as so  # noqa: E402
from oracle import tq_oracle as o  # noqa: E402
from test_gpu_views import Cache  # noqa: E402

pytestmark = pytest.mark.gpu


def _tq():
    import quantized_kv_cache_06_gb300 as tq

    return tq


def _set_norm(c, comp, seq, t, value):
    c.pages[comp][c.bt[seq, t // c.bs], t % c.bs, :, -4:] = np.frombuffer(np.float32(value).tobytes(), dtype=np.uint8)


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weight_times_norm_next_to_the_largest_fp16(dtype):
    # one token of a third tile: its score up to 6 (in powers of two) above everything before it, its
    # value norm a little under 16 times the others', so weight times norm stands at 2^16 times theirs
    # / 2^6.  A kv head per SM, so that one CTA takes a sequence's three tiles in order.
    tq = _tq()
    rng = np.random.default_rng(41)
    h, s, d, n, at = _sms(), 8, 128, 300, 270
    c = Cache(rng, [n] * s, d, h, 4, 4)
    q = torch.from_numpy(rng.standard_normal((s, h, d)).astype(np.float32)).cuda().to(w.DT[dtype])
    rq = q.float().cpu().numpy().astype(np.float64) @ o.rotation_matrix(c.signs).T
    target = np.linspace(5.999, 6.0003, s * h).reshape(s, h)  # log2 of the weight
    for i in range(s):
        blocks, off = c.bt[i, np.arange(n) // 16], np.arange(n) % 16
        c.pages[0][blocks, off, :, -4:] = 0  # key norms: every score 0
        idx = np.where(rq[i] > 0, 15, 0)
        dot = (rq[i] * c.kc[idx]).sum(1) / math.sqrt(d)
        c.pages[0][blocks[at], off[at]] = o.make_rows(idx, (target[i] * math.log(2) / dot).astype(np.float32), 4)
        c.pages[1][blocks, off, :, -4:] = np.frombuffer(np.float32(1.0).tobytes(), dtype=np.uint8)
        _set_norm(c, 1, i, at, 8 * 1.99999)
    dv = c.dev()
    zero = torch.zeros(s, 1, dtype=torch.int32, device="cuda")
    out = tq.tq_paged_tree(q, w.i32(np.arange(s)), w.i32([n] * s), zero, **dv, check=True)
    see = np.zeros((s, c.cap), dtype=bool)
    see[:, :n] = True
    w.close(out, w.exact(q, np.arange(s), see, **dv), dtype)


@pytest.mark.parametrize("cap", [1e-25, 1e-3, 200.0, 300.0, 1e4, 1e6, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_caps_of_any_size(d, dtype, cap):
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [300, 77], d, 2, 4, 4)
    q = torch.from_numpy(rng.standard_normal((5, 8, d)).astype(np.float32)).cuda().to(w.DT[dtype])
    q_seq, q_len = np.array([0, 0, 0, 1, 1]), np.array([298, 299, 300, 1, 77])
    dv = c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, softcap=cap, scale=0.3, check=True)
    see = so.biased_visible(q_seq, q_len, c.cap, 2)
    w.close(out, w.exact(q, q_seq, see, **dv, softcap=float(np.float32(cap)), scale=0.3), dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_blocks_that_no_row_sees_may_be_gone(d, dtype):
    # an engine that frees the blocks behind its window, between a prefix and the window, before the
    # documents or under rejected nodes marks them -1 in the table
    tq = _tq()
    rng = np.random.default_rng(d)
    q = torch.from_numpy(rng.standard_normal((4, 8, d)).astype(np.float32)).cuda().to(w.DT[dtype])
    q_seq, q_len = np.array([0, 0, 1, 2]), np.array([399, 400, 333, 20])
    for kw in (dict(window=70), dict(window=9, prefix=[40, 17, 1]), dict(docs=np.array([300, 310, 200, 3])),
               dict(docs=np.array([300, 310, 20, 3]), prefix=[350, 33, 17])):
        c = Cache(rng, [400, 333, 20], d, 2, 4, 4)
        docs, prefix = kw.get("docs"), kw.get("prefix")
        see = so.biased_visible(q_seq, q_len, c.cap, 3, kw.get("window", 0), prefix, docs)
        gone = 0
        for s in range(3):
            for b in range(c.width):
                if not see[q_seq == s][:, b * 16:b * 16 + 16].any():
                    c.bt[s, b] = [-1, c.nb, 10 ** 9, -2 ** 31][gone % 4]
                    gone += 1
        assert gone > 20
        dv = c.dev()
        out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True, window=kw.get("window", 0),
                                         doc_starts=None if docs is None else w.i32(docs),
                                         prefix_lens=None if prefix is None else w.i32(prefix))
        w.close(out, w.exact(q, q_seq, see, **dv), dtype)
    c = Cache(rng, [80], d, 2, 4, 4)
    c.bt[0, 3] = -1  # nodes 8 .. 23 of a context of 40 tokens
    mask = np.array([[1 << 30, 1], [3, 255], [0x800000FF, 0], [0xFF, 0]], dtype=np.uint32)
    see = so.tree_visible([0] * 4, [40], mask, c.cap)
    dv = c.dev()
    args = (q, w.i32([0] * 4), w.i32([40]), w.i32(mask.view(np.int32)))
    w.close(tq.tq_paged_tree(*args, **dv, check=True), w.exact(q, np.zeros(4, int), see, **dv), dtype)
    # and a seen one is still reported, whatever its entry
    for bad in (-1, c.nb, -2 ** 31):
        dv["block_table"][0, 4] = bad
        with pytest.raises(tq.TQError) as err:
            tq.tq_paged_tree(*args, **dv, check=True)
        assert err.value.status == tq.TQ_ERR_BLOCK_OUT_OF_RANGE
        dv["block_table"][0, 4] = 10 ** 6
        see2 = so.tree_visible([0] * 4, [40], mask, c.cap)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        w.close(tq.tq_paged_tree(*args, **dv, status=status), w.exact(q, np.zeros(4, int), see2, **dv), dtype)
        assert int(status.item()) == tq.TQ_ERR_BLOCK_OUT_OF_RANGE


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_a_long_prompt_beside_many_single_tokens(dtype):
    # many windows a part, of one tile to four: those of the prompt's first rows and of single tokens
    tq = _tq()
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 40, size=255)] + [400]
    c = Cache(rng, lens, 64, 1, 4, 4)
    q_seq = np.concatenate([np.arange(100), np.full(400, 255), np.arange(100, 255)])
    q_len = np.concatenate([lens[:100], np.arange(1, 401), lens[100:255]])
    q = torch.from_numpy(rng.standard_normal((len(q_seq), 4, 64)).astype(np.float32)).cuda().to(w.DT[dtype])
    dv = c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True)
    see = so.biased_visible(q_seq, q_len, c.cap, 256)
    w.close(out, w.exact(q, q_seq, see, **dv), dtype)


@pytest.mark.parametrize("slots", [5, 300])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prompts_in_a_table_of_mostly_idle_rows(dtype, slots):
    tq = _tq()
    rng = np.random.default_rng(4)
    c = Cache(rng, [700, 300, 650], 128, 1, 4, 4)
    c.bt = np.concatenate([c.bt, np.full((slots - 3, c.width), -1, dtype=np.int32)])
    q_seq = np.repeat([2, 0, 1], [400, 500, 300])
    q_len = np.concatenate([np.arange(251, 651), np.arange(201, 701), np.arange(1, 301)])
    q = torch.from_numpy(rng.standard_normal((1200, 2, 128)).astype(np.float32)).cuda().to(w.DT[dtype])
    dv = c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True)
    w.close(out, w.exact(q, q_seq, so.biased_visible(q_seq, q_len, c.cap, slots), **dv), dtype)


@pytest.mark.parametrize("kind", ["plain", "cap", "slopes", "blind"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_of_very_different_sizes_in_a_window(d, dtype, kind):
    # rows beside one with a query 2^40 times theirs, beside a padded one whose query is any bits and
    # which sees nothing, beside one of NaN: each as if it were alone
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [300], d, 2, 4, 4)
    q = torch.from_numpy(rng.standard_normal((7, 8, d)).astype(np.float32)).cuda()
    q_len = np.array([300, 299, 300, 0, 298, 300, 200])
    q[2] *= 0 if kind == "blind" else 2.0 ** 40
    q[3] = 1e37
    q[4] = math.nan if kind != "blind" else 0.5
    q[6] *= 2.0 ** -30
    kw = dict(softcap=20.0) if kind == "cap" else {}
    slopes = torch.from_numpy(rng.uniform(0.0, 0.2, 8).astype(np.float32)).cuda() if kind == "slopes" else None
    q_seq, dv = np.zeros(7, int), c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True, out_dtype=w.DT[dtype],
                                     alibi_slopes=slopes, **kw)
    see = so.biased_visible(q_seq, q_len, c.cap, 1)
    ref = w.exact(q, q_seq, see, **dv, slopes=slopes, q_pos=q_len - 1, **kw)
    for row in (0, 1, 5, 6):
        w.close(out, ref, dtype, rows=[row])
    assert torch.all(out[3] == 0) and bool(torch.isfinite(out[2].float()).all())
    assert kind == "blind" or bool(torch.isnan(out[4].float()).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 256])
def test_queries_whose_square_leaves_fp32(d, dtype):
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [60], d, 2, 4, 4)
    q = torch.from_numpy(rng.standard_normal((2, 8, d)).astype(np.float32)).cuda() * 1e25
    q_seq, dv = np.zeros(2, int), c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32([60, 59]), **dv, check=True, out_dtype=w.DT[dtype])
    see = so.biased_visible(q_seq, [60, 59], c.cap, 1)
    # one token has all the weight where the scores of the first two differ by more than they are off
    want = w.exact(q, q_seq, see, **dv)[0]
    almost = w.exact(q * 1e-25 * 3000, q_seq, see, **dv)[0]
    sure = np.abs(want - almost).max(-1) < 1e-9
    assert sure.sum() >= 4
    err = np.abs(out.float().cpu().numpy() - want)[sure]
    assert np.all(err <= 2.0 ** -7 * np.abs(want[sure]) + 2.0 ** -9 * np.abs(want[sure]).max())


@pytest.mark.parametrize("size", [3e5, 1e7, 1e8, 1e9, 1e12, 1e25, 1e34])
@pytest.mark.parametrize("n", [60, 300])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_of_any_size(d, dtype, n, size):
    # from where fp32 still holds fractions of a score to where its steps pass any weight's exponent;
    # masked tiles and whole ones
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [n], d, 2, 4, 4)
    q = torch.from_numpy(rng.standard_normal((3, 8, d)).astype(np.float32)).cuda()
    q_seq, q_len, dv = np.zeros(3, int), np.array([n, n - 1, n]), c.dev()
    out = tq.tq_paged_prefill_biased(q * size, w.i32(q_seq), w.i32(q_len), **dv, check=True, out_dtype=w.DT[dtype])
    # one token has all the weight where it leads by 30 / 300 of a unit query's scores: far more than the
    # 6 * 2^-11 * 16 / sqrt(3 D) * 2 = 0.014 to 0.007 that roundings to fp16 take from them
    see = so.biased_visible(q_seq, q_len, c.cap, 1)
    want = w.exact(q * size, q_seq, see, **dv)[0]
    sure = np.abs(want - w.exact(q * 300, q_seq, see, **dv)[0]).max(-1) < 1e-9
    assert sure.sum() >= 8
    got = out.float().cpu().numpy().astype(np.float64)[sure]
    size = np.linalg.norm(want[sure], axis=-1, keepdims=True) / math.sqrt(d)
    tol = w.HALF_STEP[dtype] * np.abs(want[sure]) + 6 * 2.0 ** -11 * size + 2.0 ** -11 * np.abs(want[sure])
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want[sure]) <= tol)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("giant", [2.0 ** 25, 1e20, 1e30])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_beside_one_that_sees_a_giant_norm(d, giant, dtype):
    # a drafted node with an enormous value norm that only its own row sees
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [150], d, 2, 4, 4)
    _set_norm(c, 1, 0, 146, giant)
    mask = np.array([[1], [2], [1 << 6], [5], [0]], dtype=np.uint32)
    q = torch.from_numpy(rng.standard_normal((5, 8, d)).astype(np.float32)).cuda()
    q_seq, dv = np.zeros(5, int), c.dev()
    out = tq.tq_paged_tree(q, w.i32(q_seq), w.i32([140]), w.i32(mask.view(np.int32)), **dv, check=True,
                           out_dtype=w.DT[dtype])
    ref = w.exact(q, q_seq, so.tree_visible(q_seq, [140], mask, c.cap), **dv)
    for row in (0, 1, 3, 4):
        w.close(out, ref, dtype, rows=[row])
    if dtype != "fp16":
        w.close(out, ref, dtype, rows=[2])


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("giant", [2.0 ** 25, 1e20, 1e30])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_giant_norm_without_weight(d, giant, dtype):
    # the first token's value norm is enormous and its distance leaves it no weight
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [900], d, 2, 4, 4)
    _set_norm(c, 1, 0, 0, giant)
    q = torch.from_numpy(rng.standard_normal((2, 8, d)).astype(np.float32)).cuda()
    slopes = torch.full((8,), 0.5, device="cuda")
    q_seq, q_len, dv = np.zeros(2, int), np.array([899, 900]), c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True, out_dtype=w.DT[dtype],
                                     alibi_slopes=slopes)
    see = so.biased_visible(q_seq, q_len, c.cap, 1)
    w.close(out, w.exact(q, q_seq, see, **dv, slopes=slopes, q_pos=q_len - 1), dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_lengths_far_beyond_the_table_with_a_distance_bias(dtype):
    # such a length is clamped to the table row, and so is the position that the bias counts from
    tq = _tq()
    rng = np.random.default_rng(8)
    c = Cache(rng, [96, 96], 128, 2, 4, 4)
    q = torch.from_numpy(rng.standard_normal((4, 8, 128)).astype(np.float32)).cuda().to(w.DT[dtype])
    q_seq, q_len, prefix = np.array([0, 0, 1, 1]), np.array([2 ** 30, 96, 2 ** 31 - 1, -2 ** 31]), np.array([5, 60])
    slopes = torch.from_numpy(rng.uniform(0.1, 0.4, 8).astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dv = c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, status=status, alibi_slopes=slopes,
                                     prefix_lens=w.i32(prefix))
    assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
    held = np.clip(q_len, 0, c.cap)
    see = so.biased_visible(q_seq, held, c.cap, 2, prefix_lens=prefix)
    w.close(out, w.exact(q, q_seq, see, **dv, slopes=slopes, q_pos=held - 1), dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("d", [16, 64, 128, 256])
def test_queries_and_outputs_at_any_element(d, dtype):
    # views that start one element behind a 16-byte boundary, and nothing written beside the output
    tq = _tq()
    rng = np.random.default_rng(d)
    c = Cache(rng, [200, 90], d, 2, 4, 4)
    flat = torch.from_numpy(rng.standard_normal(5 * 8 * d + 1).astype(np.float32)).cuda().to(w.DT[dtype])
    q = flat[1:].view(5, 8, d)
    hold = torch.full((5 * 8 * d + 2,), 7.0, device="cuda", dtype=w.DT[dtype])
    q_seq, q_len, dv = np.array([0, 0, 1, 1, 1]), np.array([200, 3, 90, 89, 0]), c.dev()
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, out=hold[1:-1].view(5, 8, d), check=True)
    assert float(hold[0]) == 7 and float(hold[-1]) == 7
    w.close(out, w.exact(q, q_seq, so.biased_visible(q_seq, q_len, c.cap, 2), **dv), dtype)

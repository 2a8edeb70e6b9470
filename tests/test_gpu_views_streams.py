"""The tensor-core attention over many tiles a CTA, against 64 bits: sums and products that go on over
tiles, maxima that move after the first one, copies and barriers that come round again.

Partitions: a kv head is shared by (SMs / kv heads) CTAs, so with many kv heads each of them takes a
long run of tiles; the sizes below give 9 to 60 tiles a CTA.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import views as w  # noqa: E402
from oracle import step_oracle as so  # noqa: E402
from oracle import tq_oracle as o  # noqa: E402

pytestmark = pytest.mark.gpu


def _tq():
    import quantized_kv_cache_06_gb300 as tq

    return tq


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _cache(seed, lens, d, h, kb, vb, bs=16, k_norm=None, v_norm=None):
    """Pages made on the GPU: random indices; norms sqrt(D) lognormal(0.3), or the given [S][n, H]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-n // bs) for n in lens]
    nb = sum(blocks) + 3
    perm = torch.randperm(nb, generator=g, device="cuda")
    table = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device="cuda")
    out = dict(block_table=table, signs=torch.from_numpy(o.splitmix64_signs(d, 42)).float().cuda())
    at = 0
    for s, b in enumerate(blocks):
        table[s, :b] = perm[at:at + b].int()
        at += b
    for name, bits, given in (("k", kb, k_norm), ("v", vb, v_norm)):
        pages = torch.randint(0, 256, (nb, bs, h, d * bits // 8 + 4), generator=g, device="cuda", dtype=torch.uint8)
        for s, n in enumerate(lens):
            t = torch.arange(n, device="cuda")
            nu = math.sqrt(d) * torch.exp(0.3 * torch.randn(n, h, generator=g, device="cuda")) if given is None else \
                given[s].to("cuda", torch.float32)
            rows = pages[table[s].long()[t // bs], t % bs]
            rows[..., -4:] = nu.contiguous().view(torch.uint8).reshape(n, h, 4)
            pages[table[s].long()[t // bs], t % bs] = rows
        out[f"{name}_pages"] = pages
        out[f"{name}_centroids"] = torch.from_numpy(o.codebook_f32(d, bits)[0]).cuda()
    return out


def _queries(seed, rows, hq, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    return torch.randn(rows, hq, d, generator=g, device="cuda").to(w.DT[dtype])


def _last(lens, rows):
    q_seq = np.repeat(np.arange(len(lens)), rows)
    q_len = np.concatenate([np.arange(n - r + 1, n + 1) for n, r in zip(lens, rows)])
    return q_seq, q_len


SHAPES = [
    # d, kb, vb, group, parts, lens, rows: columns of a window in the comment
    (128, 4, 4, 1, 1, [1500, 700], [1, 1]),      # 1: two streams of tiles
    (128, 4, 2, 4, 2, [4000], [3]),              # 12
    (128, 2, 4, 4, 4, [3000, 900], [6, 2]),      # 24 and 8
    (128, 3, 3, 8, 4, [3000], [9]),              # 72: whole width, or two windows (fp16)
    (128, 5, 5, 4, 4, [2500], [15]),             # 60
    (128, 4, 4, 4, 8, [6000], [40]),             # 128 and 32
    (64, 4, 4, 2, 2, [3000, 130], [5, 1]),
    (64, 3, 5, 8, 4, [4000], [16]),
    (64, 5, 2, 1, 1, [2300], [2]),
    (256, 4, 4, 4, 4, [2600], [3]),
    (256, 5, 5, 8, 4, [2000, 400], [7, 2]),
    (256, 2, 3, 1, 1, [1300], [1]),
    (256, 4, 5, 2, 2, [1400], [20]),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_k%dv%d_g%d_parts%d" % s[:5])
def test_long_runs_of_tiles(shape, dtype):
    tq = _tq()
    d, kb, vb, g, parts, lens, rows = shape
    h = _sms() // parts
    dv = _cache(d + kb, lens, d, h, kb, vb)
    q_seq, q_len = _last(lens, rows)
    q = _queries(kb, len(q_seq), h * g, d, dtype)
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True)
    cap = dv["block_table"].shape[1] * 16
    w.close(out, w.exact(q, q_seq, so.biased_visible(q_seq, q_len, cap, len(lens)), **dv), dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_runs_with_caps_masks_and_windows(d, dtype):
    tq = _tq()
    lens, rows, h = [2400, 1100], [10, 4], _sms() // 4
    dv = _cache(d, lens, d, h, 4, 4)
    cap = dv["block_table"].shape[1] * 16
    q_seq, q_len = _last(lens, rows)
    q = _queries(d, 14, 4 * h, d, dtype)
    slopes = torch.tensor([2.0 ** (-8 * (i % 8 + 1) / 8) for i in range(4 * h)], device="cuda")
    docs = np.array([300 + 10 * i for i in range(14)])
    for kw in (dict(softcap=6.0), dict(slopes=slopes), dict(window=900), dict(prefix=[700, 1000], window=300),
               dict(docs=docs, softcap=3.0, slopes=slopes, window=1500, prefix=[900, 2])):
        see = so.biased_visible(q_seq, q_len, cap, 2, kw.get("window", 0), kw.get("prefix"), kw.get("docs"))
        out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True, softcap=kw.get("softcap", 0.0),
                                         window=kw.get("window", 0), alibi_slopes=kw.get("slopes"),
                                         prefix_lens=w.i32(kw["prefix"]) if "prefix" in kw else None,
                                         doc_starts=w.i32(docs) if "docs" in kw else None)
        w.close(out, w.exact(q, q_seq, see, **dv, softcap=kw.get("softcap", 0.0), slopes=kw.get("slopes"),
                             q_pos=q_len - 1), dtype)
    ctx, mask = np.array([2390, 1096]), np.zeros((14, 1), dtype=np.uint32)
    mask[:10, 0] = [1, 3, 5, 9, 19, 35, 67, 135, 263, 519]
    mask[10:, 0] = [1, 2, 7, 15]
    out = tq.tq_paged_tree(q, w.i32(q_seq), w.i32(ctx), w.i32(mask.view(np.int32)), **dv, softcap=9.0, check=True)
    w.close(out, w.exact(q, q_seq, so.tree_visible(q_seq, ctx, mask, cap), **dv, softcap=9.0), dtype)


@pytest.mark.parametrize("slope", [0.05, 0.3, 0.65, 0.7, 1.0, 4.0])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_tile_moves_the_maximum(d, dtype, slope):
    # one CTA a kv head: tile after tile the scores rise, by 2^9 to beyond the largest float
    tq = _tq()
    h, lens, rows = _sms(), [1700], [2]
    dv = _cache(7, lens, d, h, 4, 3)
    q_seq, q_len = _last(lens, rows)
    q = _queries(d, 2, h, d, dtype)
    slopes = torch.full((h,), slope, device="cuda") * torch.linspace(0.5, 1.0, h, device="cuda")
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True, alibi_slopes=slopes)
    see = so.biased_visible(q_seq, q_len, dv["block_table"].shape[1] * 16, 1)
    w.close(out, w.exact(q, q_seq, see, **dv, slopes=slopes, q_pos=q_len - 1), dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("way", ["k_up", "k_down", "k_jump", "v_up", "v_down", "v_jump", "v_zero", "both"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_norms_that_change_along_the_run(d, way, dtype):
    # key norms (scores) and value norms that rise, fall or jump from tile to tile
    tq = _tq()
    h, n = _sms(), 1700
    tile = torch.arange(n) // 128
    g = torch.Generator().manual_seed(d)
    noise = torch.exp(0.2 * torch.randn(n, h, generator=g))
    k = v = torch.ones(n)
    if way in ("k_up", "both"):
        k = 0.3 * tile.float()
    if way == "k_down":
        k = 0.3 * (13 - tile).float()
    if way == "k_jump":
        k = torch.where(tile % 5 == 3, 4.0, 0.2)
    if way in ("v_up", "both"):
        v = 2.0 ** tile.float()
    if way == "v_down":
        v = 2.0 ** -tile.float()
    if way == "v_jump":
        v = torch.where(torch.arange(n) % 389 == 388, 2.0 ** 14, 1.0) * 2.0 ** (tile % 3).float()
    if way == "v_zero":
        v = torch.where(tile < 4, 0.0, 1.0)
    # (fp16 outputs hold up to 65504)
    v = v / v.max() * (100.0 if dtype == "fp16" else 1e6)
    dv = _cache(d, [n], d, h, 4, 4, k_norm=[k[:, None] * math.sqrt(d) * noise], v_norm=[v[:, None] * noise])
    q_seq, q_len = _last([n], [2])
    q = _queries(d, 2, h, d, dtype)
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True)
    see = so.biased_visible(q_seq, q_len, dv["block_table"].shape[1] * 16, 1)
    w.close(out, w.exact(q, q_seq, see, **dv), dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_short_windows_a_cta(d, dtype):
    # windows of one to four tiles one after the other: their queries, sums and outputs change places
    tq = _tq()
    lens = [5, 300, 128, 129, 450, 1, 256, 64, 511, 33]
    rows, h = [1, 9, 3, 30, 2, 1, 70, 12, 5, 33], _sms() // 2
    dv = _cache(d, lens, d, h, 4, 4)
    q_seq, q_len = _last(lens, rows)
    q = _queries(d, len(q_seq), h, d, dtype)
    out = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True)
    see = so.biased_visible(q_seq, q_len, dv["block_table"].shape[1] * 16, len(lens))
    w.close(out, w.exact(q, q_seq, see, **dv), dtype)


@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_agrees_with_the_prefill_in_half_outputs(d, dtype, few):
    # (each lies within its own tolerance of the exact result: the prefill's 2e-3 + 2e-3 |x|, and here
    # half a step of the output beside what 64 bits allow above)
    tq = _tq()
    lens, rows = ([700, 90, 1500, 300], [1, 1, 2, 1]) if few else ([700, 900], [33, 50])
    dv = _cache(d, lens, d, 8, 4, 4)
    q_seq, q_len = _last(lens, rows)
    q = _queries(d, len(q_seq), 32, d, dtype)
    a = tq.tq_paged_prefill_biased(q, w.i32(q_seq), w.i32(q_len), **dv, check=True).float()
    b = tq.tq_paged_prefill(q, w.i32(q_seq), w.i32(q_len), **dv, check=True).float()
    step = 2 * w.HALF_STEP[dtype]
    assert torch.all((a - b).abs() <= 4e-3 + (4e-3 + 2 * step) * b.abs())

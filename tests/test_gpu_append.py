"""tq_norm_rope and tq_append_kv against 64 bits.

Tolerances, per channel.  A row's mean square has at most 13 roundings of 2^-24 (eight squares of
a lane in two chains of four, their three joins, the exchanges of 16 lanes, mean and eps), halved by
the root; rsqrt is off by 2 ulp = 2^-22; two products follow, and in the rotation two more per
channel, relative to the pair's magnitudes.  Together below 2^-20 (|a| + |b|) for the pair (a, b).
Then one rounding to the output's type: half a step, eps / 2 of the value, or half the least
subnormal (2^-25 for fp16).

Packed rows: an index may differ, by one, only where the coordinate lies within 2^-18 of a decision
point: the pairs' errors, summed over D channels with weights 1 / (sqrt(D) nu), are at most 2^-20 2
sqrt(D) nu / (sqrt(D) nu) = 2^-19, the transform adds log2(D) = 8 roundings of 2^-24 of sums below
that bound, and the scale two.  Norms within 2^-18.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import append_oracle as ao  # noqa: E402
from oracle import tq_oracle as o  # noqa: E402

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ROUND = {F32: 2.0 ** -24, F16: 2.0 ** -11, BF16: 2.0 ** -8}
LEAST = {F32: 2.0 ** -149, F16: 2.0 ** -25, BF16: 2.0 ** -133}


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


class Inputs:
    """A projection's output of t tokens, its slices, positions, table and weights."""

    def __init__(self, tq, t, hq, h, d, dtype, rot=None, norm=True, interleaved=False, seed=0, pad=0, rows=3000):
        rng = np.random.default_rng(seed)
        x = rng.standard_normal((t, (hq + 2 * h) * d + pad)) * np.exp(0.5 * rng.standard_normal((1, (hq + 2 * h) * d + pad)))
        self.qkv = torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)
        self.q = self.qkv[:, :hq * d].unflatten(1, (hq, d))
        self.k = self.qkv[:, hq * d:(hq + h) * d].unflatten(1, (h, d))
        self.v = self.qkv[:, (hq + h) * d:(hq + 2 * h) * d].unflatten(1, (h, d))
        self.rot, self.pairs, self.dtype, self.d, self.h, self.t = rot, interleaved, dtype, d, h, t
        self.pos = rng.integers(0, rows, t).astype(np.int32)
        self.table = tq.tq_build_rope(rot, rows).cuda() if rot else None
        w = np.exp(0.3 * rng.standard_normal((2, d))).astype(np.float32)
        self.qw, self.kw = (torch.from_numpy(w[i]).cuda() if norm else None for i in (0, 1))
        self.rng = rng

    def kw_args(self):
        return dict(positions=torch.from_numpy(self.pos).cuda() if self.rot else None, cos_sin=self.table,
                    q_weight=self.qw, k_weight=self.kw, interleaved=self.pairs)

    def want(self, x, w):
        """Rows in fp64 and the size that each channel's rounding is relative to."""
        table = self.table.cpu().numpy() if self.rot else None
        return ao.norm_rope(x.double().cpu().numpy(), np.maximum(self.pos, 0), table, self.pairs,
                            None if w is None else w.cpu().numpy())


def near(got, want, size, dtype):
    off = np.abs(got.double().cpu().numpy() - want)
    tol = ROUND[dtype] * np.abs(want) * (1 + 2.0 ** -10) + LEAST[dtype] + 2.0 ** -20 * size
    assert np.all(off <= tol), float((off / tol).max())


def packed_near(tq, pages, slots, want, signs, cents, bits):
    """Rows at `slots` hold the encoding of want[T, H, D]."""
    t, h, d = want.shape
    got = pages.view(-1, h, pages.shape[3])[slots].reshape(t * h, -1).cpu().numpy()
    idx, norm, margin = ao.encode(want.reshape(t * h, d), signs.cpu().numpy().astype(np.float64), cents.cpu().numpy())
    n = o.index_bytes(d, bits)
    have = o.unpack_indices(got[:, :n], d, bits)
    off = np.abs(have - idx)
    assert np.all((off == 0) | ((off == 1) & (margin <= 2.0 ** -18)))
    nu = np.ascontiguousarray(got[:, n:n + 4]).view("<f4").reshape(-1)
    assert np.all(np.abs(nu.astype(np.float64) - norm) <= 2.0 ** -18 * norm)


def pages_of(tq, x, blocks, bs, kb, vb, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, h = x.d, x.h
    mk = lambda b: torch.randint(0, 256, (blocks, bs, h, tq.tq_row_bytes(d, b)), generator=g, device="cuda",  # noqa: E731
                                 dtype=torch.uint8)
    return (mk(kb), mk(vb), tq.tq_build_rotation(d, 42, "cuda"), tq.tq_codebook(d, kb, "cuda")[0],
            tq.tq_codebook(d, vb, "cuda")[0])


# ---------------------------------------------------------------- dense

@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("t,hq,h,d,rot,norm,pairs", [
    (1, 32, 8, 128, 128, True, False), (37, 16, 2, 128, 128, False, True), (5, 3, 1, 256, 64, True, False),
    (9, 7, 5, 64, 48, True, False), (11, 8, 8, 32, 32, True, True), (13, 5, 3, 16, 16, True, False),
    (6, 4, 4, 16, 6, False, True), (700, 8, 1, 64, 64, True, False), (3, 9, 2, 256, 256, False, False),
    (21, 6, 2, 128, 2, True, False), (8, 6, 2, 128, None, True, False), (17, 4, 2, 128, 96, True, True),
    (19, 4, 2, 256, 250, True, False)])
def test_norm_rope(tq, dtype, t, hq, h, d, rot, norm, pairs):
    x = Inputs(tq, t, hq, h, d, dtype, rot, norm, pairs, seed=t)
    q, k = tq.tq_norm_rope(x.q, x.k, **x.kw_args())
    near(q, *x.want(x.q, x.qw), dtype)
    near(k, *x.want(x.k, x.kw), dtype)


@pytest.mark.parametrize("dtype,pad", [(F32, 1), (F16, 3), (BF16, 1), (BF16, 8), (F32, 4)])
@pytest.mark.parametrize("rot,pairs", [(64, False), (64, True), (32, False), (20, True)])
def test_strides_that_break_vectors_and_in_place(tq, dtype, pad, rot, pairs):
    x = Inputs(tq, 23, 6, 2, 64, dtype, rot, True, pairs, pad=pad)
    want = [x.want(x.q, x.qw), x.want(x.k, x.kw)]
    rest, before = x.qkv[:, 8 * 64:].clone(), x.qkv[:, 10 * 64:].clone()
    q, k = tq.tq_norm_rope(x.q, x.k, **x.kw_args())
    near(q, *want[0], dtype)
    near(k, *want[1], dtype)
    q2, k2 = tq.tq_norm_rope(x.q, x.k, q_out=x.q, k_out=x.k, **x.kw_args())
    assert q2.data_ptr() == x.q.data_ptr() and torch.equal(q2, q) and torch.equal(k2, k)
    assert torch.equal(x.qkv[:, 8 * 64:], rest) and torch.equal(x.qkv[:, 10 * 64:], before)


def test_one_side_only_and_no_tokens(tq):
    x = Inputs(tq, 5, 8, 2, 128, BF16, 128)
    args = x.kw_args()
    q, k = tq.tq_norm_rope(x.q, x.k, **args)
    assert torch.equal(tq.tq_norm_rope(x.q, None, **args)[0], q) and torch.equal(tq.tq_norm_rope(None, x.k, **args)[1], k)
    args["positions"] = args["positions"][:0]
    q, k = tq.tq_norm_rope(x.q[:0], x.k[:0], **args)
    assert q.shape == (0, 8, 128) and k.shape == (0, 2, 128)


def test_padding_offsets_and_positions_beyond_the_table(tq):
    x = Inputs(tq, 40, 6, 2, 128, F16, 128, rows=50)
    pos = torch.from_numpy(x.pos).cuda()
    args = x.kw_args()
    want = tq.tq_norm_rope(x.q, x.k, **args)
    # a step's lengths (positions + 1) with offset -1; length 0 is a padding row
    lens = pos + 1
    lens[::3] = 0
    args.update(positions=lens, position_offset=-1)
    keep = torch.full((40, 6, 128), 7.0, dtype=F16, device="cuda"), torch.full((40, 2, 128), 7.0, dtype=F16, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = tq.tq_norm_rope(x.q, x.k, q_out=keep[0], k_out=keep[1], status=status, check=True, **args)
    for g, w in zip(got, want):
        assert torch.all(g[::3] == 7.0)
        live = torch.ones(40, dtype=torch.bool, device="cuda")
        live[::3] = False
        assert torch.equal(g[live], w[live])
    # a position behind the table, one that passes 2^31, and the lowest
    for bad, offset in ((50, 0), (2 ** 31 - 1, 5)):
        p = pos.clone()
        p[7] = bad
        p[9] = -2 ** 31
        args.update(positions=p, position_offset=offset)
        keep[0].fill_(7.0)
        with pytest.raises(tq.TQError) as e:
            tq.tq_norm_rope(x.q, x.k, q_out=keep[0], check=True, **args)
        assert e.value.status == tq.TQ_ERR_INVALID_ARG and torch.all(keep[0][7] == 7.0) and torch.all(keep[0][9] == 7.0)
        if offset == 0:
            assert torch.equal(keep[0][8], want[0][8]) and torch.equal(keep[0][10:], want[0][10:])


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
@pytest.mark.parametrize("dtype,scale", [(F32, 2.0 ** 80), (F32, 2.0 ** -90), (F32, 2.0 ** -60), (F32, 2.0 ** -30),
                                         (BF16, 2.0 ** 100), (BF16, 2.0 ** -70), (F16, 2.0 ** 9), (F16, 2.0 ** -14)])
def test_norms_of_rows_of_any_scale(tq, dtype, scale, eps, d):
    rng = np.random.default_rng(3)
    x = torch.from_numpy((rng.standard_normal((6, 3, d)) * scale).astype(np.float32)).cuda().to(dtype)
    x[2, 1] = 0
    w = torch.from_numpy(np.exp(rng.standard_normal(d)).astype(np.float32)).cuda()
    got, _ = tq.tq_norm_rope(x, None, q_weight=w, eps=eps)
    with np.errstate(invalid="ignore"):
        want = ao.norm_heads(x.double().cpu().numpy(), w.cpu().numpy(), float(np.float32(eps)))
    if eps == 0.0:  # 0 / 0
        assert not torch.isfinite(got[2, 1]).any()
        got, want = got.clone(), want.copy()
        got[2, 1], want[2, 1] = 0, 0
    near(got, want, np.abs(want), dtype)


def test_rows_that_are_not_finite_stay_their_own(tq):
    x = Inputs(tq, 8, 8, 2, 128, BF16, 128)
    want = tq.tq_norm_rope(x.q, x.k, **x.kw_args())[0]
    x.q[3, 2, 5], x.q[3, 4, 6] = float("nan"), float("inf")
    got = tq.tq_norm_rope(x.q, x.k, **x.kw_args())[0]
    assert torch.isnan(got[3, 2]).all() and not torch.isfinite(got[3, 4]).all()
    same = torch.ones(8, 8, dtype=torch.bool, device="cuda")
    same[3, 2] = same[3, 4] = False
    assert torch.equal(got[same], want[same])


# ---------------------------------------------------------------- packed

@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("t,hq,h,d,rot,norm,pairs,kb,vb", [
    (64, 16, 2, 128, 128, False, False, 4, 4), (33, 32, 8, 128, 128, True, False, 4, 2), (70, 8, 8, 64, 64, False, True, 3, 5),
    (19, 4, 4, 256, 64, True, False, 5, 3), (50, 6, 3, 32, 32, True, True, 2, 5), (41, 5, 5, 16, 16, True, False, 3, 4),
    (40, 4, 1, 16, 8, False, True, 5, 2), (29, 8, 1, 128, 96, True, False, 3, 3), (31, 8, 2, 64, None, True, False, 5, 4),
    (27, 9, 3, 256, 256, True, True, 2, 4)])
def test_append(tq, dtype, t, hq, h, d, rot, norm, pairs, kb, vb):
    x = Inputs(tq, t, hq, h, d, dtype, rot, norm, pairs, seed=7)
    bs = 16
    kp, vp, signs, kc, vc = pages_of(tq, x, -(-t // bs) + 3, bs, kb, vb)
    slots = torch.from_numpy(x.rng.permutation(kp.shape[0] * bs)[:t]).cuda()
    slots[::5] = -1
    before = kp.clone(), vp.clone()
    q = tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, check=True, **x.kw_args())
    assert torch.equal(q, tq.tq_norm_rope(x.q, None, **x.kw_args())[0])
    live = (slots >= 0).cpu().numpy()
    at = slots[slots >= 0]
    packed_near(tq, kp, at, x.want(x.k, x.kw)[0][live], signs, kc, kb)
    packed_near(tq, vp, at, x.v.double().cpu().numpy()[live], signs, vc, vb)
    # every other row is as it was
    for new, old in ((kp, before[0]), (vp, before[1])):
        other = torch.ones(new.shape[0] * bs, dtype=torch.bool, device="cuda")
        other[at] = False
        assert torch.equal(new.view(-1, h, new.shape[3])[other], old.view(-1, h, new.shape[3])[other])


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("d", [16, 64, 128, 256])
def test_values_are_the_writers(tq, dtype, d):
    # rows that need no norm and no rotation: the writer's, but for coordinates at a decision point
    x = Inputs(tq, 90, 2, 3, d, dtype, None, False)
    for bits in (2, 3, 4, 5):
        kp, vp, signs, kc, vc = pages_of(tq, x, 8, 16, bits, bits)
        slots = torch.randperm(128, device="cuda")[:90]
        tq.tq_append_kv(None, x.k, x.v, kp, vp, slots, signs, kc, vc)
        want = torch.zeros_like(kp)
        tq.tq_write_kv(x.k.contiguous(), want, slots, signs, kc)
        rows = [p.view(128, 3, -1)[slots][..., :-4] for p in (kp, want)]  # index bytes
        assert (rows[0] != rows[1]).float().mean() < 1e-3
        packed_near(tq, kp, slots, x.k.double().cpu().numpy(), signs, kc, bits)


@pytest.mark.parametrize("dtype,scale", [(F32, 2.0 ** 110), (F32, 2.0 ** -110), (BF16, 2.0 ** 110), (BF16, 2.0 ** -100)])
def test_rows_of_any_scale_and_rows_that_are_not_finite(tq, dtype, scale):
    x = Inputs(tq, 20, 1, 4, 128, dtype, None, False)
    kp, vp, signs, kc, vc = pages_of(tq, x, 2, 16, 4, 3)
    k = (x.k.double() * scale).to(dtype)
    v = x.v.contiguous()
    k[3, 1] = 0
    v[5, 2, 7], v[6, 3, 0] = float("nan"), float("-inf")
    slots = torch.arange(20, device="cuda")
    tq.tq_append_kv(None, k, v, kp, vp, slots, signs, kc, vc)
    packed_near(tq, kp, slots, k.double().cpu().numpy(), signs, kc, 4)
    zero = kp[3 // 16, 3 % 16, 1]
    for row in (vp[0, 5, 2], vp[0, 6, 3]):
        assert not torch.isfinite(row[-4:].clone().view(F32)).any()
    assert zero[-4:].clone().view(F32).item() == 0.0
    # their indices are the zero row's
    got = vp.view(-1, 4, vp.shape[3])[:20].clone()
    zeros = torch.zeros(1, 16, 4, vp.shape[3], dtype=torch.uint8, device="cuda")
    tq.tq_append_kv(None, None, torch.zeros(1, 4, 128, dtype=dtype, device="cuda"), None, zeros, slots[:1], signs, None, vc)
    assert torch.equal(got[5, 2, :-4], zeros[0, 0, 2, :-4]) and torch.equal(got[6, 3, :-4], zeros[0, 0, 3, :-4])


def test_slots_and_positions_out_of_range(tq):
    x = Inputs(tq, 12, 4, 2, 64, F16, 64, rows=100)
    kp, vp, signs, kc, vc = pages_of(tq, x, 2, 8, 4, 4)
    slots = torch.tensor([0, 1, 16, 3, -1, 5, 1 << 40, 7, 8, 9, 10, -(1 << 50)], device="cuda")
    want_k, want_v = kp.clone(), vp.clone()
    good = torch.tensor([0, 1, 3, 5, 7, 8, 9, 10], device="cuda")
    args = x.kw_args()
    sub = dict(args, positions=args["positions"][good])
    tq.tq_append_kv(x.q[good], x.k[good], x.v[good], want_k, want_v, slots[good], signs, kc, vc, **sub)
    with pytest.raises(tq.TQError) as e:
        tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, check=True, **args)
    assert e.value.status == tq.TQ_ERR_SLOT_OUT_OF_RANGE
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    # a token at a negative position or one behind the table is left out altogether
    p = args["positions"].clone()
    p[1], p[3] = -1, 100
    kp2, vp2 = kp.clone().fill_(9), vp.clone().fill_(9)
    q_out = torch.full_like(x.q.contiguous(), 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.arange(12, device="cuda")
    tq.tq_append_kv(x.q, x.k, x.v, kp2, vp2, slots, signs, kc, vc, q_out=q_out, status=status, **dict(args, positions=p))
    assert int(status.item()) == tq.TQ_ERR_INVALID_ARG
    rows = kp2.view(16, -1), vp2.view(16, -1)
    for i in range(16):
        left = i in (1, 3) or i >= 12
        assert all(bool((r[i] == 9).all()) == left for r in rows)
        if i < 12:
            assert bool((q_out[i] == 5).all()) == left


def test_offsets_beyond_32_bits(tq):
    # pages of more than 4 GiB, and a projection whose last token starts past element 2^31
    d, h, bs = 128, 8, 64
    rb = tq.tq_row_bytes(d, 4)
    blocks = (1 << 32) // (bs * h * rb) + 2
    kp = torch.zeros(blocks, bs, h, rb, dtype=torch.uint8, device="cuda")
    x = Inputs(tq, 3, 1, h, d, BF16, d)
    signs, kc = tq.tq_build_rotation(d, 42, "cuda"), tq.tq_codebook(d, 4, "cuda")[0]
    slots = torch.tensor([0, blocks * bs - 1, blocks * bs - 2], device="cuda")
    tq.tq_append_kv(None, x.k, None, kp, None, slots, signs, kc, None, check=True, **x.kw_args())
    packed_near(tq, kp, slots, x.want(x.k, x.kw)[0], signs, kc, 4)
    assert int((kp.view(-1, h * rb).any(1)).sum()) == 3
    del kp
    rows = torch.empty(3, 3 << 29, dtype=BF16, device="cuda")[:, : h * d].unflatten(1, (h, d))
    rows.copy_(x.k)
    got = tq.tq_norm_rope(None, rows, **x.kw_args())[1]
    assert torch.equal(got, tq.tq_norm_rope(None, x.k, **x.kw_args())[1])


def test_another_stream_and_a_replayed_graph(tq):
    x = Inputs(tq, 48, 8, 2, 128, BF16, 128)
    kp, vp, signs, kc, vc = pages_of(tq, x, 4, 16, 4, 3)
    slots = torch.randperm(64, device="cuda")[:48]
    args = x.kw_args()
    q_out = torch.empty(48, 8, 128, dtype=BF16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def work():
        tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, q_out=q_out, status=status, **args)

    work()
    torch.cuda.synchronize()
    want = q_out.clone(), kp.clone(), vp.clone()
    q_out.zero_(), kp.zero_(), vp.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    at = slots.long()
    live = lambda p: p.view(64, -1)[at]  # noqa: E731
    assert torch.equal(q_out, want[0]) and torch.equal(live(kp), live(want[1])) and torch.equal(live(vp), live(want[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    data = x.qkv.clone()
    for turn in range(3):
        x.qkv.copy_(data.roll(turn, 0))
        q_out.zero_(), kp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = q_out.clone(), live(kp).clone()
        work()
        torch.cuda.synchronize()
        assert torch.equal(q_out, got[0]) and torch.equal(live(kp), got[1])


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [64, 40])
def test_infinities_of_channels_that_stay(tq, rot, pairs):
    # a channel behind the rotated ones stays what it is, and so do the others
    x = Inputs(tq, 4, 3, 1, 128, F32, rot, False, pairs)
    want = tq.tq_norm_rope(x.q, None, **x.kw_args())[0].clone()
    for at in (rot, rot + 1, 127, rot + 16):
        x.q[2, 1, at] = float("inf")
        want[2, 1, at] = float("inf")
    assert torch.equal(tq.tq_norm_rope(x.q, None, **x.kw_args())[0], want)


def test_more_runs_a_token_than_warps(tq):
    # 16384 heads of 256: 8192 groups a token, more runs in a block than the GPU holds warps
    for t in (1, 2, 7):
        x = Inputs(tq, t, 16384, 1, 256, BF16, 256, True, seed=t)
        q, k = tq.tq_norm_rope(x.q, x.k, **x.kw_args())
        for lo in range(0, 16384, 4096):
            near(q[:, lo:lo + 4096], *x.want(x.q[:, lo:lo + 4096], x.qw), BF16)
        near(k, *x.want(x.k, x.kw), BF16)


@pytest.mark.parametrize("t", [1, 3, 4, 5, 150, 1217, 4099])
@pytest.mark.parametrize("hq,h", [(32, 8), (5, 3)])
def test_every_token_whatever_the_cut(tq, t, hq, h):
    # runs of one to eight groups, blocks of one and four tokens, cut off at the last
    x = Inputs(tq, t, hq, h, 64, BF16, 64, True, seed=t)
    kp, vp, signs, kc, vc = pages_of(tq, x, -(-t // 16), 16, 4, 3)
    slots = torch.randperm(kp.shape[0] * 16, device="cuda")[:t]
    q = tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, check=True, **x.kw_args())
    near(q, *x.want(x.q, x.qw), BF16)
    packed_near(tq, kp, slots, x.want(x.k, x.kw)[0], signs, kc, 4)
    packed_near(tq, vp, slots, x.v.double().cpu().numpy(), signs, vc, 3)


def test_refusals_of_the_bindings(tq):
    x = Inputs(tq, 6, 4, 2, 64, F16, 64)
    kp, vp, signs, kc, vc = pages_of(tq, x, 2, 8, 4, 4)
    slots = torch.arange(6, device="cuda")
    rope = x.kw_args()
    for bad in (dict(q=x.q.transpose(1, 2)), dict(q=x.q.float()), dict(k=x.k[:5]), dict(q=x.q[:, ::2]), dict(q_out=x.q[:, :3]),
                dict(positions=rope["positions"].long()), dict(positions=rope["positions"][:5]), dict(positions=None),
                dict(cos_sin=x.table.double()), dict(cos_sin=x.table[:0]), dict(q_weight=x.qw[:63]), dict(k_weight=x.kw.half()),
                dict(k=x.k.cpu()), dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            tq.tq_norm_rope(**{**dict(q=x.q, k=x.k), **rope, **bad})
    args = dict(q=x.q, k=x.k, v=x.v, k_pages=kp, v_pages=vp, slots=slots, signs=signs, k_centroids=kc, v_centroids=vc, **rope)
    for bad in (dict(slots=slots.int()), dict(slots=slots[:5]), dict(signs=signs[:32]), dict(k_pages=kp[..., :-4]), dict(v_pages=vp[:1]),
                dict(k_centroids=kc[:5]), dict(v_centroids=vc.double()), dict(v=x.v[:, :1]), dict(k_pages=None), dict(v_centroids=None),
                dict(k_pages=kp.to(torch.int8)), dict(v=x.v.float())):
        with pytest.raises(ValueError):
            tq.tq_append_kv(**{**args, **bad})
    with pytest.raises(tq.TQError) as e:  # a table wider than the heads
        tq.tq_norm_rope(x.q, x.k, rope["positions"], tq.tq_build_rope(128, 10, device="cuda"))
    assert e.value.status == tq.TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,bits,h", [(BF16, 4, 8), (F16, 2, 8), (BF16, 2, 12), (F16, 4, 4)])
def test_values_of_many_tokens(tq, dtype, bits, h):
    # enough tokens for whole runs of values; among them skipped slots, padding rows, zero rows, rows beyond
    # fp32's squares and rows that are not finite
    t = 5201
    x = Inputs(tq, t, 2 * h, h, 128, dtype, 128, True, seed=h)
    v = x.v.clone()
    v[7::501] = 0
    if dtype is BF16:
        v[8::503] *= 2.0 ** 70
        v[9::505] *= 2.0 ** -80
    x.qkv[:, 3 * h * 128:].unflatten(1, (h, 128)).copy_(v)
    kp, vp, signs, kc, vc = pages_of(tq, x, -(-t // 16) + 1, 16, 4, bits)
    slots = torch.randperm(vp.shape[0] * 16, device="cuda")[:t]
    slots[3::7] = -1
    pos = torch.from_numpy(x.pos).cuda()
    pos[5::97] = -1
    args = dict(x.kw_args(), positions=pos)
    before = vp.clone()
    tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, check=True, **args)
    live = (slots >= 0) & (pos >= 0)
    packed_near(tq, vp, slots[live], x.v[live].double().cpu().numpy(), signs, vc, bits)
    packed_near(tq, kp, slots[live], x.want(x.k, x.kw)[0][live.cpu().numpy()], signs, kc, 4)
    rest = torch.ones(vp.shape[0] * 16, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    assert torch.equal(vp.view(-1, h * vp.shape[3])[rest], before.view(-1, h * vp.shape[3])[rest])
    bad = torch.tensor([100, 5000, 5200], device="cuda")
    unused = torch.ones(vp.shape[0] * 16, dtype=torch.bool, device="cuda")
    unused[slots[slots >= 0]] = False
    slots[bad], pos[bad] = torch.nonzero(unused)[:3, 0], 1
    x.v[100, 1, 9], x.v[5000, h - 1, 100], x.v[5200, 2, 0] = float("nan"), float("inf"), float("-inf")
    tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, **dict(args, positions=pos))
    zeros = torch.zeros(1, 16, h, vp.shape[3], dtype=torch.uint8, device="cuda")
    tq.tq_append_kv(None, None, torch.zeros(1, h, 128, dtype=dtype, device="cuda"), None, zeros, slots[:1] * 0, signs, None, vc)
    rows = vp.view(-1, h, vp.shape[3])
    for i, head in ((100, 1), (5000, h - 1), (5200, 2)):
        row = rows[slots[i], head]
        assert torch.equal(row[:-4], zeros[0, 0, head, :-4]) and not torch.isfinite(row[-4:].clone().view(F32)).any()
        other = x.v[i:i + 1].clone()
        other[0, head] = 0
        got = rows[slots[i]].clone()
        got[head] = zeros[0, 0, head]
        packed_near(tq, got[None, None], torch.zeros(1, dtype=torch.int64, device="cuda"), other.double().cpu().numpy(), signs, vc, bits)

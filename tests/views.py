"""Attention over packed pages in 64 bits on the GPU, and the bounds the tensor-core outputs keep.

`exact` is the definition: softmax over the visible tokens of cap tanh(scale nu_k <Rq, c> / cap)
- slope |pos - t|, times the values nu_v c, rotated back.

Bound.  With weights off by factors e^(+-dx) and rounded once to fp16 (half a step 2^-11),
  |out - exact| <= (2 dx + 2^-11) sum_t p_t |v_t| + 6 * 2^-11 / sqrt(3) sum_t p_t ||v_t|| / sqrt(D)
                   + half a step of the output.
The second term are the centroids, rounded in rotated space: a coordinate of R^T v gathers D of
their errors, each uniform within 2^-11 of a coordinate of about ||v|| / sqrt(D) and divided by
sqrt(D), so sqrt(D) times that in all, six standard deviations; where R^T v is small it is not.
dx is the error of a score: D independent roundings of queries and centroids to fp16, six standard
deviations, on terms of root sum of squares S / sqrt(D) times two (rotated coordinates are near
Gaussian), S the largest |scale| |q| |k| among the row's tokens.
fp32 outputs: D products summed in order, dx = (D + 24) 2^-24 S, and sums of n terms, sqrt(n) 2^-24.
"""

import math

import numpy as np
import torch

from oracle import tq_oracle as o

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).cuda()


def _rows(pages, bits, d, cents):
    """Packed rows [..., RB] -> centroids [..., D] and norms [...], fp64."""
    nb = d * bits // 8
    b = torch.arange(8, device="cuda")
    bit = ((pages[..., :nb, None].to(torch.int32) >> b) & 1).reshape(*pages.shape[:-1], d, bits)
    idx = (bit << torch.arange(bits, device="cuda")).sum(-1)
    norm = pages[..., nb:nb + 4].contiguous().view(torch.float32)[..., 0].double()
    return cents.double()[idx], norm


def exact(q, q_seq, see, k_pages, v_pages, block_table, signs, k_centroids, v_centroids, scale=None, softcap=0.0,
          slopes=None, q_pos=None):
    """q [T, Hq, D] (any type, on the GPU), see [T, cap] bool -> out, sum_t p_t |v_t|, and per
    (row, head) S and sum_t p_t ||v_t||, fp64 on the host.  Rows that see nothing are zero; blocks outside the pages are
    left out."""
    t_rows, hq, d = q.shape
    nb, bs, h, _ = k_pages.shape
    g = hq // h
    kb, vb = (int(math.log2(c.numel())) for c in (k_centroids, v_centroids))
    rot = torch.from_numpy(o.rotation_matrix(signs.cpu().numpy().astype(np.float64))).cuda()
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    q = q.double()
    out, mass = torch.zeros_like(q), torch.zeros_like(q)
    most, size = torch.zeros(2, t_rows, hq, dtype=torch.float64, device="cuda")
    for s in sorted({int(x) for x in q_seq if 0 <= x < block_table.shape[0]}):
        mine = [i for i in range(t_rows) if q_seq[i] == s]
        toks = torch.from_numpy(np.nonzero(see[mine].any(0))[0]).cuda()
        if not len(toks):
            continue
        blk = block_table[s].long()[toks // bs]
        ok = (blk >= 0) & (blk < nb)
        toks, blk = toks[ok], blk[ok]
        kc, kn = _rows(k_pages[blk, toks % bs], kb, d, k_centroids)
        vc, vn = _rows(v_pages[blk, toks % bs], vb, d, v_centroids)
        vis = torch.from_numpy(see[mine]).cuda()[:, toks]
        rq = (q[mine] @ rot.T).reshape(len(mine), h, g, d)
        x = scale * torch.einsum("mhgd,nhd->mhgn", rq, kc) * kn.T[None, :, None, :]
        top = abs(scale) * rq.norm(dim=-1)[..., None] * (kc.norm(dim=-1) * kn).T[None, :, None, :]
        v = vc * vn[..., None]
        m = vis[:, None, None, :]
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        if slopes is not None:
            pos = torch.as_tensor(np.asarray(q_pos)[mine], device="cuda").double()
            x = x - slopes.double().reshape(1, h, g, 1) * (pos[:, None, None, None] - toks).abs()
        x = torch.where(m, x, -math.inf)
        p = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)  # (rows that see nothing)
        out[mine] = (torch.einsum("mhgn,nhd->mhgd", p, v) @ rot).reshape(len(mine), hq, d)
        # |R^T v| of every token, weighted
        mass[mine] = torch.einsum("mhgn,nhd->mhgd", p, (v @ rot).abs()).reshape(len(mine), hq, d)
        size[mine] = torch.einsum("mhgn,nh->mhg", p, v.norm(dim=-1)).reshape(len(mine), hq)
        most[mine] = torch.where(m, top, 0.0).amax(-1).reshape(len(mine), hq)
    return out.cpu().numpy(), mass.cpu().numpy(), most.cpu().numpy(), size.cpu().numpy()


def close(got, ref, dtype, rows=None, tokens=8192):
    """Whether `got` lies within the bound of `exact`'s result, and the whole error within what
    independent roundings leave: 2^-10 of the norm for fp16, 2^-8 for bf16, 1e-5 for fp32, and one
    standard deviation of the scores' error."""
    want, mass, most, size = ref
    got = got.float().cpu().numpy().astype(np.float64)
    if rows is not None:
        got, want, mass, most, size = got[rows], want[rows], mass[rows], most[rows], size[rows]
    d = want.shape[-1]
    if dtype == "fp32":
        dx = (d + 24) * 2.0 ** -24 * most + math.sqrt(tokens) * 2.0 ** -24
        # (values and sums likewise: the centroids are exact, their rotation back rounds log2 D times)
        tol = 2 * dx[..., None] * mass + 16 * 2.0 ** -24 / math.sqrt(d) * 6 * size[..., None]
    else:
        dx = 6 * 2.0 ** -11 / math.sqrt(3) * most / math.sqrt(d) * 2
        tol = (2 * dx[..., None] + 2.0 ** -11) * mass + 6 * 2.0 ** -11 / math.sqrt(3 * d) * size[..., None]
    # (fp16 outputs below its normal range keep half a step of 2^-24)
    tol = tol + HALF_STEP[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "fp16" else 1e-37)
    assert np.all(np.isfinite(got)), np.argwhere(~np.isfinite(got))[:4]
    err = np.abs(got - want)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4])
    norm = {"fp32": 1e-5 + 4 * 2.0 ** -24 * most.max(), "fp16": 2.0 ** -10, "bf16": 2.0 ** -8}[dtype]
    if dtype != "fp32":  # one standard deviation of the scores
        norm += math.sqrt(2) * 2.0 ** -11 / math.sqrt(3) * most.max() / math.sqrt(d)
    assert np.linalg.norm(got - want) <= norm * np.linalg.norm(want) + 1e-12, \
        np.linalg.norm(got - want) / np.linalg.norm(want)

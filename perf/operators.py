"""Operators of a speculative-decoding step over the packed KV cache, and what they are
measured on.

  plan    tq_plan_step              block tables and slot maps from request lengths
  tree    tq_paged_tree             attention of drafted tokens (a tree) over packed pages
  commit  tq_commit_tree            accepted rows moved behind their sequence's context
  biased  tq_paged_prefill_biased   prefill / decode with capped scores, a distance bias, a
                                    sliding window, a bidirectional prefix, documents

Where `own` is false `run` computes the plain forms below (elementary torch, fp32); where it
is true it calls the library.
"""

import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a serving step of 64 running requests, one new token each: the smallest call, where
        # only latency counts
        dict(name="plan_decode_64", op="plan", seqs=64, ctx=8192, new=1, block_size=16, finished=0),
        # a step that admits long prompts beside running and finished requests: ~131072 rows
        dict(name="plan_mixed_1024", op="plan", seqs=1024, ctx=2048, new=256, block_size=16, finished=37),
        # eight requests after the verification of 16 drafted tokens, K4/V2 rows
        dict(name="commit_8", op="commit", seqs=8, ctx=2048, nodes=16, path=4, kv_heads=8, head_dim=128, k_bits=4,
             v_bits=2, block_size=16),
        # a large batch: up to 8 accepted of 64 drafted tokens each
        dict(name="commit_1024", op="commit", seqs=1024, ctx=256, nodes=64, path=8, kv_heads=8, head_dim=128,
             k_bits=4, v_bits=4, block_size=16),
        # the contract example's shapes (16 / 2 heads, 64 fp32 tokens) with 8 drafted tokens
        dict(name="tree_tiny_fp32", op="tree", seqs=1, ctx=64, ragged=False, nodes=8, q_heads=16, kv_heads=2,
             head_dim=128, k_bits=4, v_bits=4, block_size=16, dtype="fp32", softcap=0.0),
        # eight ragged requests, K4/V2, 16 drafted tokens each
        dict(name="tree_ragged_8", op="tree", seqs=8, ctx=2048, ragged=True, nodes=16, q_heads=32, kv_heads=8,
             head_dim=128, k_bits=4, v_bits=2, block_size=16, dtype="fp16", softcap=0.0),
        # the large decode batch with 32 drafted tokens a request
        dict(name="tree_64x8192", op="tree", seqs=64, ctx=8192, ragged=False, nodes=32, q_heads=32, kv_heads=8,
             head_dim=128, k_bits=4, v_bits=4, block_size=16, dtype="bf16", softcap=0.0),
        # long contexts, 8 query heads per kv head, capped scores
        dict(name="tree_4x131072", op="tree", seqs=4, ctx=131072, ragged=False, nodes=12, q_heads=64, kv_heads=8,
             head_dim=128, k_bits=4, v_bits=2, block_size=16, dtype="fp16", softcap=30.0),
        # single tokens of a model with a sliding window and capped scores
        dict(name="biased_decode_64x8192", op="biased", seqs=64, ctx=8192, ragged=False, new=1, window=4096,
             softcap=50.0, alibi=False, prefix=0, docs=0, q_heads=32, kv_heads=8, head_dim=128, k_bits=4, v_bits=4,
             block_size=16, dtype="bf16"),
        # single tokens with a distance bias, 3-bit rows of 64 channels, one query head per kv head
        dict(name="biased_alibi_16x4096", op="biased", seqs=16, ctx=4096, ragged=True, new=1, window=0, softcap=0.0,
             alibi=True, prefix=0, docs=0, q_heads=8, kv_heads=8, head_dim=64, k_bits=3, v_bits=3, block_size=16,
             dtype="fp16"),
        # prompt chunks of packed documents behind a bidirectional prefix
        dict(name="biased_chunk_4x1000", op="biased", seqs=4, ctx=8000, ragged=True, new=1000, window=0, softcap=0.0,
             alibi=False, prefix=200, docs=3, q_heads=32, kv_heads=8, head_dim=128, k_bits=4, v_bits=4,
             block_size=16, dtype="bf16"),
        # wide heads, 5-bit rows, a few rows a sequence, bias and window together
        dict(name="biased_d256_16x4096", op="biased", seqs=16, ctx=4096, ragged=True, new=5, window=1500, softcap=0.0,
             alibi=True, prefix=4, docs=0, q_heads=32, kv_heads=8, head_dim=256, k_bits=5, v_bits=5, block_size=16,
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "commit", "tree", "tree", "biased", "biased"])
    bs = rng.choice([8, 16, 32, 64])
    if op == "plan":
        seqs = _log(rng, 1, 1024)
        return dict(op=op, seqs=seqs, ctx=_log(rng, 16, 8192 if seqs <= 128 else 2048),
                    new=_log(rng, 1, min(2048, 131072 // seqs)), block_size=bs, finished=rng.randrange(0, 1 + seqs // 8))
    heads = rng.choice([(16, 2), (32, 8), (8, 8), (16, 8), (32, 4), (64, 8), (8, 1)])
    common = dict(q_heads=heads[0], kv_heads=heads[1], head_dim=rng.choice([64, 128, 128, 256]),
                  k_bits=rng.choice([2, 3, 4, 4, 5]), v_bits=rng.choice([2, 3, 4, 4, 5]), block_size=bs)
    if op == "commit":
        common.pop("q_heads")
        nodes = _log(rng, 2, 64)
        return dict(op=op, seqs=_log(rng, 1, 1024), ctx=_log(rng, 1, 256), nodes=nodes,
                    path=rng.randrange(1, 1 + min(nodes, 12)), **common)
    common["dtype"] = rng.choice(["bf16", "fp16"])
    ctx = _log(rng, 16, 32768)
    seqs = _log(rng, 1, max(1, min(64, 262144 // ctx)))
    if op == "tree":
        return dict(op=op, seqs=seqs, ctx=ctx, ragged=rng.random() < 0.7, nodes=_log(rng, 1, 64),
                    softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), **common)
    new = rng.choice([1, 1, _log(rng, 2, 64), _log(rng, 2, max(2, min(600, 4000 // seqs)))])
    return dict(op=op, seqs=seqs, ctx=max(ctx, new), ragged=rng.random() < 0.7, new=new,
                window=rng.choice([0, 0, _log(rng, 1, 4096)]), softcap=rng.choice([0.0, 0.0, 30.0]),
                alibi=rng.random() < 0.4, prefix=rng.choice([0, 0, _log(rng, 1, 512)]), docs=rng.choice([0, 0, 3]),
                **common)


def _lengths(case):
    """Lengths of the sequences (tokens before this step) and rows each brings: fixed by the
    case, spread evenly over the range where it is ragged."""
    s = np.arange(case["seqs"])
    spread = ((s + 1) * 0.6180339887498949) % 1.0
    if case["op"] in ("plan", "commit"):
        ctx = 1 + np.floor(spread * case["ctx"]).astype(np.int64)
        return np.minimum(ctx, case["ctx"]), s
    ctx = np.maximum(1, np.floor(spread * case["ctx"])).astype(np.int64) if case["ragged"] else \
        np.full(case["seqs"], case["ctx"], dtype=np.int64)
    if case["op"] == "tree":
        turn = ((s + 1) * 0.7548776662466927) % 1.0
        rows = 1 + np.floor(turn * case["nodes"]).astype(np.int64) if case["ragged"] else \
            np.full(case["seqs"], case["nodes"], dtype=np.int64)
        return ctx, np.minimum(rows, case["nodes"])
    rows = np.minimum(case["new"], ctx)  # biased: ctx counts the new tokens too
    return ctx, rows


def _plan_new(case, ctx):
    """New tokens per sequence (-1: finished): one each, or ragged around `new`."""
    s = np.arange(case["seqs"])
    turn = ((s + 1) * 0.7548776662466927) % 1.0
    new = np.full(case["seqs"], case["new"], dtype=np.int64) if case["new"] == 1 else \
        np.floor(turn * case["new"]).astype(np.int64)
    if case["finished"]:
        new[:: max(1, case["seqs"] // case["finished"])] = -1
    return new


# ---------------------------------------------------------------- inputs

@functools.lru_cache(maxsize=None)
def _codebook(head_dim, bits):
    """Lloyd-Max centroids of one coordinate of a random unit vector (fp64)."""
    n = 1 << 17
    x = (np.arange(n) + 0.5) / n
    f = (1 - x * x) ** ((head_dim - 3) / 2)
    edge = np.arange(n + 1) / n
    m0, m1 = np.concatenate([[0], np.cumsum(f)]), np.concatenate([[0], np.cumsum(f * x)])
    k = 1 << (bits - 1)  # positive half
    c = (np.arange(k) + 0.5) / k * 2.5 / math.sqrt(head_dim)
    for _ in range(20000):
        b = np.concatenate([[0], (c[1:] + c[:-1]) / 2, [1]])
        i0, i1 = np.interp(b, edge, m0), np.interp(b, edge, m1)
        new = np.diff(i1) / np.diff(i0)
        moved = np.abs(new - c).max()
        c = new
        if moved < 1e-13:
            break
    return np.concatenate([-c[::-1], c])


@functools.lru_cache(maxsize=None)
def _signs(head_dim):
    return np.where(np.random.RandomState(42).randint(0, 2, head_dim) > 0, 1.0, -1.0)


def _rotation(head_dim, dtype):
    h = np.ones((1, 1))
    while h.shape[0] < head_dim:
        h = np.block([[h, h], [h, -h]])
    return torch.tensor(h * _signs(head_dim)[None, :] / math.sqrt(head_dim), dtype=dtype, device=DEV)


def _row_bytes(head_dim, bits):
    return head_dim * bits // 8 + 4


def _encode(x, rot, cents, bits):
    """Rows x[n, D] -> packed rows [n, RB]: norm, rotation, nearest centroid, indices LSB first."""
    n, d = x.shape
    nu = x.norm(dim=1, keepdim=True)
    y = (x / nu) @ rot.T
    idx = torch.bucketize(y, (cents[1:] + cents[:-1]) / 2).to(torch.uint8)
    bit = (idx[:, :, None] >> torch.arange(bits, dtype=torch.uint8, device=DEV)) & 1
    byte = (bit.reshape(n, d * bits // 8, 8) << torch.arange(8, dtype=torch.uint8, device=DEV)).sum(2, dtype=torch.uint8)
    return torch.cat([byte, nu.contiguous().view(torch.uint8).reshape(n, 4)], 1)


def _pages(gen, slots, num_blocks, bs, heads, head_dim, bits):
    """Pages whose rows at `slots` hold encoded rows (normal, with a scale per head and
    channel); every other row is stale bytes."""
    rb = _row_bytes(head_dim, bits)
    pages = torch.randint(0, 256, (num_blocks * bs, heads, rb), generator=gen, device=DEV, dtype=torch.uint8)
    rot = _rotation(head_dim, torch.float32)
    cents = torch.tensor(_codebook(head_dim, bits), dtype=torch.float32, device=DEV)
    scale = torch.exp(0.5 * torch.randn(heads, head_dim, generator=gen, device=DEV))
    step = max(1, (1 << 24) // (heads * head_dim))
    for i in range(0, slots.numel(), step):
        at = slots[i:i + step]
        x = torch.randn(at.numel(), heads, head_dim, generator=gen, device=DEV) * scale
        pages[at] = _encode(x.reshape(-1, head_dim), rot, cents, bits).reshape(at.numel(), heads, rb)
    return pages.reshape(num_blocks, bs, heads, rb), cents


def _table(gen, lens, bs, spare=3):
    """A block table over randomly ordered blocks, and the slots of all tokens in order."""
    blocks = -(-lens // bs)
    num, width = int(blocks.sum()) + spare, int(blocks.max())
    perm = torch.randperm(num, generator=gen, device=DEV)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device=DEV)
    col = torch.arange(width, device=DEV)
    cnt = torch.tensor(blocks, device=DEV)
    live = col[None, :] < cnt[:, None]
    table[live] = perm[: int(blocks.sum())].to(torch.int32)
    length = torch.tensor(lens, device=DEV)
    t = torch.arange(width * bs, device=DEV)
    slot = table.long().repeat_interleave(bs, 1) * bs + t % bs
    return table, num, slot[t[None, :] < length[:, None]], slot


def _slopes(heads):
    """The geometric slopes that distance biases use: 2^(-8 i / heads)."""
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / heads) for i in range(heads)], dtype=torch.float32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ctx, rows = _lengths(case)
    bs = case["block_size"]
    i32 = functools.partial(torch.tensor, dtype=torch.int32, device=DEV)
    if case["op"] == "plan":
        new = _plan_new(case, ctx)
        blocks = -(-ctx // bs)
        after = np.where(new < 0, 0, -(-(ctx + np.maximum(new, 0)) // bs))
        width = int(max(after.max(), blocks.max()))
        need = int(np.maximum(0, after - blocks).sum())
        total = int(blocks.sum()) + need + 17
        perm = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros(case["seqs"], width, dtype=torch.int32, device=DEV)
        live = torch.arange(width, device=DEV)[None, :] < torch.tensor(blocks, device=DEV)[:, None]
        used = int(blocks.sum())
        table[live] = perm[:used]
        head = int(torch.randint(0, total, (1,), generator=gen, device=DEV))
        ring = torch.zeros(total, dtype=torch.int32, device=DEV)
        ring[(head + torch.arange(total - used, device=DEV)) % total] = perm[used:]
        max_rows = int(np.maximum(new, 0).sum()) + 5  # the step's row buffers are a little larger
        return dict(case=case, lens=i32(ctx), new=i32(new), blocks=i32(blocks), table=table, ring=ring,
                    free=i32([head, total - used]), bs=bs, max_rows=max_rows)
    if case["op"] == "commit":
        table, num, _, _ = _table(gen, ctx + case["nodes"], bs)
        h, d = case["kv_heads"], case["head_dim"]
        shape = lambda b: (num, bs, h, _row_bytes(d, b))  # noqa: E731
        pages = [torch.randint(0, 256, shape(case[k]), generator=gen, device=DEV, dtype=torch.uint8)
                 for k in ("k_bits", "v_bits")]
        pick = torch.rand(case["seqs"], case["nodes"], generator=gen, device=DEV).argsort(1)[:, :case["path"]]
        path = pick.sort(1).values.to(torch.int32)
        count = torch.randint(0, case["path"] + 1, (case["seqs"],), generator=gen, device=DEV, dtype=torch.int32)
        return dict(case=case, table=table, k=pages[0], v=pages[1], ctx=i32(ctx), path=path, count=count)
    h, hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    total = ctx + rows if case["op"] == "tree" else ctx
    table, num, slots, _ = _table(gen, total, bs)
    k, kc = _pages(gen, slots, num, bs, h, d, case["k_bits"])
    v, vc = _pages(gen, slots, num, bs, h, d, case["v_bits"])
    t = int(rows.sum())
    q = torch.randn(t, hq, d, generator=gen, device=DEV).to(DTYPES[case["dtype"]])
    q_seq = i32(np.repeat(np.arange(case["seqs"]), rows))
    st = dict(case=case, q=q, q_seq=q_seq, k=k, v=v, kc=kc, vc=vc, table=table, scale=1.0 / math.sqrt(d),
              signs=torch.tensor(_signs(d), dtype=torch.float32, device=DEV), rows=rows, bs=bs)
    node = np.concatenate([np.arange(r) for r in rows])
    if case["op"] == "tree":
        # node i of a sequence hangs on an earlier node or on the context; it sees its
        # ancestors and itself
        r = int(rows.max())
        parent = (torch.rand(case["seqs"], r, generator=gen, device=DEV) * torch.arange(r, device=DEV)).long()
        see = torch.zeros(case["seqs"], r, r, dtype=torch.bool, device=DEV)
        for i in range(r):
            if i:
                see[:, i] = see[torch.arange(case["seqs"], device=DEV), parent[:, i]]
            see[:, i, i] = True
        words = -(-r // 32)
        bit = torch.zeros(case["seqs"], r, words * 32, dtype=torch.int64, device=DEV)
        bit[:, :, :r] = see.long()
        word = (bit.reshape(case["seqs"], r, words, 32) << torch.arange(32, device=DEV)).sum(3)
        word = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
        st["mask"] = word[q_seq.long(), torch.tensor(node, device=DEV)].contiguous()
        st["ctx"] = i32(ctx)
        return st
    # biased: the rows are the last tokens of their sequences
    q_len = np.repeat(ctx - rows, rows) + node + 1
    st["q_len"] = i32(q_len)
    st["slopes"] = _slopes(hq) if case["alibi"] else None
    st["prefix"] = i32(np.minimum(case["prefix"], ctx)) if case["prefix"] else None
    st["docs"] = None
    if case["docs"]:  # each sequence holds `docs` documents; a row sees its own
        size = np.repeat(-(-ctx // case["docs"]), rows)
        st["docs"] = i32((q_len - 1) // size * size)
    return st


# ---------------------------------------------------------------- plain forms

def _plain_plan(s):
    lens, new, blocks, bs = s["lens"].long(), s["new"].long(), s["blocks"].long(), s["bs"]
    table, ring, total = s["table"], s["ring"], s["ring"].numel()
    head, count = s["free"][0].long(), s["free"][1].long()
    gone = new < 0
    add = new.clamp(min=0)
    need = torch.where(gone, 0, ((lens + add + bs - 1) // bs - blocks).clamp(min=0))
    base = need.cumsum(0) - need
    ends = add.cumsum(0)
    col = torch.arange(table.shape[1], device=DEV)
    j = col[None, :] - blocks[:, None]
    fresh = (j >= 0) & (j < need[:, None])
    out = torch.where(fresh, ring[(head + base[:, None] + j) % total], table)
    r = torch.arange(s["max_rows"], device=DEV)
    live = r < ends[-1]
    q = torch.searchsorted(ends, r, right=True).clamp(max=lens.numel() - 1)
    t = lens[q] + r - (ends - add)[q]
    slot = out.reshape(-1)[(q * table.shape[1] + t // bs).clamp(max=table.numel() - 1)].long() * bs + t % bs
    back = torch.where(gone, blocks, 0)
    place = (head + count + (back.cumsum(0) - back)[:, None] + col[None, :]) % total
    place = torch.where(col[None, :] < back[:, None], place, total)
    ring2 = torch.cat([ring, ring[:1]])
    ring2[place.reshape(-1)] = table.reshape(-1)
    free = torch.stack([(head + need.sum()) % total, count - need.sum() + back.sum()])
    i32 = torch.int32
    return dict(slots=torch.where(live, slot, -1), q_seq=torch.where(live, q, -1).to(i32),
                q_len=torch.where(live, t + 1, 0).to(i32), row_start=torch.cat([ends[:1] * 0, ends]).to(i32),
                seq_lens=torch.where(gone, 0, lens + add).to(i32),
                seq_blocks=torch.where(gone, 0, blocks + need).to(i32), free=free.to(i32), table=out,
                ring=ring2[:total])


def _plain_commit(s):
    ctx, path, count, bs = s["ctx"].long(), s["path"].long(), s["count"].long(), s["case"]["block_size"]
    j = torch.arange(path.shape[1], device=DEV)[None, :]
    to = ctx[:, None] + j
    frm = torch.where(j < count[:, None], ctx[:, None] + path, to)

    def slot(t):
        return torch.gather(s["table"].long(), 1, t // bs) * bs + t % bs

    a, b = slot(frm).reshape(-1), slot(to).reshape(-1)
    for pages in (s["k"], s["v"]):
        flat = pages.view(-1, pages.shape[2] * pages.shape[3])
        flat[b] = flat[a]
    return dict(k=s["k"], v=s["v"], seq_lens=(ctx + count).to(torch.int32))


def _plain_rows(pages, table, cents, bits, head_dim):
    """Rows of all table entries in rotated space: nu c[idx], fp32 [S, tokens, H, D]."""
    got = pages[table.long()].flatten(1, 2)
    j = torch.arange(head_dim, device=DEV) * bits
    wide = got[..., :-4].to(torch.int16)
    wide = wide | (torch.cat([wide[..., 1:], wide[..., :1] * 0], -1) << 8)
    idx = (wide[..., j // 8] >> (j % 8).to(torch.int16)) & ((1 << bits) - 1)
    nu = got[..., -4:].contiguous().view(torch.float32)
    return cents[idx.int()], nu.squeeze(-1)


def _plain_attention(s):
    case = s["case"]
    h, hq, d = case["kv_heads"], case["q_heads"], case["head_dim"]
    g, n, t = hq // h, case["seqs"], s["q"].shape[0]
    most = int(s["rows"].max())
    starts = torch.tensor(np.cumsum(s["rows"]) - s["rows"], device=DEV)
    seq = s["q_seq"].long()
    at = seq * most + torch.arange(t, device=DEV) - starts[seq]  # the row's place in [n, most]

    def spread(x):
        y = torch.zeros((n * most,) + x.shape[1:], dtype=x.dtype, device=DEV)
        y[at] = x
        return y.reshape((n, most) + x.shape[1:])

    rot = _rotation(d, torch.float32)
    q = spread(s["q"].float() @ rot.T).reshape(n, most, h, g, d).permute(0, 2, 1, 3, 4).reshape(n, h, most * g, d)
    c, nu = _plain_rows(s["k"], s["table"], s["kc"], case["k_bits"], d)
    tokens = c.shape[1]
    x = q @ c.permute(0, 2, 3, 1)
    del c
    x *= (nu * s["scale"]).permute(0, 2, 1)[:, :, None, :]
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    x = x.reshape(n, h, most, g, tokens)
    pos = torch.arange(tokens, device=DEV)
    if case["op"] == "tree":
        ctx = s["ctx"].long()[:, None, None]
        j = (pos - ctx).clamp(min=0)
        word = spread(s["mask"])
        words = word.shape[2]
        hit = torch.gather(word, 2, (j // 32).clamp(max=words - 1).expand(n, most, tokens)) >> (j % 32).int()
        see = (pos < ctx) | ((hit & 1).bool() & (pos - ctx < 32 * words))
        see &= spread(torch.ones(t, dtype=torch.bool, device=DEV))[:, :, None]
    else:
        length = spread(s["q_len"]).long()[:, :, None]
        see = pos < length
        if case["window"]:
            see &= pos >= length - case["window"]
        if s["prefix"] is not None:
            see |= pos < s["prefix"].long()[:, None, None]
        if s["docs"] is not None:
            see &= pos >= spread(s["docs"]).long()[:, :, None]
        if case["alibi"]:
            x -= s["slopes"].reshape(1, h, 1, g, 1) * (pos - (length - 1)).abs().float()[:, None, :, None, :]
    x = x.masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    c, nu = _plain_rows(s["v"], s["table"], s["vc"], case["v_bits"], d)
    nu = torch.where(see.any(1)[:, :, None], nu, 0.0)  # stale rows hold any bytes
    o = x.reshape(n, h, most * g, tokens) @ (c * nu[..., None]).permute(0, 2, 1, 3)
    o = o.reshape(n, h, most, g, d) / torch.where(total > 0, total, 1.0)
    o = (o @ rot).permute(0, 2, 1, 3, 4).reshape(n * most, hq, d)
    return o[at].to(s["q"].dtype)


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        import quantized_kv_cache_06_gb300 as tq

        if case["op"] == "plan":
            p = tq.tq_plan_step(s["lens"], s["new"], s["blocks"], s["table"], s["ring"], s["free"], s["bs"],
                                s["max_rows"])
            return dict(slots=p.slots, q_seq=p.q_seq, q_len=p.q_len, row_start=p.row_start, seq_lens=p.seq_lens,
                        seq_blocks=p.seq_blocks, free=p.free_state, table=s["table"], ring=s["ring"])
        if case["op"] == "commit":
            lens = tq.tq_commit_tree(s["k"], s["v"], s["table"], s["ctx"], s["path"], s["count"])
            return dict(k=s["k"], v=s["v"], seq_lens=lens)
        if case["op"] == "tree":
            return tq.tq_paged_tree(s["q"], s["q_seq"], s["ctx"], s["mask"], s["k"], s["v"], s["table"], s["signs"],
                                    s["kc"], s["vc"], scale=s["scale"], softcap=case["softcap"])
        return tq.tq_paged_prefill_biased(s["q"], s["q_seq"], s["q_len"], s["k"], s["v"], s["table"], s["signs"],
                                          s["kc"], s["vc"], scale=s["scale"], softcap=case["softcap"],
                                          window=case["window"], alibi_slopes=s["slopes"], prefix_lens=s["prefix"],
                                          doc_starts=s["docs"])
    if case["op"] == "plan":
        return _plain_plan(s)
    if case["op"] == "commit":
        return _plain_commit(s)
    return _plain_attention(s)


# ---------------------------------------------------------------- what a pass cannot do without

def _seen(case):
    """Per sequence: the tokens some row sees, and the (row, token) pairs."""
    ctx, rows = _lengths(case)
    tokens = pairs = 0.0
    for n, r in zip(ctx, rows):
        n, r = int(n), int(r)
        if case["op"] == "tree":  # on average a node of a random tree has ln(r) ancestors
            tokens += n + r
            pairs += r * (n + 1 + math.log(max(1, r)))
            continue
        length = np.arange(n - r + 1, n + 1)
        pre = min(case["prefix"], n)
        lo = np.maximum(0, length - case["window"]) if case["window"] else np.zeros(r, dtype=np.int64)
        doc = np.zeros(r, dtype=np.int64)
        if case["docs"]:
            size = -(-n // case["docs"])
            doc = (length - 1) // size * size
        # two intervals, [doc, pre) and [max(lo, doc), length); their union, with the overlap once
        a, b = doc, np.maximum(doc, pre)
        c, e = np.maximum(lo, doc), length
        pairs += float((b - a + np.maximum(0, e - np.maximum(c, b))).sum())
        hit = np.zeros(n + 1, dtype=np.int64)
        np.add.at(hit, a, 1)
        np.add.at(hit, b, -1)
        np.add.at(hit, np.minimum(c, e), 1)
        np.add.at(hit, e, -1)
        tokens += float((np.cumsum(hit)[:n] > 0).sum())
    return tokens, pairs


def work(case):
    ctx, rows = _lengths(case)
    s = case["seqs"]
    if case["op"] == "plan":
        new = _plan_new(case, ctx)
        bs = case["block_size"]
        blocks = -(-ctx // bs)
        need = np.where(new < 0, 0, np.maximum(0, -(-(ctx + np.maximum(new, 0)) // bs) - blocks)).sum()
        back = np.where(new < 0, blocks, 0).sum()
        total = int(np.maximum(new, 0).sum()) + 5
        # per row slot, sequence and length; per sequence three lengths in, three out; each
        # new or returned block read and written once
        return dict(bytes=float(total * 16 + s * 24 + (need + back) * 8 + 16), flops=0.0)
    if case["op"] == "commit":
        moved = s * case["path"] / 2
        row = case["kv_heads"] * sum(_row_bytes(case["head_dim"], case[k]) for k in ("k_bits", "v_bits"))
        return dict(bytes=2.0 * moved * row + s * (case["path"] * 4 + 12), flops=0.0)
    tokens, pairs = _seen(case)
    row = case["kv_heads"] * sum(_row_bytes(case["head_dim"], case[k]) for k in ("k_bits", "v_bits"))
    size = 4 if case["dtype"] == "fp32" else 2
    t = int(rows.sum())
    return dict(bytes=float(tokens * row + 2 * t * case["q_heads"] * case["head_dim"] * size + tokens / case["block_size"] * 4),
                flops=float(4 * pairs * case["q_heads"] * case["head_dim"]))


# ---------------------------------------------------------------- 64 bits

def _exact_rows(pages, slots, cents, bits, head_dim):
    """Dense rows nu R^T c[idx] at `slots`, fp64 [H, tokens, D]."""
    got = pages.view(-1, pages.shape[2], pages.shape[3])[slots].transpose(0, 1).contiguous()
    h, n, _ = got.shape
    bit = (got[..., :-4, None] >> torch.arange(8, dtype=torch.uint8, device=DEV)) & 1
    bit = bit.reshape(h, n, head_dim, bits)
    idx = torch.zeros(h, n, head_dim, dtype=torch.int32, device=DEV)
    for i in range(bits):
        idx += bit[..., i].int() << i
    nu = got[..., -4:].contiguous().view(torch.float32).double()
    return (cents.double()[idx] @ _rotation(head_dim, torch.float64)) * nu


def exact(case, seed):
    if case["op"] in ("plan", "commit"):
        return None  # whole numbers, which have to be equal
    s = prepare(case, seed)
    ctx, rows = _lengths(case)
    h, hq, d, bs = case["kv_heads"], case["q_heads"], case["head_dim"], case["block_size"]
    g = hq // h
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    first = 0
    for b in range(case["seqs"]):
        r = int(rows[b])
        tokens = int(ctx[b]) + (r if case["op"] == "tree" else 0)
        mine = slice(first, first + r)
        first += r
        pos = torch.arange(tokens, device=DEV)
        slots = s["table"][b].long()[pos // bs] * bs + pos % bs
        k = _exact_rows(s["k"], slots, s["kc"], case["k_bits"], d)
        v = _exact_rows(s["v"], slots, s["vc"], case["v_bits"], d)
        q = s["q"][mine].double().reshape(r, h, g, d)
        see = torch.zeros(r, tokens, dtype=torch.bool, device=DEV)
        dist = None
        for i in range(r):
            if case["op"] == "tree":
                see[i, :int(ctx[b])] = True
                w = s["mask"][first - r + i].tolist()
                for j in range(r):
                    see[i, int(ctx[b]) + j] = bool((w[j // 32] >> (j % 32)) & 1)
                continue
            if i == 0:
                length = [int(x) for x in s["q_len"][mine]]
                start = [int(x) for x in s["docs"][mine]] if s["docs"] is not None else [0] * r
            lo = max(0, length[i] - case["window"]) if case["window"] else 0
            see[i, lo:length[i]] = True
            see[i, :min(case["prefix"], int(ctx[b]))] = True
            see[i, :start[i]] = False
        if case["op"] == "biased":
            dist = (pos[None, :] - (torch.tensor(length, device=DEV)[:, None] - 1)).abs().double()
        step = max(1, (1 << 28) // max(1, tokens * r))
        for j in range(0, hq, step):  # query heads at a time
            for c in range(j, min(hq, j + step)):
                x = (q[:, c // g, c % g] @ k[c // g].T) / math.sqrt(d)
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if case["op"] == "biased" and case["alibi"]:
                    x = x - float(s["slopes"][c]) * dist
                x = torch.where(see, x, -math.inf)
                p = torch.softmax(x, 1)
                p = torch.where(see.any(1, keepdim=True), p, 0.0)
                out[mine, c] = p @ v[c // g]
    return out

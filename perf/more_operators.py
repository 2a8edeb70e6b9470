"""Operators around a serving step's attention, and what they are measured on.

  rope    tq_norm_rope     norms of each query and key head and the position rotation, one pass
  append  tq_append_kv     the same on the way into the packed pages: queries out, K and V rows
                           encoded at their slots (read back dense, as the values they stand for)
  verify  tq_verify_tree   drafted tokens against the target's probabilities from given random
                           numbers: the accepted path and the next token

Where `own` is false `run` computes the plain forms below (elementary torch, fp32; the
distributions that tokens are drawn from in fp64); where it is true it calls the library.
"""

import functools
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
POSITIONS = 131072  # rows of the cos / sin table: the longest context of the benchmark's workloads
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one new token of 64 running requests: the smallest call, where only latency counts
        dict(name="rope_decode_64", op="rope", tokens=64, seqs=64, q_heads=32, kv_heads=8, head_dim=128, rot=128,
             style="half", norm=True, dtype="bf16"),
        # wide heads of which a part rotates, pairs of neighbours, ragged prompt chunks
        dict(name="rope_partial_1000", op="rope", tokens=1000, seqs=7, q_heads=16, kv_heads=8, head_dim=256, rot=64,
             style="pairs", norm=False, dtype="fp16"),
        # a long prompt
        dict(name="rope_prompt_32768", op="rope", tokens=32768, seqs=4, q_heads=32, kv_heads=8, head_dim=128, rot=128,
             style="half", norm=True, dtype="bf16"),
        # the contract example's shapes: 64 fp32 tokens, 16 / 2 heads
        dict(name="append_tiny_fp32", op="append", tokens=64, seqs=1, q_heads=16, kv_heads=2, head_dim=128, rot=128,
             style="half", norm=False, dtype="fp32", k_bits=4, v_bits=4, block_size=16, skipped=0.0),
        # single tokens of 64 requests into the large decode batch's pages
        dict(name="append_decode_64", op="append", tokens=64, seqs=64, q_heads=32, kv_heads=8, head_dim=128, rot=128,
             style="half", norm=True, dtype="bf16", k_bits=4, v_bits=4, block_size=16, skipped=0.0),
        # eight ragged prompts, K4/V2, a tenth of the slots skipped
        dict(name="append_ragged_8", op="append", tokens=8200, seqs=8, q_heads=32, kv_heads=8, head_dim=128, rot=64,
             style="half", norm=True, dtype="fp16", k_bits=4, v_bits=2, block_size=16, skipped=0.1),
        # narrow heads whose rows cross byte borders, pairs of neighbours
        dict(name="append_d64_k3v5", op="append", tokens=16001, seqs=16, q_heads=32, kv_heads=8, head_dim=64, rot=64,
             style="pairs", norm=False, dtype="bf16", k_bits=3, v_bits=5, block_size=16, skipped=0.0),
        # a bulk prompt write
        dict(name="append_prompt_32768", op="append", tokens=32768, seqs=4, q_heads=32, kv_heads=8, head_dim=128,
             rot=128, style="half", norm=True, dtype="bf16", k_bits=4, v_bits=4, block_size=16, skipped=0.05),
        # one request, four drafted tokens with the drafter's probabilities
        dict(name="verify_chain_1", op="verify", seqs=1, nodes=5, ragged=False, tree=False, draft=True, vocab=32768,
             dtype="bf16", greedy=0.0),
        # eight ragged requests, drafted trees without probabilities, a vocabulary of odd size
        dict(name="verify_tree_8", op="verify", seqs=8, nodes=16, ragged=True, tree=True, draft=False, vocab=50001,
             dtype="fp32", greedy=0.0),
        # a batch of drafted chains with the drafter's probabilities
        dict(name="verify_chain_64", op="verify", seqs=64, nodes=5, ragged=False, tree=False, draft=True, vocab=131072,
             dtype="bf16", greedy=0.0),
        # the largest: trees of a big batch, every fourth request greedy
        dict(name="verify_tree_256", op="verify", seqs=256, nodes=8, ragged=True, tree=True, draft=False, vocab=131072,
             dtype="bf16", greedy=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "verify", "verify"])
    if op == "verify":
        vocab = _log(rng, 1000, 140000)
        nodes = _log(rng, 1, 48)
        draft = nodes > 1 and rng.random() < 0.5
        rows = min(4096, 150000000 // vocab)
        return dict(op=op, seqs=_log(rng, 1, max(1, min(512, rows // nodes))), nodes=nodes, ragged=rng.random() < 0.6,
                    tree=not draft and rng.random() < 0.7, draft=draft, vocab=vocab,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), greedy=rng.choice([0.0, 0.0, 0.3]))
    heads = rng.choice([(16, 2), (32, 8), (8, 8), (16, 8), (32, 4), (64, 8), (8, 1), (5, 5)])
    d = rng.choice([64, 128, 128, 256])
    tokens = _log(rng, 1, min(32768, 32768 * 48 * 128 // ((heads[0] + 2 * heads[1]) * d)))
    case = dict(op=op, tokens=tokens, seqs=_log(rng, 1, min(64, tokens)), q_heads=heads[0], kv_heads=heads[1],
                head_dim=d, rot=rng.choice([d, d, d // 2, 3 * d // 4]), style=rng.choice(["half", "half", "pairs"]),
                norm=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "append":
        if case["dtype"] == "fp32":
            case["tokens"] = 1 + case["tokens"] // 2
            case["seqs"] = min(case["seqs"], case["tokens"])
        case.update(k_bits=rng.choice([2, 3, 4, 4, 5]), v_bits=rng.choice([2, 3, 4, 4, 5]),
                    block_size=rng.choice([8, 16, 32, 64]), skipped=rng.choice([0.0, 0.0, 0.1]))
    elif case["dtype"] == "fp32":
        case["tokens"] = 1 + case["tokens"] // 2
        case["seqs"] = min(case["seqs"], case["tokens"])
    return case


# ---------------------------------------------------------------- inputs

@functools.lru_cache(maxsize=None)
def _codebook(head_dim, bits):
    """Lloyd-Max centroids of one coordinate of a random unit vector (fp64)."""
    n = 1 << 16
    x = (np.arange(n) + 0.5) / n
    f = (1 - x * x) ** ((head_dim - 3) / 2)
    edge = np.arange(n + 1) / n
    m0, m1 = np.concatenate([[0], np.cumsum(f)]), np.concatenate([[0], np.cumsum(f * x)])
    k = 1 << (bits - 1)  # positive half
    c = (np.arange(k) + 0.5) / k * 2.5 / math.sqrt(head_dim)
    for _ in range(4000):
        b = np.concatenate([[0], (c[1:] + c[:-1]) / 2, [1]])
        i0, i1 = np.interp(b, edge, m0), np.interp(b, edge, m1)
        new = np.diff(i1) / np.diff(i0)
        moved = np.abs(new - c).max()
        c = new
        if moved < 1e-11:
            break
    return np.concatenate([-c[::-1], c])


@functools.lru_cache(maxsize=None)
def _signs(head_dim):
    return np.where(np.random.RandomState(42).randint(0, 2, head_dim) > 0, 1.0, -1.0)


@functools.lru_cache(maxsize=None)
def _rotation(head_dim, dtype):
    h = np.ones((1, 1))
    while h.shape[0] < head_dim:
        h = np.block([[h, h], [h, -h]])
    return torch.tensor(h * _signs(head_dim)[None, :] / math.sqrt(head_dim), dtype=dtype, device=DEV)


@functools.lru_cache(maxsize=4)
def _table(rot):
    """cos and sin of position * 10000^(-2 i / rot), angles in fp64, fp32 [POSITIONS, rot]."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = torch.arange(POSITIONS, dtype=torch.float64, device=DEV)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _row_bytes(head_dim, bits):
    return head_dim * bits // 8 + 4


def _shares(total, parts):
    """`total` cut into `parts` uneven positive numbers."""
    spread = 0.25 + ((np.arange(parts) + 1) * 0.6180339887498949) % 1.0
    cut = np.floor(np.cumsum(spread) / spread.sum() * (total - parts)).astype(np.int64)
    return np.diff(np.concatenate([[0], cut])) + 1


def _prepare_tokens(case, gen):
    t, hq, h, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    i32 = functools.partial(torch.tensor, dtype=torch.int32, device=DEV)
    # the projection's output: queries, keys and values of a token side by side
    scale = torch.exp(0.5 * torch.randn((hq + 2 * h) * d, generator=gen, device=DEV))
    qkv = torch.randn(t, (hq + 2 * h) * d, generator=gen, device=DEV).mul_(scale).to(DTYPES[case["dtype"]])
    lens = _shares(t, case["seqs"])
    # tokens already cached before these: anywhere in the context
    room = POSITIONS - lens
    ctx = np.floor(((np.arange(case["seqs"]) + 1) * 0.7548776662466927) % 1.0 * room).astype(np.int64)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, lens)])
    s = dict(case=case, qkv=qkv, q=qkv[:, :hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + h) * d].view(t, h, d),
             v=qkv[:, (hq + h) * d:].view(t, h, d), pos=i32(pos), table=_table(case["rot"]), qw=None, kw=None)
    if case["norm"]:
        s["qw"] = torch.exp(0.3 * torch.randn(d, generator=gen, device=DEV))
        s["kw"] = torch.exp(0.3 * torch.randn(d, generator=gen, device=DEV))
    if case["op"] == "append":
        bs = case["block_size"]
        blocks = -(-t // bs) + 5
        s["kc"], s["vc"] = (torch.tensor(_codebook(d, case[b]), dtype=torch.float32, device=DEV)
                            for b in ("k_bits", "v_bits"))
        s["kp"], s["vp"] = (torch.zeros(blocks, bs, h, _row_bytes(d, case[b]), dtype=torch.uint8, device=DEV)
                            for b in ("k_bits", "v_bits"))
        perm = torch.randperm(blocks, generator=gen, device=DEV)
        at = torch.arange(t, device=DEV)
        slots = perm[at // bs] * bs + at % bs
        skip = torch.rand(t, generator=gen, device=DEV) < case["skipped"]
        s["slots"] = torch.where(skip, -1, slots)
        s["signs"] = torch.tensor(_signs(d), dtype=torch.float32, device=DEV)
    return s


def _rows(case):
    """Rows (the root and its drafted nodes) of every request."""
    n = np.full(case["seqs"], case["nodes"], dtype=np.int64)
    if case["ragged"]:
        turn = ((np.arange(case["seqs"]) + 1) * 0.7548776662466927) % 1.0
        n = np.minimum(1 + np.floor(turn * case["nodes"]).astype(np.int64), case["nodes"])
    return n


def _prepare_verify(case, gen):
    i32 = functools.partial(torch.tensor, dtype=torch.int32, device=DEV)
    rows, v = _rows(case), case["vocab"]
    start = np.concatenate([[0], np.cumsum(rows)])
    t = int(start[-1])
    node = np.concatenate([np.arange(r) for r in rows])
    seq = np.repeat(np.arange(case["seqs"]), rows)
    parent = node - 1
    if case["tree"]:  # three children a node, in breadth-first order
        parent = (node + 2) // 3 - 1
    up = torch.tensor(start[seq] + np.maximum(parent, 0), device=DEV)
    # a language model's logits: a broad bulk, a few likely tokens, some tokens that are never allowed
    logits = torch.randn(t, v, generator=gen, device=DEV).mul_(1.8)
    likely = torch.randint(0, v, (t, 12), generator=gen, device=DEV)
    boost = torch.randn(t, 12, generator=gen, device=DEV).mul_(1.5).add_(9.0 + math.log(v / 50000.0))
    logits.scatter_(1, likely, boost)
    logits[:, v - v // 50:] = -math.inf
    s = dict(case=case, start=i32(start), seq=torch.tensor(seq, device=DEV), up=up, rows=rows,
             node=torch.tensor(node, device=DEV), parents=i32(parent), draft=None, ua=None)
    temp = torch.rand(case["seqs"], generator=gen, device=DEV) * 0.6 + 0.6
    greedy = (np.arange(case["seqs"]) + 1) * 0.6180339887498949 % 1.0 < case["greedy"]
    s["temp"] = torch.where(torch.tensor(greedy, device=DEV), 0.0, temp)
    if case["draft"]:
        # a drafter that is near the target, and tokens drawn from it
        near = logits + 0.7 * torch.randn(t, v, generator=gen, device=DEV)
        draft = torch.softmax(near / s["temp"].clamp(min=0.6)[s["seq"]][:, None], 1)
        del near
        s["draft"] = draft
        drawn = torch.empty(t, dtype=torch.int64, device=DEV)
        noise = torch.rand(t, generator=gen, device=DEV).double()
        for i in range(0, t, 512):
            cum = draft[i:i + 512].double().cumsum(1)
            drawn[i:i + 512] = (cum <= noise[i:i + 512, None] * cum[:, -1:]).sum(1).clamp(max=v - 1)
        tokens = drawn[up]
        s["ua"] = torch.rand(t, generator=gen, device=DEV)
    else:
        # the likeliest tokens of the parent's row, one for each child of it
        top = torch.cat([logits[i:i + 512].topk(3, 1).indices for i in range(0, t, 512)])
        child = torch.tensor((node + 2) % 3 if case["tree"] else node * 0, device=DEV)
        tokens = top[up, child]
    s["logits"] = logits.to(DTYPES[case["dtype"]])
    s["tokens"] = tokens.to(torch.int32)
    s["us"] = torch.rand(t, generator=gen, device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return _prepare_verify(case, gen) if case["op"] == "verify" else _prepare_tokens(case, gen)


# ---------------------------------------------------------------- plain forms

def _plain_rope(x, weight, s):
    case, r = s["case"], s["case"]["rot"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    cos, sin = s["table"][s["pos"].long()][:, None].chunk(2, -1)
    if case["style"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., r:]], -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., r:]], -1)


def _plain_encode(x, pages, cents, bits, slots):
    """Rows x[T, H, D] into pages: norm, rotation, nearest centroid, indices LSB first; the rows
    read back, fp16 (zero where the slot is skipped)."""
    t, h, d = x.shape
    rot = _rotation(d, torch.float32)
    nu = x.norm(dim=-1, keepdim=True)
    idx = torch.bucketize((x / nu) @ rot.T, (cents[1:] + cents[:-1]) / 2)
    bit = ((idx[..., None] >> torch.arange(bits, device=DEV)) & 1).to(torch.uint8)
    byte = (bit.reshape(t, h, d * bits // 8, 8) << torch.arange(8, dtype=torch.uint8, device=DEV)).sum(3, dtype=torch.uint8)
    row = torch.cat([byte, nu.contiguous().view(torch.uint8).reshape(t, h, 4)], 2)
    live = slots >= 0
    pages.view(-1, h, row.shape[2])[slots[live]] = row[live]
    return torch.where(live[:, None, None], nu * (cents[idx] @ rot), 0.0).to(torch.float16)


def _plain_tokens(s):
    out = DTYPES[s["case"]["dtype"]]
    q = _plain_rope(s["q"], s["qw"], s).to(out)
    k = _plain_rope(s["k"], s["kw"], s)
    if s["case"]["op"] == "rope":
        return dict(q=q, k=k.to(out))
    return dict(q=q, k=_plain_encode(k, s["kp"], s["kc"], s["case"]["k_bits"], s["slots"]),
                v=_plain_encode(s["v"].float(), s["vp"], s["vc"], s["case"]["v_bits"], s["slots"]))


def _plain_pick(weights, u):
    """First index whose running sum passes u times the whole sum."""
    cum = weights.cumsum(1)
    return (cum <= u.double()[:, None] * cum[:, -1:]).sum(1)


def _plain_verify(s):
    case, seqs, t = s["case"], s["case"]["seqs"], s["logits"].shape[0]
    temp = s["temp"][s["seq"]].double()
    greedy = temp == 0
    z = s["logits"].double() / torch.where(greedy, 1.0, temp)[:, None]
    top = z.amax(1, keepdim=True)
    best = torch.where(z == top, torch.arange(z.shape[1], device=DEV), z.shape[1]).amin(1)
    p = (z - top).exp_()
    del z
    tokens, up = s["tokens"].long(), s["up"]
    if case["draft"]:
        at = up, tokens
        kept = s["ua"].double() * s["draft"][at].double() < p[at] / p.sum(1)[up]
        kept = torch.where(greedy, tokens == best[up], kept)
    else:
        pick = torch.where(greedy, best, _plain_pick(p, s["us"]))
        kept = tokens == pick[up]
    kept |= s["node"] == 0
    for _ in range(max(1, case["nodes"] - 1).bit_length()):  # and every ancestor kept
        kept = kept & kept[up]
        up = up[up]
    first = s["start"][:-1].long()
    count = torch.zeros(seqs, dtype=torch.int64, device=DEV).index_add_(0, s["seq"], kept.long())
    rank = kept.long().cumsum(0)
    rank = rank - rank[first][s["seq"]]
    path = torch.full((seqs, case["nodes"] + 1), -1, dtype=torch.int64, device=DEV)
    path[s["seq"], torch.where(kept, rank, case["nodes"])] = torch.where(kept, s["node"], -1)
    last = first + torch.zeros(seqs, dtype=torch.int64, device=DEV).scatter_reduce_(
        0, s["seq"], torch.where(kept, s["node"], 0), "amax")
    if case["draft"]:
        w = p[last] / p[last].sum(1, keepdim=True)
        leaf = last + 1 == s["start"][1:]  # nothing was drafted behind it
        w -= torch.where(leaf[:, None], 0.0, s["draft"][last].double())
        after = torch.where(greedy[last], best[last], _plain_pick(w.clamp_(min=0), s["us"][last]))
    else:
        after = pick[last]
    i32 = torch.int32
    return dict(path=path[:, :case["nodes"]].to(i32), path_lens=count.to(i32), next=after.to(i32))


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        import quantized_kv_cache_06_gb300 as tq

        pairs = case.get("style") == "pairs"
        if case["op"] == "rope":
            q, k = tq.tq_norm_rope(s["q"], s["k"], s["pos"], s["table"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                   interleaved=pairs)
            return dict(q=q, k=k)
        if case["op"] == "append":
            q = tq.tq_append_kv(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["slots"], s["signs"], s["kc"], s["vc"],
                                positions=s["pos"], cos_sin=s["table"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
                                interleaved=pairs)
            return dict(q=q, k=tq.tq_dequant_rows(s["kp"], s["slots"], s["signs"], s["kc"], check=False),
                        v=tq.tq_dequant_rows(s["vp"], s["slots"], s["signs"], s["vc"], check=False))
        r = tq.tq_verify_tree(s["logits"], s["start"], s["tokens"], s["us"], case["nodes"], parents=s["parents"],
                              temperature=s["temp"], draft_probs=s["draft"], u_accept=s["ua"])
        return dict(path=r.path, path_lens=r.path_lens, next=r.next_token)
    return _plain_verify(s) if case["op"] == "verify" else _plain_tokens(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "verify":
        rows = int(_rows(case).sum())
        size = 4 if case["dtype"] == "fp32" else 2
        # every row of logits, the drafter's probabilities where one token of a request is refused
        need = rows * (case["vocab"] * size + 16.0) + case["seqs"] * (case["nodes"] * 4 + 12.0)
        if case["draft"]:
            need += case["seqs"] * case["vocab"] * 4.0
        return dict(bytes=need, flops=6.0 * rows * case["vocab"])
    t, hq, h, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    per = (hq + h) * d * size + 4.0 + case["rot"] * 4.0  # queries, keys, position and its table row
    flops = (hq + h) * d * (7.0 if case["norm"] else 3.0)
    if case["op"] == "rope":
        return dict(bytes=t * (per + (hq + h) * d * size), flops=t * flops)
    # values, slot; queries out, packed rows out and the dense rows read back from them
    per += h * d * size + 8 + hq * d * size + h * (_row_bytes(d, case["k_bits"]) + _row_bytes(d, case["v_bits"]) + 4.0 * d)
    return dict(bytes=t * per, flops=t * (flops + 2 * h * d * (2 * math.log2(d) + 8)))


# ---------------------------------------------------------------- 64 bits

def _exact_rope(x, weight, pos, table, rot, style):
    """By complex numbers: the pair (a, b) as a + ib times cos + i sin."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * weight.double()
    turn = torch.complex(table[pos.long(), :rot // 2].double(), table[pos.long(), rot // 2:].double())[:, None]
    head, tail = x[..., :rot], x[..., rot:]
    if style == "half":
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
        return torch.cat([z.real, z.imag, tail], -1)
    z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).reshape(head.shape), tail], -1)


def _exact_held(x, cents, slots):
    """What packed rows of x stand for: nearest centroid of each coordinate of the rotated unit row."""
    d = x.shape[-1]
    rot = _rotation(d, torch.float64)
    out = torch.zeros_like(x)
    step = max(1, (1 << 24) // (x.shape[1] * d))
    for i in range(0, x.shape[0], step):
        part = x[i:i + step]
        nu = part.pow(2).sum(-1, keepdim=True).sqrt()
        y = torch.einsum("thd,ed->the", part / nu, rot)
        best = torch.zeros_like(y)
        off = torch.full_like(y, math.inf)
        for c in cents.double().tolist():
            near = (y - c).abs()
            best = torch.where(near < off, c, best)
            off = torch.minimum(near, off)
        out[i:i + step] = nu * torch.einsum("the,ed->thd", best, rot)
    out[slots < 0] = 0
    return out


def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers, which have to be equal
    s = prepare(case, seed)
    q, k = (_exact_rope(s[x], s[w], s["pos"], s["table"], case["rot"], case["style"]) for x, w in (("q", "qw"), ("k", "kw")))
    if case["op"] == "rope":
        return dict(q=q, k=k)
    return dict(q=q, k=_exact_held(k, s["kc"], s["slots"]), v=_exact_held(s["v"].double(), s["vc"], s["slots"]))

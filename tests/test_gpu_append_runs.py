"""tq_norm_rope and tq_append_kv where a warp takes its longest runs (eight groups of heads, four of fp32,
over blocks of four tokens): each form of the kernel against calls of few tokens, where runs are of one
group.  A row's arithmetic does not depend on the cut, so the two are equal bit for bit; a sample of the
tokens is compared with 64 bits, with tests/test_gpu_append.py's tolerances."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_append import BF16, F16, F32, Inputs, near, packed_near, pages_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


def tokens_of_longest_runs(sides, d, dtype):
    """Tokens from which a warp's runs are the longest: 16 warps an SM, two runs' worth each."""
    group = 32 // (d // 16)
    groups = sum(-(-h // group) for h in sides)
    most = 4 if dtype is F32 else 8
    warps = torch.cuda.get_device_properties(0).multi_processor_count * 16
    return -(-most * 2 * warps // groups) + 3  # (not a whole block of four)


@pytest.mark.parametrize("dtype,d,hq,h,rot,norm,pairs,pad,kb,vb", [
    (F32, 128, 6, 3, 128, True, False, 0, 4, 4),
    (F32, 64, 9, 3, 32, True, False, 0, 3, 5),       # lane exchange
    (BF16, 64, 12, 5, 64, False, True, 0, 3, 5),     # pairs
    (F16, 128, 6, 3, 64, True, False, 0, 4, 2),      # lane exchange
    (F16, 128, 6, 3, 96, True, False, 0, 4, 2),      # by shared memory
    (BF16, 256, 4, 3, 256, True, False, 0, 2, 4),
    (BF16, 128, 6, 3, None, True, False, 0, 4, 4),   # norms alone
    (BF16, 32, 20, 9, 32, True, False, 0, 4, 3),     # the kernel for every call
    (BF16, 128, 6, 3, 128, True, False, 3, 4, 4),    # and by its alignment
    (F16, 16, 40, 33, 16, False, True, 0, 2, 5)])
def test_longest_runs(tq, dtype, d, hq, h, rot, norm, pairs, pad, kb, vb):
    t = tokens_of_longest_runs((hq, h, h), d, dtype)
    x = Inputs(tq, t, hq, h, d, dtype, rot, norm, pairs, seed=d + hq, pad=pad)
    kp, vp, signs, kc, vc = pages_of(tq, x, -(-t // 16) + 2, 16, kb, vb)
    slots = torch.randperm(kp.shape[0] * 16, device="cuda")[:t]
    slots[5::11] = -1
    args = x.kw_args()
    if rot:
        args["positions"][7::13] = -1
        pad_rows = args["positions"] < 0
    else:
        pad_rows = torch.zeros(t, dtype=torch.bool, device="cuda")
    out = torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda")
    small_k, small_v, small = kp.clone(), vp.clone(), out.clone()
    q = tq.tq_append_kv(x.q, x.k, x.v, kp, vp, slots, signs, kc, vc, q_out=out, check=True, **args)
    dense = tq.tq_norm_rope(x.q, x.k, **args)
    step = 60
    for at in range(0, t, step):
        part = slice(at, min(t, at + step))
        some = dict(args, positions=args["positions"][part] if rot else None)
        tq.tq_append_kv(x.q[part], x.k[part], x.v[part], small_k, small_v, slots[part], signs, kc, vc, q_out=small[part], **some)
    assert torch.equal(q.view(torch.uint8), small.view(torch.uint8))
    assert torch.equal(kp, small_k) and torch.equal(vp, small_v)
    assert torch.equal(dense[0][~pad_rows], q[~pad_rows]) and torch.all(q[pad_rows] == 7.0)
    live = torch.nonzero(~pad_rows & (slots >= 0))[:, 0]
    pick = torch.cat([live[:40], live[-40:], live[::max(1, len(live) // 80)]]).unique()
    at = pick.cpu().numpy()
    x.pos = x.pos[at]
    near(q[pick], *x.want(x.q[pick], x.qw), dtype)
    near(dense[1][pick], *x.want(x.k[pick], x.kw), dtype)
    packed_near(tq, kp, slots[pick], x.want(x.k[pick], x.kw)[0], signs, kc, kb)
    packed_near(tq, vp, slots[pick], x.v[pick].double().cpu().numpy(), signs, vc, vb)


@pytest.mark.parametrize("dtype,d,h,bits", [(F32, 64, 3, 4), (F16, 256, 3, 5), (BF16, 64, 9, 3)])
def test_longest_runs_of_values_alone(tq, dtype, d, h, bits):
    t = tokens_of_longest_runs((h,), d, dtype)
    x = Inputs(tq, t, 1, h, d, dtype, None, False, seed=h)
    _, vp, signs, _, vc = pages_of(tq, x, -(-t // 16), 16, bits, bits)
    slots = torch.randperm(vp.shape[0] * 16, device="cuda")[:t]
    slots[3::7] = -1
    small = vp.clone()
    tq.tq_append_kv(None, None, x.v, None, vp, slots, signs, None, vc, check=True)
    for at in range(0, t, 200):
        part = slice(at, min(t, at + 200))
        tq.tq_append_kv(None, None, x.v[part], None, small, slots[part], signs, None, vc)
    assert torch.equal(vp, small)
    pick = torch.nonzero(slots >= 0)[::max(1, t // 100), 0]
    packed_near(tq, vp, slots[pick], x.v[pick].double().cpu().numpy(), signs, vc, bits)

"""Norms that tq_append_kv stores: rows of small whole numbers have an exact sum of squares in fp32 whatever
the order, so the stored norm has to be its root, correctly rounded, times the row's power of two."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def tq():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for the gpu tests")
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


@pytest.mark.parametrize("dtype,power", [(F32, 0), (F16, 0), (BF16, 0), (F32, 110), (F32, -120), (BF16, 90), (F16, -10)])
@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("h", [3, 8])
def test_stored_norms_are_rounded_once(tq, dtype, power, d, h):
    t, bits = 200, 4
    rng = np.random.default_rng(d + h)
    x = rng.integers(-3, 4, (t, 2, h, d))
    rows = torch.from_numpy(x * 2.0 ** power).cuda().to(dtype)
    pages = [torch.zeros(-(-t // 16), 16, h, tq.tq_row_bytes(d, bits), dtype=torch.uint8, device="cuda") for _ in range(2)]
    signs, cents = tq.tq_build_rotation(d, 42, "cuda"), tq.tq_codebook(d, bits, "cuda")[0]
    slots = torch.arange(t, device="cuda")
    tq.tq_append_kv(None, rows[:, 0], rows[:, 1], *pages, slots, signs, cents, cents, check=True)
    root = np.sqrt((x * x).sum(-1).astype(np.float32)) * np.float32(2.0 ** power)
    for side in range(2):
        row = pages[side].view(-1, h, pages[side].shape[3])[:t]
        got = row[..., -4:].contiguous().view(F32)[..., 0].cpu().numpy()
        assert got.tobytes() == np.ascontiguousarray(root[:, side]).tobytes()
    if power == 0 and d == 32:  # and the fp32 writer's (the tensor-core one has its norms from rotated rows)
        want = torch.zeros_like(pages[1])
        tq.tq_write_kv(rows[:, 1].contiguous(), want, slots, signs, cents)
        assert torch.equal(want[..., -4:], pages[1][..., -4:])

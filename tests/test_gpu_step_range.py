"""tq_commit_tree at the end of its lengths' range."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", torch.int32)


def test_commit_refuses_lengths_beyond_32_bits():
    # a table of more than 2^31 tokens: the new length would not fit
    import quantized_kv_cache_06_gb300 as tq

    pages = torch.zeros(1, 1 << 30, 1, 1, dtype=torch.uint8, device="cuda")
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ctx = _dev(np.array([2 ** 31 - 1, 2 ** 31 - 3]))
    lens = tq.tq_commit_tree(pages, None, table, ctx, _dev(np.array([[0, 1], [0, 1]])), _dev(np.array([1, 2])),
                             status=status)
    assert lens.tolist() == [2 ** 31 - 1, 2 ** 31 - 1]
    assert int(status.item()) == tq.TQ_ERR_BLOCK_OUT_OF_RANGE  # (the later code: no block is inside the pages)

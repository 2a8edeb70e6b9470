"""Numbers that the library takes in 32 bits are refused beyond them, not cut off."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def tq():
    from quantized_kv_cache_06_gb300 import build

    build.build_library()
    import quantized_kv_cache_06_gb300 as tq

    return tq


def test_host_calls(tq):
    for rot_dim in (2 ** 32 + 2, -2 ** 32 + 2):
        with pytest.raises(ValueError, match="32 bits"):
            tq.tq_build_rope(rot_dim, 0)
    assert tq.tq_verify_tree_workspace(2 ** 32 + 1, 8, 1) == 0 and tq.tq_verify_tree_workspace(1, 8, 2 ** 32 + 1) == 0
    assert tq.tq_verify_tree_workspace(1, 2 ** 32 + 8, 1) == 0


@pytest.mark.gpu
def test_device_calls(tq):
    x = torch.randn(3, 2, 64, device="cuda")
    pos = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    table = tq.tq_build_rope(64, 8, device="cuda")
    signs, cents = tq.tq_build_rotation(64, 42, "cuda"), tq.tq_codebook(64, 4, "cuda")[0]
    pages = torch.zeros(1, 16, 2, tq.tq_row_bytes(64, 4), dtype=torch.uint8, device="cuda")
    slots = torch.arange(3, device="cuda")
    before = x.clone()
    for offset in (2 ** 32, 2 ** 31, -2 ** 31 - 1, -2 ** 32):
        with pytest.raises(ValueError, match="32 bits"):
            tq.tq_norm_rope(x, None, pos, table, position_offset=offset, q_out=x)
        with pytest.raises(ValueError, match="32 bits"):
            tq.tq_append_kv(None, x, x, pages, pages.clone(), slots, signs, cents, cents, pos, table, position_offset=offset)
    assert torch.equal(x, before) and not pages.any()
    # the ends themselves: every position beyond the table, or a padding row's
    with pytest.raises(tq.TQError):
        tq.tq_norm_rope(x, None, pos, table, position_offset=2 ** 31 - 1, q_out=x, check=True)
    tq.tq_norm_rope(x, None, pos, table, position_offset=-2 ** 31, q_out=x, check=True)
    assert torch.equal(x, before)
    with pytest.raises(ValueError, match="32 bits"):
        tq.tq_verify_tree(torch.zeros(1, 8, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                          torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"), 2 ** 32 + 1)

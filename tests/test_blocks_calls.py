"""What the Python calls of the 8-bit operators take and refuse, where nothing is launched.  No GPU needed."""
import pytest
import torch

from mla_decode_attention_absorbed_gb300 import mla


@pytest.mark.parametrize("paged", [False, True])
def test_rows_of_blocks_take_no_scale(paged):
    """Their width alone tells them from codes with one scale: a scale beside them is one or the other gone wrong."""
    prob = mla.Problem(2, 16, 1, 128, 32, 64, 64, 1.0)
    lens, table = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32) if paged else None
    rows = torch.zeros(2, 64, 128 + 16 + 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="kv_scale"):
        mla.make_cache(prob, rows, lens, table, kv_scale=0.5)
    assert mla.make_cache(prob, rows, lens, table).kv_dtype == mla.KV_E4M3_BLOCKS
    assert mla.make_cache(prob, rows[:, :, :160].contiguous(), lens, table, kv_scale=0.5).kv_dtype == mla.KV_E4M3

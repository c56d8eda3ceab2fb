"""Host-side checks of the serving library's corners (no GPU needed)."""
import pytest
import torch

from dynamic_block_sparse_fp_b200 import serve


def test_a_workspace_is_a_plain_buffer():
    here = torch.device("cpu")
    serve._buffer(torch.empty(1000, dtype=torch.uint8), here)
    for ws in (torch.empty(1).expand(1000), torch.empty(100)[::2], 1 << 20):
        with pytest.raises(ValueError, match="workspace"):
            serve._buffer(ws, here)
    with pytest.raises(ValueError, match="workspace"):
        serve._buffer(torch.empty(1000, device="meta"), here)

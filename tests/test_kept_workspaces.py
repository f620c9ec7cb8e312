"""The workspaces that the binding keeps."""
import pytest
import torch

import long_context_mqa_b200 as hs2


def test_no_workspace_yet_is_none():
    """A key that no call has used: None, without asking CUDA for a stream (CPU only)."""
    for key in ("full", "sparse", "bridge", "nothing", "paged_attn"):
        if not torch.cuda.is_available():
            assert hs2.cached_workspace(key, torch.device("cuda", 0)) is None
    assert hs2.cached_workspace("nothing", torch.device("cuda", 0)) is None


@pytest.mark.gpu
def test_a_stream_that_kept_none():
    side = torch.cuda.Stream()
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    hs2.page_table_update(table, i, i, torch.arange(6, dtype=torch.int32, device="cuda"), i, 16, 0)
    assert hs2.cached_workspace("page_table") is not None
    assert hs2.cached_workspace("page_table", torch.device("cuda", torch.cuda.current_device())) is not None
    assert hs2.cached_workspace("page_table", stream=torch.cuda.current_stream()) is not None
    assert hs2.cached_workspace("page_table", stream=side) is None

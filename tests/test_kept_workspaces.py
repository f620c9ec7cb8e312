"""The workspaces that the binding keeps, and the calls that need none."""
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


@pytest.mark.gpu
def test_backward_without_weights_needs_no_workspace():
    """The scratch holds the weights' gradients: without weights the call is captured without one, and the C entry takes
    none."""
    g = torch.Generator(device="cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    q, k, dq, dk = new(37, 4, 64), new(37, 2, 64), new(37, 4, 64), new(37, 2, 64)
    pos = torch.arange(37, dtype=torch.int32, device="cuda")
    freq, _ = hs2.rope_frequencies(32)
    want = hs2.qk_norm_rope_bwd(q, k, pos, freq, dq, dk)
    assert want[2] is None and want[3] is None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = hs2.qk_norm_rope_bwd(q, k, pos, freq, dq, dk)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    xq, xk = torch.zeros_like(q), torch.zeros_like(k)
    code = hs2.lib.hs2_qk_norm_rope_bwd(q.data_ptr(), k.data_ptr(), 256, 64, 128, 64, pos.data_ptr(), freq.data_ptr(), 37, 4, 2,
                                        64, 32, 0, 1.0, 1e-6, None, None, 0, dq.data_ptr(), dk.data_ptr(), 0, xq.data_ptr(),
                                        xk.data_ptr(), None, None, None, 0, torch.cuda.current_stream().cuda_stream)
    assert code == hs2.OK
    assert torch.equal(xq, want[0]) and torch.equal(xk, want[1])
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hs2.qk_norm_rope_bwd(q, k, pos, freq, dq, dk, q_weight=w, k_weight=w)

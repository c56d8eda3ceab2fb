"""Host-side checks of the serving library's corners (no GPU needed)."""
import pytest
import torch
from test_serve_host import FAKE, PAST, WS, L, batch, cache, needs_no_gpu, paged  # noqa: F401

from dynamic_block_sparse_fp_b200 import ops, serve

NARROW = dict(dtype=serve.FP_E4M3, k_exps=FAKE, v_exps=FAKE)


def test_a_workspace_is_a_plain_buffer():
    here = torch.device("cpu")
    serve._buffer(torch.empty(1000, dtype=torch.uint8), here)
    for ws in (torch.empty(1).expand(1000), torch.empty(100)[::2], 1 << 20):
        with pytest.raises(ValueError, match="workspace"):
            serve._buffer(ws, here)
    with pytest.raises(ValueError, match="workspace"):
        serve._buffer(torch.empty(1000, device="meta"), here)


@needs_no_gpu
def test_fp32_queries_need_no_workspace(L):  # noqa: F811
    b = batch(max_q_len=100, total_q=200)
    assert paged(cache(**NARROW), b) == WS
    assert paged(cache(**NARROW), b, dtype=ops.FP_F32) in PAST


def test_chunks_over_8_bits_copy_the_batchs_pages_not_the_pool(L):  # noqa: F811
    def copies(**kw):
        b = batch(max_q_len=100, total_q=200, **kw)
        return (serve.fp_paged_attn_workspace(cache(n_pages=n_pages, **NARROW), b, 4)
                - serve.fp_paged_attn_workspace(cache(n_pages=n_pages), b, 4))

    page = 4 * 2 * 16 * 128  # of K and V, in bf16
    n_pages = 2 ** 20
    assert 0 <= copies() - 8 * page <= 1024  # (2 sequences of 4 pages; alignment)
    n_pages = 5
    assert 0 <= copies() - 5 * page <= 1024


def test_a_workspace_is_asked_for_and_its_size_checked(L):  # noqa: F811
    b = batch(max_pages=4096)
    for c in (cache(), cache(**NARROW)):
        need = serve.fp_paged_attn_workspace(c, b, 4)
        assert need > 0
        assert paged(c, b) == WS
        assert paged(c, b, ws=FAKE, ws_bytes=need - 1) == WS
        assert paged(c, b, ws=FAKE + 128, ws_bytes=need) == WS

"""Corners of the serving operators, against the 64-bit oracle with the tolerances
of test_serve_gpu.py: units in which nothing is visible, values that are infinities
or NaN, pages behind a window, large batches."""
import math

import numpy as np
import pytest
import torch
from test_serve_gpu import (BF, DEV, F8, _lib, _status, check_group, contents,  # noqa: F401
                            make_batch, make_cache, np64, sequence)

from dynamic_block_sparse_fp_b200 import ops, serve

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEVICE_CHECK = ops.STATUS_CODES["FP_ERR_DEVICE_CHECK"]


# ------------------------------------------------ units that see nothing --

@pytest.mark.parametrize("cache_dtype", [BF, F8])
@pytest.mark.parametrize("q_len", [1, 9, 40])
def test_units_without_a_visible_key_leave_the_others_alone(cache_dtype, q_len):
    """The pages of the first half of a sequence are missing, so whole units see no
    key; the logits of the rest lie near -200 (2^-288), which a reference of 0 would
    flush to nothing."""
    hq, hkv, d, page, length = 8, 2, 128, 64, 9000
    n_pages = -(-length // page)
    cache = make_cache(cache_dtype, n_pages, hkv, page, d, 1)
    b, table, off = make_batch([length], [q_len], page, n_pages, 1, slack_pages=100)
    g = torch.Generator(device=DEV).manual_seed(5)
    k = -200 / math.sqrt(d) + 0.3 * torch.randn(1, hkv, length, d, generator=g, device=DEV)
    v = torch.randn(1, hkv, length, d, generator=g, device=DEV)
    every = serve.Batch(b.page_table, b.kv_lens, max_q_len=length)
    serve.kv_write(cache, every, k.to(BF), v.to(BF))
    q = torch.ones(q_len * hq, d, dtype=BF, device=DEV)
    gone = 70
    b.page_table[0, :gone] = -1
    out, lse = serve.paged_attn(q, cache, b)
    assert serve.fp_serve_last_device_status() == DEVICE_CHECK
    hidden = np.arange(length) < gone * page
    kd, vd = (sequence(x, table, 0, length, page) for x in contents(cache))
    o, x = (np64(y).reshape(hkv, hq // hkv, q_len, d) for y in (out, q))
    ls = np64(lse).reshape(hkv, hq // hkv, q_len)
    for h in range(hkv):
        check_group(o[h], ls[h], x[h], kd[h], vd[h], length - q_len, 0, 0, BF, hidden)

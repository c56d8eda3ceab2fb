"""Corners of the serving operators, against the 64-bit oracle with the tolerances
of test_serve_gpu.py: units in which nothing is visible, values that are infinities
or NaN, pages behind a window, large batches."""
import math

import numpy as np
import pytest
import torch
from test_serve_gpu import (BF, DEV, F8, F32, _lib, _status, check_group,  # noqa: F401
                            contents, make_batch, make_cache, np64, sequence)

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


# ------------------------------------------------------ ends of the range --

@pytest.mark.parametrize("cache_dtype", [BF, F8])
@pytest.mark.parametrize("hq,q_len", [(2, 1), (8, 5), (8, 40)])
@pytest.mark.parametrize("q_exp,k_exp,meet", [(100, 100, False), (127, 119, False),
                                              (-110, 112, True), (-122, 119, True),
                                              (110, -112, True), (127, -126, True)])
def test_queries_and_keys_near_the_ends_of_their_range(cache_dtype, hq, q_len, q_exp, k_exp, meet):
    """Large queries and keys in different channels have logits of 0; large ones and
    small ones in the same channels have ordinary logits."""
    hkv, d, page, length = 2, 128, 64, 300
    cache = make_cache(cache_dtype, 5, hkv, page, d, 1)
    b, table, _ = make_batch([length], [q_len], page, 5, 1)
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn(1, hkv, length, d, generator=g, device=DEV).to(BF) for _ in range(2))
    q = torch.randn(q_len * hq, d, generator=g, device=DEV).clamp(-1.9, 1.9).to(BF)
    k = k.clamp(-1.9, 1.9)
    if not meet:
        k[..., :64], q[:, 64:] = 0, 0
    # (two steps: 2^127 has no double in fp32)
    q, k = q.double() * 2.0 ** q_exp, k.double() * 2.0 ** k_exp
    q, k = q.to(BF), k.to(BF)
    assert q.isfinite().all() and k.isfinite().all()
    every = serve.Batch(b.page_table, b.kv_lens, max_q_len=length)
    serve.kv_write(cache, every, k, v)
    out, lse = serve.paged_attn(q, cache, b)
    kd, vd = (sequence(x, table, 0, length, page) for x in contents(cache))
    o, x = (np64(y).reshape(hkv, hq // hkv, q_len, d) for y in (out, q))
    ls = np64(lse).reshape(hkv, hq // hkv, q_len)
    for h in range(hkv):
        check_group(o[h], ls[h], x[h], kd[h], vd[h], length - q_len, 0, 0, BF)


# ------------------------------------------- infinities and NaNs in values --

def fastest(call, runs=5):
    best = math.inf
    for _ in range(runs):
        a, z = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        z.record()
        z.synchronize()
        best = min(best, a.elapsed_time(z))
    return best


ODD_CASES = [([16001], [1], 0, 0), ([700, 16001, 40], [1, 9, 3], 0, 0), ([9000, 2500], [1, 16], 90, 5),
             ([12001], [200], 0, 0), ([9000, 300], [333, 2], 700, 70)]


@pytest.mark.parametrize("missing", [False, True])
@pytest.mark.parametrize("case", range(len(ODD_CASES)))
def test_odd_values_reach_those_who_see_them_and_cost_little(case, missing):
    """Infinities and NaNs in values all over long sequences: each row has those of
    the keys that it sees (and what they make together), and no call takes 20 times as
    long for them.  One of the pages is missing, or none."""
    hq, hkv, d, page = 8, 2, 128, 64
    kv_lens, q_lens, window, sinks = ODD_CASES[case]
    n_pages = sum(-(-x // page) for x in kv_lens)
    cache = make_cache(BF, n_pages, hkv, page, d, case)
    b, table, off = make_batch(kv_lens, q_lens, page, n_pages, case)
    g = torch.Generator(device=DEV).manual_seed(case)
    q = torch.randn(b.total_q * hq, d, generator=g, device=DEV).to(BF)
    hidden = [np.zeros(x, bool) for x in kv_lens]
    s = int(np.argmax(kv_lens))
    if missing:
        gone = (kv_lens[s] - 80) // page if window else kv_lens[s] // page // 3
        b.page_table[s, gone] = -1
        hidden[s][gone * page:(gone + 1) * page] = True
    ws = serve.workspace(cache, b, hq)
    call = lambda: serve.paged_attn(q, cache, b, window=window, sinks=sinks, ws=ws)  # noqa: E731
    clean, clean_lse = call()
    quiet = fastest(call)
    # where they stand: (key from the sequence's end, column, value)
    odd = [(0, 3, math.inf), (0, 9, math.inf), (1, 9, -math.inf), (63, 17, math.nan),
           (64, 20, -math.inf), (100, 21, math.inf), (700, 40, math.inf), (2000, 41, math.nan),
           (kv_lens[s] - 3, 50, -math.inf), (kv_lens[s] - 65, 51, math.inf)]
    want = np64(clean).copy()
    rows = want[off[s] * hq:off[s + 1] * hq].reshape(hkv, hq // hkv, q_lens[s], d)
    for back, col, x in odd:
        key = kv_lens[s] - 1 - back
        if hidden[s][key]:
            continue
        cache.v[int(table[s, key // page]), 1, key % page, col] = x
        for t in range(q_lens[s]):
            i = kv_lens[s] - q_lens[s] + t
            if key <= i and (window == 0 or i - key < window or key < sinks):
                with np.errstate(invalid="ignore"):  # inf - inf
                    rows[1, :, t, col] += x
    out, lse = call()
    assert np.array_equal(np64(out), want, equal_nan=True)
    assert torch.equal(lse, clean_lse)
    assert fastest(call) <= 20 * quiet + 0.1
    cache.v[int(table[s, (kv_lens[s] - 1) // page])] = math.nan
    out, _ = call()
    # (a sequence's rows are [hq, n_s, d]: the last token's)
    assert out[off[s] * hq:off[s + 1] * hq].view(hq, q_lens[s], d)[:, -1].isnan().all()
    assert fastest(call) <= 20 * quiet + 0.1
    if missing:
        assert serve.fp_serve_last_device_status() == DEVICE_CHECK


# ---------------------------------------------------------------- refusals --

def test_workspaces_that_are_no_buffers_are_refused():
    """(before anything is launched)"""
    cache = make_cache(BF, 100, 2, 64, 128, 0)
    b, _, _ = make_batch([6000], [1], 64, 100, 0, slack_pages=200)
    q = torch.zeros(8, 128, dtype=BF, device=DEV)
    n = serve.workspace(cache, b, 8).numel()
    assert n > 0
    for ws in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(n),
               torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2],
               torch.empty(n, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            serve.paged_attn(q, cache, b, ws=ws)
    with pytest.raises(ops.FPError, match="FP_ERR_WORKSPACE"):
        serve.paged_attn(q, cache, b, ws=torch.empty(n - 1, dtype=torch.uint8, device=DEV))


# ------------------------------------------------- copies of 8-bit pages --

@pytest.mark.parametrize("pages", [0, 3, 500])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks_over_8_bits_in_pools_of_any_size(pages, window, sinks, d):
    """Bitwise the attention over a bf16 cache of the same values, in pools with
    fewer and more pages than the table has places; two sequences share pages, one
    page is missing, and the workspace held NaNs."""
    kv_lens, q_lens, page, hq, hkv = [700, 333, 640], [70, 100, 130], 32, 8, 2
    n_pages = sum(-(-x // page) for x in kv_lens) + pages
    cache = make_cache(F8, n_pages, hkv, page, d, 4)
    b, table, off = make_batch(kv_lens, q_lens, page, n_pages, 4)
    b.page_table[2, :8] = b.page_table[0, :8]
    b.page_table[1, 333 // page - 4] = n_pages
    wide = serve.KVCache(*(torch.tensor(x, dtype=BF, device=DEV) for x in contents(cache)))
    q = torch.randn(b.total_q * hq, d, generator=torch.Generator(device=DEV).manual_seed(2),
                    device=DEV).to(BF)
    ws = serve.workspace(cache, b, hq)
    ws.fill_(255)
    out, lse = serve.paged_attn(q, cache, b, window=window, sinks=sinks, ws=ws)
    want, want_lse = serve.paged_attn(q, wide, b, window=window, sinks=sinks)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert out.isfinite().all()
    assert serve.fp_serve_last_device_status() == DEVICE_CHECK


# ------------------------------------------------ pages behind the window --

@pytest.mark.parametrize("q_dtype,cache_dtype", [(BF, BF), (BF, F8), (F32, F32), (F32, F8)])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("q_len,window,sinks", [(1, 90, 0), (1, 37, 20), (12, 90, 1), (12, 1, 0),
                                                (70, 100, 0), (70, 25, 33)])
def test_entries_behind_the_window_may_be_anything(q_dtype, cache_dtype, page, q_len, window,
                                                   sinks):
    """Pages that no new token sees were given back: their entries are no page
    numbers, or another's page that holds bytes of all kinds.  That is no error, and
    changes nothing."""
    hq, hkv, d, kv_lens = 8, 2, 128, [1000, 300, 555]
    n_pages = sum(-(-x // page) for x in kv_lens) + 1
    cache = make_cache(cache_dtype, n_pages, hkv, page, d, 2)
    b, table, off = make_batch(kv_lens, [q_len] * 3, page, n_pages, 2)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn(b.total_q * hq, d, generator=g, device=DEV).to(q_dtype)
    want, want_lse = serve.paged_attn(q, cache, b, window=window, sinks=sinks)
    spare = (set(range(n_pages)) - {int(table[s, p]) for s in range(3)
                                    for p in range(-(-kv_lens[s] // page))}).pop()
    for x in (cache.k, cache.v):
        x[spare] = math.nan  # (0x7f in 8 bits)
    if cache_dtype == F8:
        cache.k_exps[spare] = 0
        cache.v_exps[spare] = 127
    for entry in (-1, n_pages, spare):
        for s, length in enumerate(kv_lens):
            low = length - q_len - window + 1  # the first key of the first window
            for p in range(-(-length // page)):
                if (p + 1) * page <= low and p * page >= sinks:
                    b.page_table[s, p] = entry
        out, lse = serve.paged_attn(q, cache, b, window=window, sinks=sinks)
        assert serve.fp_serve_last_device_status() == 0
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # one page more is an error
    low = kv_lens[0] - q_len - window + 1
    b.page_table[0, low // page] = -1
    serve.paged_attn(q, cache, b, window=window, sinks=sinks)
    assert serve.fp_serve_last_device_status() == DEVICE_CHECK

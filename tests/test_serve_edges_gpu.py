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


# ------------------------------------------------------------ large batches --

def check_some(out, lse, q, data, table, off, case, hq, hkv, which):
    kv_lens, q_lens, page, window, sinks = case
    d = q.shape[-1]
    for s in which:
        length, n = kv_lens[s], q_lens[s]
        if n == 0:
            continue
        sl = slice(off[s] * hq, off[s + 1] * hq)
        o, x = (np64(y[sl]).reshape(hkv, hq // hkv, n, d) for y in (out, q))
        ls = np64(lse[sl]).reshape(hkv, hq // hkv, n)
        k, v = (sequence(y, table, s, length, page) for y in data)
        for h in range(hkv):
            check_group(o[h], ls[h], x[h], k[h], v[h], length - n, window, sinks, BF)


def run_all(cache, b, q, hq, window, sinks):
    """paged_attn into outputs that were NaN: whatever is not written shows."""
    out, lse = torch.full_like(q, math.nan), torch.full((len(q),), math.nan, device=DEV)
    ws = serve.workspace(cache, b, hq)
    assert serve.fp_paged_attn(cache.struct, b.struct, hq, ops.FP_BF16, window, sinks, q, out, lse,
                               ws) == 0
    assert not out.isnan().any() and not lse.isnan().any()
    return out, lse


@pytest.mark.parametrize("cache_dtype", [BF, F8])
@pytest.mark.parametrize("hq,hkv,q_len", [(8, 2, 1), (16, 1, 3), (32, 2, 4)])
@pytest.mark.parametrize("n_seqs,longest,slack", [(100, 200, 100), (100, 1500, 0), (1100, 100, 100),
                                                  (1100, 40, 0)])
def test_many_sequences_of_few_rows(cache_dtype, hq, hkv, q_len, n_seqs, longest, slack):
    """Units and their join, and whole items, against the oracle; one sequence much
    longer than the others."""
    page = 16
    kv_lens = [1 + (longest * (7 * s + 3)) // (7 * n_seqs) for s in range(n_seqs)]
    kv_lens[n_seqs // 3] = 5000
    q_lens = [max(0, q_len - s % 2) for s in range(n_seqs)]
    case = (kv_lens, q_lens, page, 0, 0)
    n_pages = sum(-(-x // page) for x in kv_lens) + 1
    cache = make_cache(cache_dtype, n_pages, hkv, page, 128, n_seqs)
    b, table, off = make_batch(kv_lens, q_lens, page, n_pages, n_seqs, slack_pages=slack)
    g = torch.Generator(device=DEV).manual_seed(n_seqs)
    q = torch.randn(b.total_q * hq, 128, generator=g, device=DEV).to(BF)
    out, lse = run_all(cache, b, q, hq, 0, 0)
    some = sorted({0, 2, 7, n_seqs // 3, n_seqs // 3 + 1, n_seqs // 2, n_seqs - 2, n_seqs - 1})
    check_some(out, lse, q, contents(cache), table, off, case, hq, hkv, some)


@pytest.mark.parametrize("cache_dtype", [BF, F8])
@pytest.mark.parametrize("n_seqs,chunk,window", [(5, 1500, 0), (64, 2048, 0), (64, 2048, 333),
                                                 (20, 700, 0)])
def test_single_tokens_beside_a_chunk(cache_dtype, n_seqs, chunk, window):
    """One sequence brings a chunk, the others a token each (one of them none)."""
    hq, hkv, page = 8, 2, 64
    kv_lens = [(37 * s * s) % 2900 + 1 for s in range(n_seqs)]
    q_lens = [1] * n_seqs
    kv_lens[2], q_lens[2], q_lens[1] = chunk + 500, chunk, 0
    kv_lens[3] = 9000
    case = (kv_lens, q_lens, page, window, 5)
    n_pages = sum(-(-x // page) for x in kv_lens) + 1
    cache = make_cache(cache_dtype, n_pages, hkv, page, 128, n_seqs)
    b, table, off = make_batch(kv_lens, q_lens, page, n_pages, n_seqs)
    g = torch.Generator(device=DEV).manual_seed(n_seqs)
    q = torch.randn(b.total_q * hq, 128, generator=g, device=DEV).to(BF)
    out, lse = run_all(cache, b, q, hq, window, 5)
    check_some(out, lse, q, contents(cache), table, off, case, hq, hkv,
               sorted({0, 2, 3, 4, n_seqs - 1}))


def test_calls_repeat_themselves_bitwise():
    """Every operator, twice on the same inputs with other calls between."""
    for cache_dtype, q_len in ((BF, 1), (F8, 1), (BF, 150), (F8, 150)):
        kv_lens, page = [9000, 200, 3333], 64
        n_pages = sum(-(-x // page) for x in kv_lens)
        cache = make_cache(cache_dtype, n_pages, 2, page, 128, 1)
        b, _, _ = make_batch(kv_lens, [q_len] * 3, page, n_pages, 1)
        g = torch.Generator(device=DEV).manual_seed(2)
        q = torch.randn(b.total_q * 8, 128, generator=g, device=DEV).to(BF)
        x = torch.randn(1, 4, 900, 128, generator=g, device=DEV).to(BF)
        kv = torch.randn(b.total_q * 2, 128, generator=g, device=DEV).to(BF)
        seen = []
        for _ in range(3):
            serve.kv_write(cache, b, kv, kv)
            seen.append([*serve.paged_attn(q, cache, b), *serve.window_attn(x, x, x, 100, 4),
                         *serve.kv_read(cache, b), cache.k.view(torch.uint8).clone()])
        assert all(torch.equal(y, z) for later in seen[1:] for y, z in zip(seen[0], later))


@pytest.mark.parametrize("hq,hkv", [(2, 1), (8, 2), (32, 8), (24, 24)])
@pytest.mark.parametrize("seed", range(6))
def test_every_row_is_written_however_the_lengths_fall(hq, hkv, seed):
    """The cut of random batches on the device: no row is left out (NaN), and each
    sequence comes out as when it is called by itself, up to the weights' rounding
    (2^-8 of the values' size each) and the output's, for both."""
    rng = np.random.default_rng(seed)
    page, d = 64, 64
    n_pages = 700
    cache = make_cache(BF, n_pages, hkv, page, d, seed)
    top = float(cache.v.abs().max())
    for _ in range(8):
        n = int(rng.choice([1, 2, 5, 31, 32, 33, 70, 140, 500]))
        longest = int(2 ** rng.uniform(2, 14))
        kv_lens = [int(rng.choice([longest, rng.integers(0, longest + 1), 0])) for _ in range(n)]
        most = int(rng.choice([1, 1, 3, 20, 300]))
        q_lens = [int(rng.integers(0, most + 1)) for _ in range(n)]
        q_lens[0] = most
        # (pages are shared among the sequences)
        table = rng.integers(0, n_pages, (n, longest // page + 1 + int(rng.choice([0, 50, 500]))))
        table = torch.tensor(table, dtype=torch.int32, device=DEV)
        off = np.concatenate([[0], np.cumsum(q_lens)])
        b = serve.Batch(table, torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                        torch.tensor(off, dtype=torch.int32, device=DEV), max_q_len=most,
                        total_q=int(off[-1]))
        q = torch.randn(b.total_q * hq, d, device=DEV).to(BF)
        window = int(rng.choice([0, 0, 100]))
        out, lse = run_all(cache, b, q, hq, window, 3)
        for s in {0, n // 2, n - 1}:
            if q_lens[s] == 0:
                continue
            one = serve.Batch(table[s:s + 1].contiguous(), b.kv_lens[s:s + 1].contiguous(),
                              max_q_len=q_lens[s])
            sl = slice(int(off[s]) * hq, int(off[s + 1]) * hq)
            o, x = serve.paged_attn(q[sl].view(1, hq, q_lens[s], d), cache, one, window, 3)
            assert (o.view(-1, d).float() - out[sl].float()).abs().max() <= 4 * 2.0 ** -8 * top
            x, y = x.view(-1), lse[sl]
            assert torch.equal(x.isinf(), y.isinf())
            assert ((x - y)[~x.isinf()].abs() <= 1e-4 * (1 + y[~x.isinf()].abs())).all()

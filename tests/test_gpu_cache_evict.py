"""Accumulation of attention mass and eviction of pages against their definitions."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE = 128


def plain_evict(table, lens, w, budget, sink, window):
    """The definition, request by request: sums in fp32 and head order, stable ranking."""
    B, H, cols = w.shape
    new_t, freed = np.full((B, cols), -1, np.int32), np.full((B, cols), -1, np.int32)
    new_w, new_n, count = np.zeros_like(w), np.array(lens, np.int32), np.zeros(B, np.int32)
    for b, n in enumerate(lens):
        if n < 0 or n > cols * PAGE:
            new_t[b], new_w[b] = table[b, :cols], w[b]
            continue
        nb = -(-n // PAGE)
        total = w[b, 0, :nb].copy()
        for h in range(1, H):
            total = total + w[b, h, :nb]
        rank = np.where(np.isnan(total), -np.inf, total.astype(np.float64))
        order = sorted(range(nb), key=lambda j: (not (j < sink or j >= nb - window), bool(np.isnan(total[j])),
                                                 -rank[j], j))
        keep = np.array(sorted(order[:budget]), dtype=np.int64)
        gone = np.setdiff1d(np.arange(nb), keep)
        new_t[b, :len(keep)], freed[b, :len(gone)] = table[b, keep], table[b, gone]
        new_w[b, :, :len(keep)] = w[b][:, keep]
        count[b], new_n[b] = len(gone), n - PAGE * len(gone)
    return new_t, new_n, new_w, freed, count


def make(seed, lens, H, cols, kind):
    r = np.random.default_rng(seed)
    B = len(lens)
    table = r.permutation(B * cols).reshape(B, cols).astype(np.int32)
    w = (r.random((B, H, cols)).astype(np.float32) + 1e-3) ** -2
    if kind == "ties":
        w = r.integers(0, 3, (B, H, cols)).astype(np.float32)
    elif kind == "zeros":
        w[:] = 0.0
        w[:, :, ::5] = -0.0
    elif kind == "odd":  # negative, infinite and NaN weights
        w *= r.choice([-1.0, 1.0], w.shape).astype(np.float32)
        w[r.random(w.shape) < 0.1] = np.nan
        w[r.random(w.shape) < 0.1] = np.inf
        w[r.random(w.shape) < 0.05] = -np.inf
    return table, w


CASES = [
    ([1], 4, 1, 1, 0, 1, "spread"),
    ([0, 1, 128, 129, 4000, 6400], 4, 50, 7, 1, 2, "spread"),
    ([6400, 6399, 3000], 2, 50, 3, 1, 2, "ties"),
    ([6400, 6399, 3000], 1, 50, 49, 0, 1, "ties"),
    ([6400, 129], 4, 50, 20, 3, 5, "zeros"),
    ([6400, 5000, 130], 3, 50, 21, 1, 2, "odd"),
    ([PAGE * 1500, PAGE * 1499 + 1, 70000], 4, 1500, 1000, 1, 2, "spread"),
    ([PAGE * 8192 - 5, PAGE * 4096], 2, 8192, 2049, 1, 2, "ties"),
    ([PAGE * 32768, 1], 1, 32768, 5, 2, 3, "spread"),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{c[2]}h{c[1]}b{c[3]}{c[6]}")
def test_evict_matches_the_definition(case, in_place):
    import sparse_attention_decode_gb300 as msa
    lens, H, cols, budget, sink, window, kind = case
    table, w = make(3, lens, H, cols, kind)
    B = len(lens)
    wide = torch.full((B, cols + 3), 77, dtype=torch.int32, device="cuda")  # a strided table
    wide[:, :cols] = torch.from_numpy(table)
    t, n, ww = wide[:, :cols], torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.from_numpy(w).cuda()
    out = (t, n, ww) if in_place else (torch.full_like(t.contiguous(), 5), torch.full_like(n, 5), torch.full_like(ww, 5))
    freed = torch.full((B, cols), 5, dtype=torch.int32, device="cuda")
    count = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_cache_evict(t, n, ww, budget, sink, window, *out, freed, count, ws)
    want = plain_evict(table, lens, w, budget, sink, window)
    for got, r, name in zip((*out, freed, count), want, ("table", "lens", "weights", "freed", "n_freed")):
        np.testing.assert_array_equal(got.cpu().numpy(), r, err_msg=name)
    assert bool((wide[:, cols:] == 77).all()) and msa.msa_indexer_get_error(ws) == 0


def test_a_bad_length_passes_the_request_through():
    import sparse_attention_decode_gb300 as msa
    lens = [6400, -1, 6401, 5000]
    table, w = make(4, lens, 2, 50, "spread")
    t, n, ww = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), \
        torch.from_numpy(w).cuda()
    freed, count = torch.empty_like(t), torch.empty_like(n)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_cache_evict(t, n, ww, 10, 1, 2, t, n, ww, freed, count, ws)
    want = plain_evict(table, lens, w, 10, 1, 2)
    for got, r in zip((t, n, ww, freed, count), want):
        np.testing.assert_array_equal(got.cpu().numpy(), r)
    assert msa.msa_indexer_get_error(ws) == msa.MSA_FAULT_SEQ_LEN


@pytest.mark.parametrize("q_len,H,sel,k,rows", [(1, 4, 4, 16, None), (4, 4, 4, 16, [0, 1, 2, 3, 4]), (3, 8, 2, 32, [3, 0, 2]),
                                                (2, 1, 1, 1, None), (64, 2, 2, 5, [64, 63])])
def test_accumulate_in_position_order(q_len, H, sel, k, rows):
    import sparse_attention_decode_gb300 as msa
    r = np.random.default_rng(8)
    B, cols = len(rows) if rows else 3, 70
    w = r.random((B, H, cols)).astype(np.float32) * 100
    ids = np.stack([[r.permutation(cols)[:k] for _ in range(sel)] for _ in range(B * q_len)]).astype(np.int32)
    ids[r.random(ids.shape) < 0.2] = -1
    if k > 4:
        ids[0, 0, 3] = ids[0, 0, 4] = 9  # equal ids add up in slot order
    mass = r.random((B * q_len, H, k)).astype(np.float32)
    want = w.copy()
    for b in range(B):
        for i in range(rows[b] if rows else q_len):
            for h in range(H):
                for j in range(k):
                    x = ids[b * q_len + i, h // (H // sel), j]
                    if x >= 0:
                        want[b, h, x] += mass[b * q_len + i, h, j]
    dev = torch.from_numpy(w).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_cache_accumulate(dev, torch.from_numpy(ids).cuda(), torch.from_numpy(mass).cuda(), ws, q_len=q_len,
                             n_rows=torch.tensor(rows, dtype=torch.int32, device="cuda") if rows else None)
    np.testing.assert_array_equal(dev.cpu().numpy(), want)  # the same sums in the same order
    assert msa.msa_indexer_get_error(ws) == 0


def test_accumulate_reports_what_it_skips():
    import sparse_attention_decode_gb300 as msa
    w = torch.zeros(2, 1, 10, device="cuda")
    ids = torch.tensor([[[3, 10]], [[4, 5]]], dtype=torch.int32, device="cuda")
    mass = torch.ones(2, 1, 2, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_cache_accumulate(w, ids, mass, ws, n_rows=torch.tensor([1, 2], dtype=torch.int32, device="cuda"))
    assert msa.msa_indexer_get_error(ws) == msa.MSA_FAULT_BLOCK_ID | msa.MSA_FAULT_SEQ_LEN
    want = torch.zeros(2, 1, 10)
    want[0, 0, 3] = 1
    assert torch.equal(w.cpu(), want)


def test_refusals():
    import sparse_attention_decode_gb300 as msa
    t = torch.zeros(1, 8, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.zeros(1, 2, 8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    run = lambda *a, ws=ws: msa.msa_cache_evict(t, n, w, *a, t, n, w, t.clone(), n.clone(), ws)  # noqa: E731
    run(3, 1, 2)
    for bad in ((2, 1, 2), (3, 1, 0), (3, -1, 2)):
        with pytest.raises(msa.MsaError) as e:
            run(*bad)
        assert e.value.status == msa.MSA_ERR_INVALID_ARG
    with pytest.raises(msa.MsaError) as e:
        run(3, 1, 2, ws=ws[:255])
    assert e.value.status == msa.MSA_ERR_WORKSPACE_TOO_SMALL
    wide = torch.zeros(1, 32769, dtype=torch.int32, device="cuda")
    ww = torch.zeros(1, 1, 32769, device="cuda")
    with pytest.raises(msa.MsaError) as e:
        msa.msa_cache_evict(wide, n, ww, 3, 1, 2, wide, n, ww, wide.clone(), n.clone(), ws)
    assert e.value.status == msa.MSA_ERR_UNSUPPORTED
    with pytest.raises(AssertionError):
        msa.msa_cache_evict(t, n, w.double(), 3, 1, 2, t, n, w, t.clone(), n.clone(), ws)

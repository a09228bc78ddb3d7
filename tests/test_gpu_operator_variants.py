"""Kernel forms that are chosen by the batch's size or the width of a table, against the definitions."""

import numpy as np
import pytest
import torch

import test_gpu_attention_prefix as prefix
import test_gpu_attention_sparse as sparse
import test_gpu_cache_evict as evict
import test_gpu_verify_draft as verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,S,V", [(100, 3, 1000), (100, 2, 1021), (152, 1, 79), (160, 3, 1000), (160, 2, 1021), (300, 4, 512)])
def test_verification_of_many_requests(B, S, V, dtype):
    """More than five eighths of a request an SM: rows one at a time, clusters of 4, then of 2; whole and shifted rows."""
    import sparse_attention_decode_gb300 as msa
    w = verify.make(51, B, S, V, dtype, greedy=9)
    assert verify.check(msa, w) == 0
    assert verify.check(msa, w, n_draft=False) == 0


@pytest.mark.parametrize("case", [(5000, list(range(40)), 1, 4, 16, "hnd"), (300, [130] * 50, 2, 2, 16, "nhd"),
                                  (0, [3 * i for i in range(40)], 1, 4, 16, "hnd")], ids=["p5000", "p300", "p0"])
def test_prefix_with_more_joined_rows_than_warps_at_once(case):
    import sparse_attention_decode_gb300 as msa
    assert prefix.verify(msa, prefix.make(52, *case)) == 0


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("cols,H,budget,kind", [(64, 4, 20, "spread"), (64, 1, 9, "ties"), (1024, 2, 700, "odd"), (1024, 5, 33, "ties"),
                                                (1501, 4, 900, "spread"), (1502, 2, 40, "odd"), (1027, 3, 1000, "zeros")])
def test_evict_at_other_widths(cols, H, budget, kind, in_place):
    evict.test_evict_matches_the_definition(([evict.PAGE * cols, evict.PAGE * (cols - 1) + 1, evict.PAGE * (cols // 2), 0], H, cols,
                                             budget, 1, 2, kind), in_place)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("B,k,G", [(19, 16, 16), (24, 16, 16), (13, 32, 5), (20, 16, 33), (60, 32, 16)])
def test_lists_of_many_requests(B, k, G, e4m3):
    """Clusters of 3, 2 and 1 CTAs, also with the mass of 32 blocks."""
    import sparse_attention_decode_gb300 as msa
    w = sparse.make(53, [300 + 290 * i % 4700 for i in range(B)], 1, 4, G, 4, k, "hnd", e4m3)
    assert sparse.verify(msa, w) == 0


def test_mass_and_weights_agree_with_the_accumulated_sums():
    """What attention reports as mass is what accumulation adds: over all blocks of a row it sums to the head group."""
    import sparse_attention_decode_gb300 as msa
    w = sparse.make(54, [900, 1500], 2, 2, 12, 2, 12, "hnd", False)
    mass = sparse.call(msa, w)[2]
    weights = torch.zeros(2, 2, 12, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_cache_accumulate(weights, w["ids"].cuda(), mass, ws, q_len=2)
    assert msa.msa_indexer_get_error(ws) == 0
    np.testing.assert_allclose(weights.sum(2).cpu().numpy(), 2 * 12, rtol=2e-5)

"""Attention over selected blocks of an E4M3 cache whose V scales differ by many powers of two: any finite scale >= 0."""

import pytest

from test_gpu_attention_sparse import PAGE, make, verify

pytestmark = pytest.mark.gpu

SHAPES = [([1500, 900], 1, 4, 16, 4, 16, "hnd"), ([700, 130], 3, 2, 32, 1, 7, "nhd"), ([1100], 2, 1, 64, 1, 9, "hnd")]


@pytest.mark.parametrize("tiny", [1e-38, 2e-39, 1e-40, 1e-45])
@pytest.mark.parametrize("shape", SHAPES, ids=["g16", "g32", "g64"])
def test_scales_next_to_zero(shape, tiny):
    """Half of every page has scales next to zero (a floor under a run of empty tokens); the others carry the rows."""
    import sparse_attention_decode_gb300 as msa
    w = make(41, *shape, True)
    w["vs"][:, :, :PAGE // 2] = tiny
    assert verify(msa, w) == 0
    w["vs"][:] = tiny  # and every token of the cache
    assert verify(msa, w) == 0


def test_a_scale_of_zero_everywhere():
    import sparse_attention_decode_gb300 as msa
    w = make(42, *SHAPES[0], True)
    w["vs"][:] = 0.0
    assert verify(msa, w) == 0

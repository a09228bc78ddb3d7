"""Attention over selected blocks of an E4M3 cache whose V scales differ by many powers of two: any finite scale >= 0."""

import pytest
import torch

from test_gpu_attention_sparse import D, PAGE, make, verify

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


def unattended(shape, factor):
    """A token in every eighth place whose score is far below all others and whose V scale is `factor` times theirs."""
    w = make(43, *shape, True)
    up = torch.nn.functional.normalize(torch.randn(D, generator=torch.Generator().manual_seed(2)), dim=0)
    w["q"] = (w["q"].float() + 6 * up).to(torch.bfloat16)
    low = (up * -1500).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for pool, code in ((w["kp"], low), (w["vp"], None)):
        for page in range(pool.shape[0]):
            for t in range(3, PAGE, 8):
                if int(pool[page, t, 0, 0]) != 0x7F and code is not None:  # (0x7F: past a request's last token)
                    pool[page, t] = code
    w["ks"][:, :, 3::8] = 1.0
    w["vs"][:, :, 3::8] *= factor
    return w


@pytest.mark.parametrize("factor", [1e6, 1e12, 1e25])
@pytest.mark.parametrize("shape", SHAPES, ids=["g16", "g32", "g64"])
def test_a_large_scale_without_weight_takes_nothing_from_the_others(shape, factor):
    import sparse_attention_decode_gb300 as msa
    assert verify(msa, unattended(shape, factor)) == 0


def test_each_row_keeps_its_own_range():
    """One row's heaviest token has a scale 2^30 times that of another row's: both keep their precision."""
    import sparse_attention_decode_gb300 as msa
    w = make(44, [1000], 1, 1, 16, 1, 8, "hnd", True)
    g = torch.Generator().manual_seed(3)
    up = torch.nn.functional.normalize(torch.randn(D, generator=g), dim=0)
    sign = torch.ones(16)
    sign[::2] = -1.0  # even rows look away from the marked tokens, odd rows at them
    w["q"] = (w["q"].float() + 6 * sign[None, :, None] * up).to(torch.bfloat16)
    code = (up * 1000).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for page in range(w["kp"].shape[0]):
        for t in range(5, 100, 16):
            w["kp"][page, t] = code
    w["ks"][:, :, 5:100:16] = 1.0
    w["vs"][:, :, 5:100:16] *= 2.0 ** 30
    assert verify(msa, w) == 0


def test_a_running_maximum_that_leaves_large_scales_behind():
    """Scores grow along the pages while the scales fall: what the first pages carried fades by 2^-40 a page."""
    import sparse_attention_decode_gb300 as msa
    w = make(45, [1000], 1, 1, 16, 1, 8, "hnd", True)
    up = torch.nn.functional.normalize(torch.randn(D, generator=torch.Generator().manual_seed(4)), dim=0)
    w["q"] = (w["q"].float() + 6 * up).to(torch.bfloat16)
    for j in range(8):
        page = int(w["table"][0, j])
        code = (up * (40.0 * j)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        w["kp"][page, :100] = code
        w["ks"][page] = 1.0
        w["vs"][page] *= 2.0 ** (30 - 10 * j)
    w["ids"][0, 0] = torch.arange(8)
    assert verify(msa, w) == 0


def test_the_largest_scales():
    """Codes of at most 1 beside scales up to 2^127: the outputs are finite still."""
    import sparse_attention_decode_gb300 as msa
    w = make(46, *SHAPES[0], True)
    lens, table = w["lens"], w["table"]
    v = (torch.rand(w["vp"].shape, generator=torch.Generator().manual_seed(5)) * 2 - 1).to(torch.float8_e4m3fn)
    w["vp"] = v.view(torch.uint8)
    for b, n in enumerate(lens):  # past the last token: NaN
        w["vp"][int(table[b, n // PAGE]), n % PAGE:] = 0x7F
    w["vs"][:] = 2.0 ** 126
    w["vs"][:, :, ::3] = 1.9 * 2.0 ** 126
    assert verify(msa, w) == 0

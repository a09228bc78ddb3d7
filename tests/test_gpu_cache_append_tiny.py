"""Norms of tiny heads, of heads of zeros and with an eps of 0: the formula in 64 bits, without what underflows in fp32."""

import pytest
import torch

import test_gpu_cache_append as append

pytestmark = pytest.mark.gpu

FORMULA = append.plain
SIZES = [0.0, 1e-10, 1e-16, 1e-22, 1e-25, 1e-30, 1e-37, 3e-39]  # (the last: bf16 without a leading 1)


def at_eps(monkeypatch, eps):
    """append.verify with this eps; heads of zeros are zero."""
    def plain(x, weight, _, *more):
        y, tol = FORMULA(x, weight, eps, *more)
        nothing = (x == 0).all(-1, keepdim=True)
        return torch.where(nothing, torch.zeros_like(y), y), torch.where(nothing, torch.zeros_like(tol), tol)
    monkeypatch.setattr(append, "plain", plain)


def sized(w, g):
    """Every head of a size of its own; one head with values of all sizes."""
    x = torch.randn(w["x"].shape, generator=g, dtype=torch.float64).clamp(-3, 3)
    size = torch.tensor(SIZES, dtype=torch.float64)[torch.randint(0, len(SIZES), x.shape[:2], generator=g)]
    x *= size[..., None]
    x[0, 0] = torch.logspace(-38, -17, 128, dtype=torch.float64)
    x[-1, -1] = 0.0
    w["x"] = x.to(torch.bfloat16)
    return w


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-30, 1e-25, 1e-24, 1e-6])
@pytest.mark.parametrize("inter", [False, True], ids=["halves", "interleaved"])
@pytest.mark.parametrize("rows", [6, 200], ids=["few", "many"])
def test_norms_of_tiny_heads(monkeypatch, rows, inter, eps):
    import sparse_attention_decode_gb300 as msa
    w = sized(append.make(81, [rows + 50], [rows], 3, 20, 64, inter, True, "hnd", False), torch.Generator().manual_seed(82))
    at_eps(monkeypatch, eps)
    got = append.call(msa, w, eps=eps)
    assert got["fault"] == 0 and bool(got["q"].isfinite().all())
    append.verify(w, got)


@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("rows", [6, 200], ids=["few", "many"])
def test_norms_of_tiny_heads_e4m3(monkeypatch, rows, eps):
    """Values below 2^-117 are zero by definition: they are of ordinary size here."""
    import sparse_attention_decode_gb300 as msa
    w = sized(append.make(83, [rows + 50], [rows], 2, 22, 128, False, True, "nhd", True), torch.Generator().manual_seed(84))
    w["x"][:, 24:] = torch.randn(rows, 2, 128, generator=torch.Generator().manual_seed(85)).to(torch.bfloat16)
    w["kw"] = w["kw"] + 0.5
    at_eps(monkeypatch, eps)
    if eps:  # a key whose eps outweighs it by far would be below 2^-117 again
        w["x"][:, 22:24] = torch.where(w["x"][:, 22:24].abs().amax(-1, keepdim=True) < 1e-24, torch.zeros(()).bfloat16(),
                                       w["x"][:, 22:24])
    got = append.call(msa, w, eps=eps)
    assert got["fault"] == 0
    append.verify(w, got)


def test_one_weight_alone(monkeypatch):
    """Keys with a norm, queries without: these are taken as they are, however small."""
    import sparse_attention_decode_gb300 as msa
    w = sized(append.make(86, [40], [9], 2, 6, 32, False, True, "hnd", False), torch.Generator().manual_seed(87))
    w["qw"] = None
    at_eps(monkeypatch, 0.0)
    got = append.call(msa, w, eps=0.0)
    assert got["fault"] == 0
    append.verify(w, got)

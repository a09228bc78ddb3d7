"""The largest sizes of the operators around the indexer, and many small ones."""

import math

import pytest
import torch

import test_gpu_attention_paged as paged
import test_gpu_cache_append as append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("case", [([200, 64, 63, 0, 1], 64, 1, 64), ([70, 300], 1, 40, 3), ([129, 500, 2], 64, 2, 1),
                                  ([300], 33, 1, 31)], ids=lambda c: f"q{c[1]}h{c[2]}g{c[3]}")
def test_attention_of_many_rows_and_heads(case, e4m3):
    import sparse_attention_decode_gb300 as msa
    lens, q_len, H, G = case
    assert paged.verify(msa, paged.make(101, lens, q_len, H, G, "nhd", e4m3)) == 0


def test_attention_of_the_largest_batch():
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator().manual_seed(102)
    lens = torch.randint(0, 40, (4096,), generator=g).tolist()
    w = paged.make(102, lens, 1, 1, 2, "hnd", False)
    assert paged.verify(msa, w) == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("eps", [1e-5, 0.0])
def test_append_of_many_heads(monkeypatch, e4m3, eps):
    import sparse_attention_decode_gb300 as msa
    formula = append.plain
    monkeypatch.setattr(append, "plain", lambda x, w, _, *more: formula(x, w, eps, *more))
    w = append.make(103, [3, 140], [2, 2], 1024, 2500, 64, False, True, "nhd", e4m3)
    got = append.call(msa, w, eps=eps)
    assert got["fault"] == 0
    append.verify(w, got)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_append_of_the_largest_batch(e4m3):
    """4096 requests with a row each, half of them padded."""
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator().manual_seed(104)
    lens = (torch.randint(1, 30, (4096,), generator=g) * torch.randint(0, 2, (4096,), generator=g)).tolist()
    w = append.make(104, lens, [1] * 4096, 1, 3, 32, True, True, "hnd", e4m3)
    got = append.call(msa, w)
    assert got["fault"] == 0
    append.verify(w, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("R,V", [(2, 1 << 24), (40, 1 << 20), (200000, 3), (1, 1)])
def test_log_probabilities_of_long_rows_and_of_many(R, V, dtype):
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator(device="cuda").manual_seed(105)
    x = torch.randn(R, V, device="cuda", generator=g).mul_(2.0).to(dtype)
    n = min(V, 32)
    tokens = torch.randint(0, V, (R, 2), device="cuda", generator=g, dtype=torch.int32)
    out, ent, top = torch.zeros(R, 2, device="cuda"), torch.zeros(R, device="cuda"), torch.zeros(R, n, device="cuda")
    ids, ws = torch.zeros(R, n, dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_token_logprobs(x, tokens, out, ws, out_entropy=ent, out_top_ids=ids, out_top_logprobs=top)
    assert msa.msa_indexer_get_error(ws) == 0
    for r0 in range(0, R, 20000):
        at = slice(r0, r0 + 20000)
        z = x[at].double()
        z -= z.logsumexp(1, keepdim=True)
        # as in test_gpu_token_logprobs: terms by (|y| + 3) 2^-23 with |y| below 40, sums by 2^-17, and the entropy's by |y| as much
        tol = 40 * 2.0 ** -23 + 2.0 ** -17
        order = torch.sort(-x[at].float(), dim=1, stable=True).indices[:, :n]
        assert torch.equal(ids[at].long(), order)
        for got, want in ((out[at], z.gather(1, tokens[at].long())), (top[at], z.gather(1, order))):
            assert float(((got.double() - want).abs() - 2.0 ** -22 * want.abs()).max()) <= tol
        entropy = -(z.exp() * z).sum(1)
        assert float((ent[at].double() - entropy).abs().max()) <= 40 * tol + 2.0 ** -22 * math.log(V + 1)

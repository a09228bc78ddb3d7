"""Calls from host threads that have made no CUDA call before: they have no current context of their own yet."""

import threading

import pytest
import torch

import test_gpu_attention_prefix as prefix

pytestmark = pytest.mark.gpu

D = 128


def in_a_thread(body):
    raised = []

    def work():
        try:
            body()
        except Exception as e:  # handed to the test
            raised.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if raised:
        raise raised[0]


def test_attention():
    import sparse_attention_decode_gb300 as msa
    w = prefix.make(61, 700, [300, 20], 1, 2, 16, "hnd")
    want = prefix.call(msa, w)[0]
    kp, vp = (prefix.ref.to_cuda(w[n]) for n in ("kp", "vp"))
    q, shared, table = w["q"].cuda(), w["shared"].cuda(), w["table"].cuda()
    n = torch.tensor([700], dtype=torch.int32, device="cuda")
    seq = torch.tensor(w["lens"], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(msa.msa_attention_prefix_workspace_bytes(2, 32, 2, 128 * shared.numel()), dtype=torch.uint8, device="cuda")
    handle = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    in_a_thread(lambda: msa.msa_attention_prefix(q, kp, vp, shared, n, table, seq, out, ws, scale=w["scale"], stream=handle))
    assert torch.equal(out, want)
    ids = torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda")
    first, again = torch.zeros_like(q), torch.zeros_like(q)
    call = lambda to: msa.msa_attention_sparse(q, kp, vp, table, seq, ids, to, ws, scale=0.1, stream=handle)  # noqa: E731
    call(first)
    torch.cuda.synchronize()
    in_a_thread(lambda: call(again))
    assert torch.equal(first, again)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_indexer(e4m3):
    import sparse_attention_decode_gb300 as msa
    g = torch.Generator(device="cuda").manual_seed(62)
    B, k, limit = 2, 16, 2560
    q = torch.randn(B, 4, D, device="cuda", generator=g).to(torch.bfloat16)
    pool = torch.randn(40, 128, D, device="cuda", generator=g)
    pool = (pool * 50).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else pool.to(torch.bfloat16)
    scale = torch.full((40, 128), 0.02, device="cuda")
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(B, 20)
    seq = torch.tensor([2500, 1700], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    ws = msa.new_workspace(B, limit, k, device="cuda")
    pws = torch.zeros(msa.msa_indexer_prefill_workspace_bytes(B, limit), dtype=torch.uint8, device="cuda")
    handle = torch.cuda.current_stream().cuda_stream

    def decode(ids, scores):
        if e4m3:
            msa.msa_indexer_decode_fp8(q, pool, scale, table, seq, k, 1, 2, ids, scores, ws, max_model_len=limit, stream=handle)
        else:
            msa.msa_indexer_decode(q, pool, table, seq, k, 1, 2, ids, scores, ws, max_model_len=limit, stream=handle)

    def prefill(ids, scores):
        if e4m3:
            msa.msa_indexer_prefill_fp8(q, cu, pool, scale, table, seq, k, 1, 2, ids, scores, pws, max_model_len=limit,
                                        stream=handle)
        else:
            msa.msa_indexer_prefill(q, cu, pool, table, seq, k, 1, 2, ids, scores, pws, max_model_len=limit, stream=handle)

    for call in (decode, prefill):
        got = [(torch.zeros(B, 4, k, dtype=torch.int32, device="cuda"), torch.zeros(B, 4, k, device="cuda")) for _ in range(2)]
        call(*got[0])
        torch.cuda.synchronize()
        in_a_thread(lambda: call(*got[1]))
        assert all(torch.equal(a, b) for a, b in zip(*got))

"""Queries that the append writes between the rows of its inputs, over them, and in place."""

import pytest
import torch

import attention_ref as ref
import test_gpu_cache_append as append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [5, 200], ids=["few", "many"])
def test_queries_between_the_projection_s_rows(rows):
    """One tensor: a row's queries, keys, values, and room for the prepared queries."""
    import sparse_attention_decode_gb300 as msa
    w = append.make(91, [rows + 20], [rows], 2, 22, 64, False, True, "hnd", False)
    base = append.call(msa, w)
    wide = torch.full((rows, 26 + 22, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :26] = w["x"].cuda()
    kp, vp, ws = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), torch.zeros(256, dtype=torch.uint8, device="cuda")
    msa.msa_cache_append(wide[:, 22:24], wide[:, 24:26], kp, vp, w["table"].cuda(),
                         torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), ws, q=wide[:, :22], out_q=wide[:, 26:],
                         q_weight=w["qw"].cuda(), k_weight=w["kw"].cuda(), eps=1e-5, inv_freq=w["inv"].cuda(), q_len=rows)
    torch.cuda.synchronize()
    assert append.same(wide[:, 26:].cpu(), base["q"]) and append.same(wide[:, :26].cpu(), w["x"])
    assert append.same(kp.cpu(), base["kp"]) and append.same(vp.cpu(), base["vp"])


@pytest.mark.parametrize("rows", [3, 200], ids=["few", "many"])
def test_outputs_over_inputs_are_refused(rows):
    import sparse_attention_decode_gb300 as msa
    w = append.make(92, [rows + 20], [rows], 2, 22, 64, False, True, "hnd", False)
    x = w["x"].cuda()
    kp, vp, ws = ref.to_cuda(w["kp"]), ref.to_cuda(w["vp"]), torch.zeros(256, dtype=torch.uint8, device="cuda")
    seq, table = torch.tensor(w["lens"], dtype=torch.int32, device="cuda"), w["table"].cuda()

    def status(q, out_q, k=x[:, 22:24], v=x[:, 24:]):
        try:
            msa.msa_cache_append(k, v, kp, vp, table, seq, ws, q=q, out_q=out_q, q_len=rows)
        except msa.MsaError as e:
            return e.status
        return 0

    assert status(x[:, :22], x[:, 1:23]) == msa.MSA_ERR_INVALID_ARG       # a head on
    assert status(x[:, :22], x[:, 4:26]) == msa.MSA_ERR_INVALID_ARG
    assert status(x[:, 2:24], x[:, 2:24]) == msa.MSA_ERR_INVALID_ARG      # in place, over the keys
    assert status(x[:, 4:26], x[:, 4:26]) == msa.MSA_ERR_INVALID_ARG      # and the values
    assert append.same(x.cpu(), w["x"])
    assert status(x[:, :22], x[:, :22]) == 0

"""Empty batches and prefixes: tensors without elements have no address, and are no errors."""

import ctypes

import pytest
import torch

import test_attention_abi as abi
import test_gpu_attention_prefix as prefix

lib = abi.lib


def test_an_empty_batch_needs_no_pointers(lib):
    from sparse_attention_decode_gb300 import _attention as A
    st = A._Strides(4 * 128 * 128, 128, 128 * 128)
    assert A._fn("msa_attention_sparse")(None, 512, None, st, None, st, 10, None, 8, None, 0, 1, 4, 1, 1024, None, 4, 16, 1.0,
                                         None, None, None, None, 0, None) == 0
    assert A._fn("msa_attention_sparse_fp8")(None, 512, None, st, None, None, st, None, 10, None, 8, None, 0, 1, 4, 1, 1024,
                                             None, 4, 16, 1.0, None, None, None, None, 0, None) == 0
    assert A._fn("msa_attention_prefix")(None, 512, None, st, None, st, 10, None, None, 1000, None, 8, None, 0, 1, 4, 1, 1024,
                                         1.0, None, None, None, 0, None) == 0
    assert A._fn("msa_cache_accumulate")(None, 8, None, None, None, 0, 1, 2, 2, 3, None, 0, None) == 0
    assert A._fn("msa_cache_evict")(None, 8, None, None, 8, 0, 2, 1024, 4, 1, 2, None, 8, None, None, None, None, None, 0,
                                    None) == 0
    assert A._fn("msa_verify_draft")(None, 0, 400, 100, None, None, None, None, None, None, 0, 3, 100, None, None, None, None,
                                     0, None) == 0
    # sizes are looked at all the same
    assert A._fn("msa_cache_accumulate")(None, 8, None, None, None, 0, 1, 2, 2, 33, None, 0, None) == 2
    assert A._fn("msa_verify_draft")(None, 0, 400, 99, None, None, None, None, None, None, 0, 3, 100, None, None, None, None, 0,
                                     None) == 1


def test_an_empty_prefix_needs_no_table(lib):
    from sparse_attention_decode_gb300 import _attention as A
    if torch.cuda.is_available():
        pytest.skip("host-only check: never hand placeholder pointers to a process with a GPU")
    fake, st = ctypes.c_void_p(1 << 20), A._Strides(4 * 128 * 128, 128, 128 * 128)

    def call(table, bound):
        return A._fn("msa_attention_prefix")(fake, 512, fake, st, fake, st, 10, table, fake, bound, fake, 8, fake, 2, 1, 4, 1,
                                             1024, 1.0, fake, None, fake, 1 << 40, None)
    assert call(None, 1) == 1
    assert call(None, 0) == call(fake, 0) == 4  # past every check: there is no GPU here


@pytest.mark.gpu
def test_attention_over_own_tokens_alone():
    import sparse_attention_decode_gb300 as msa
    w = prefix.make(71, 0, [0, 1, 300, 129], 1, 2, 16, "hnd")
    w["shared"] = w["shared"][:0]
    assert prefix.verify(msa, w) == 0


@pytest.mark.gpu
def test_calls_on_an_empty_batch():
    import sparse_attention_decode_gb300 as msa
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    i32, bf16 = torch.int32, torch.bfloat16
    kv, ws = z(4, 128, 2, 128, dtype=bf16), z(256, dtype=torch.uint8)
    q, table, seq, ids = z(0, 8, 128, dtype=bf16), z(0, 5, dtype=i32), z(0, dtype=i32), z(0, 2, 3, dtype=i32)
    msa.msa_attention_sparse(q, kv, kv, table, seq, ids, q, ws, scale=0.1, q_len=2, out_mass=z(0, 2, 3))
    codes, scale = z(4, 128, 2, 128, dtype=torch.uint8), z(4, 2, 128)
    msa.msa_attention_sparse_fp8(q, codes, scale, codes, scale, table, seq, ids, q, ws, scale=0.1)
    pws = z(msa.msa_attention_prefix_workspace_bytes(0, 8, 2, 256), dtype=torch.uint8)
    msa.msa_attention_prefix(q, kv, kv, z(2, dtype=i32), z(1, dtype=i32), table, seq, q, pws, scale=0.1)
    msa.msa_cache_accumulate(z(0, 2, 5), ids, z(0, 2, 3), ws)
    msa.msa_cache_evict(table, seq, z(0, 2, 5), 4, 1, 2, table, seq, z(0, 2, 5), z(0, 5, dtype=i32), z(0, dtype=i32), ws)
    msa.msa_verify_draft(z(0, 3, 9), z(0, 2, 9), z(0, 2, dtype=i32), z(0, 2), z(0, 9), z(0, 3, dtype=i32), z(0, dtype=i32), ws)
    torch.cuda.synchronize()
    assert msa.msa_indexer_get_error(ws) == 0

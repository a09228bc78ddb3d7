"""Binding of the serving operators declared in include/msa_attention.h (argument marshalling only).

Like the indexer's calls: each function has the name of the C entry point it calls, takes torch CUDA tensors,
enqueues on the current stream (or ``stream=``) and raises MsaError on a bad status.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._binding import MSA_HEAD_DIM, MSA_PAGE_TOKENS, _check, _ptr, _stream_ptr, load

MSA_FAULT_BLOCK_ID = 0x10
MSA_FAULT_TOKEN = 0x20
MSA_MAX_GROUP = 64
MSA_MAX_CACHE_BLOCKS = 32768
MSA_MAX_DRAFT = 63

ATTENTION_EXPORTED = (
    "msa_attention_prefix",
    "msa_attention_prefix_workspace_bytes",
    "msa_attention_sparse",
    "msa_attention_sparse_fp8",
    "msa_cache_accumulate",
    "msa_cache_evict",
    "msa_verify_draft",
)

_Strides = ctypes.c_int64 * 3
_P, _i64, _int, _size, _f32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float)
_bound = {}


def _fn(name):
    """The C entry point with its argument types set (once)."""
    f = _bound.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes, f.restype = _ARGTYPES[name]
        _bound[name] = f
    return f


_ARGTYPES = {
    "msa_attention_prefix_workspace_bytes": ([_int, _int, _int, _int], _size),
    "msa_attention_prefix": ([_P, _i64, _P, _Strides, _P, _Strides, _i64, _P, _P, _int, _P, _i64, _P, _int, _int, _int,
                              _int, _int, _f32, _P, _P, _P, _size, _P], _int),
    "msa_attention_sparse": ([_P, _i64, _P, _Strides, _P, _Strides, _i64, _P, _i64, _P, _int, _int, _int, _int, _int,
                              _P, _int, _int, _f32, _P, _P, _P, _P, _size, _P], _int),
    "msa_attention_sparse_fp8": ([_P, _i64, _P, _Strides, _P, _P, _Strides, _P, _i64, _P, _i64, _P, _int, _int, _int,
                                  _int, _int, _P, _int, _int, _f32, _P, _P, _P, _P, _size, _P], _int),
    "msa_cache_accumulate": ([_P, _i64, _P, _P, _P, _int, _int, _int, _int, _int, _P, _size, _P], _int),
    "msa_cache_evict": ([_P, _i64, _P, _P, _i64, _int, _int, _int, _int, _int, _int, _P, _i64, _P, _P, _P, _P, _P,
                         _size, _P], _int),
    "msa_verify_draft": ([_P, _int, _i64, _i64, _P, _P, _P, _P, _P, _P, _int, _int, _int, _P, _P, _P, _P, _size, _P],
                         _int),
}


def _cache(pool, e4m3: bool, what: str):
    """Strides (page, token, head) of a cache [pages, 128, kv_heads, 128] in any memory order."""
    shape = pool.shape
    assert pool.element_size() == 1 if e4m3 else pool.dtype == torch.bfloat16, f"{what}: wrong type"
    assert len(shape) == 4 and shape[1] == MSA_PAGE_TOKENS and shape[3] == MSA_HEAD_DIM, \
        f"{what}: [pages, 128, kv_heads, 128]"
    s = pool.stride()
    assert s[3] == 1, f"{what}: the head dimension is contiguous"
    return _Strides(s[0], s[1], s[2])


def _queries(q, out, rows: int):
    assert q.dtype == torch.bfloat16 and q.dim() == 3 and q.shape[2] == MSA_HEAD_DIM, "q: bf16 [rows, heads, 128]"
    assert q.stride(2) == 1 and (q.stride(1) == MSA_HEAD_DIM or q.shape[1] == 1), "q: heads of a row are contiguous"
    assert q.shape[0] == rows, "q: batch * q_len rows"
    assert out.dtype == torch.bfloat16 and out.shape == q.shape and out.is_contiguous(), "out: bf16 like q, contiguous"
    return int(q.shape[1]), (q.stride(0) if rows > 1 else q.shape[1] * MSA_HEAD_DIM)


def _requests(block_table, seq_lens):
    assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.stride(1) == 1, \
        "block_table: int32 [batch, blocks]"
    assert seq_lens.dtype == torch.int32 and seq_lens.is_contiguous(), "seq_lens: int32 [batch]"
    batch = int(block_table.shape[0])
    assert seq_lens.shape == (batch,), "seq_lens: int32 [batch]"
    cols = int(block_table.shape[1])
    return batch, cols, (block_table.stride(0) if batch > 1 else cols)


def _f32_out(t, shape, what: str):
    assert t is None or (t.dtype == torch.float32 and tuple(t.shape) == shape and t.is_contiguous()), \
        f"{what}: fp32 {list(shape)}, contiguous"
    return _ptr(t)


def _ws(workspace):
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _sparse(name, q, k, k_scale, v, v_scale, block_table, seq_lens, ids, out, workspace, scale, q_len, max_model_len,
            out_lse, out_mass, stream):
    e4m3 = k_scale is not None
    ks, vs = _cache(k, e4m3, "k"), _cache(v, e4m3, "v")
    assert k.shape == v.shape, "k and v: one shape"
    pages, kv_heads = int(k.shape[0]), int(k.shape[2])
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    rows = batch * q_len
    heads, q_stride = _queries(q, out, rows)
    assert heads % kv_heads == 0, "q heads: a multiple of kv_heads"
    assert ids.dtype == torch.int32 and ids.dim() == 3 and ids.is_contiguous() and ids.shape[0] == rows, \
        "ids: int32 [rows, sel_heads, k], contiguous"
    sel, topk = int(ids.shape[1]), int(ids.shape[2])
    if e4m3:
        for s in (k_scale, v_scale):
            assert s.dtype == torch.float32 and s.is_contiguous() and \
                tuple(s.shape) == (pages, kv_heads, MSA_PAGE_TOKENS), "scales: fp32 [pages, kv_heads, 128], contiguous"
        cache = (k.data_ptr(), ks, k_scale.data_ptr(), v.data_ptr(), vs, v_scale.data_ptr())
    else:
        cache = (k.data_ptr(), ks, v.data_ptr(), vs)
    st = _fn(name)(q.data_ptr(), q_stride, *cache, pages, block_table.data_ptr(), bt_stride, seq_lens.data_ptr(),
                   batch, q_len, kv_heads, heads // kv_heads,
                   MSA_PAGE_TOKENS * cols if max_model_len is None else max_model_len, ids.data_ptr(), sel, topk,
                   scale, out.data_ptr(), _f32_out(out_lse, (rows, heads), "out_lse"),
                   _f32_out(out_mass, (rows, kv_heads, topk), "out_mass"), *_ws(workspace), _stream_ptr(stream))
    _check(st, name)


def msa_attention_sparse(q, k, v, block_table, seq_lens, ids, out, workspace, *, scale: float, q_len: int = 1,
                         max_model_len: Optional[int] = None, out_lse=None, out_mass=None, stream=None) -> None:
    """Attention of q [batch * q_len, heads, 128] over the blocks ids [batch * q_len, sel_heads, k] of a bf16 cache.

    ``k`` and ``v``: [pages, 128, kv_heads, 128] in any memory order whose last axis is contiguous (a head-major cache
    is passed as ``pool.permute(0, 2, 1, 3)``).  See include/msa_attention.h.
    """
    _sparse("msa_attention_sparse", q, k, None, v, None, block_table, seq_lens, ids, out, workspace, scale, q_len,
            max_model_len, out_lse, out_mass, stream)


def msa_attention_sparse_fp8(q, k, k_scale, v, v_scale, block_table, seq_lens, ids, out, workspace, *, scale: float,
                             q_len: int = 1, max_model_len: Optional[int] = None, out_lse=None, out_mass=None,
                             stream=None) -> None:
    """msa_attention_sparse on E4M3 codes with fp32 scales [pages, kv_heads, 128]."""
    _sparse("msa_attention_sparse_fp8", q, k, k_scale, v, v_scale, block_table, seq_lens, ids, out, workspace, scale,
            q_len, max_model_len, out_lse, out_mass, stream)


def _is(t, dtype, shape, what: str):
    assert t.dtype == dtype and tuple(t.shape) == shape and t.is_contiguous(), f"{what}: {dtype} {list(shape)}, contiguous"
    return t.data_ptr()


def msa_cache_accumulate(weights, ids, mass, workspace, *, q_len: int = 1, n_rows=None, stream=None) -> None:
    """Adds the mass of each request's first n_rows positions to weights [batch, kv_heads, blocks], in place.

    ``ids`` [batch * q_len, sel_heads, k] and ``mass`` [batch * q_len, kv_heads, k] as msa_attention_sparse takes and
    gives them.  See include/msa_attention.h.
    """
    batch, kv_heads, cols = (int(x) for x in weights.shape)
    rows, sel, topk = (int(x) for x in ids.shape)
    assert rows == batch * q_len, "ids: batch * q_len rows"
    st = _fn("msa_cache_accumulate")(
        _is(weights, torch.float32, (batch, kv_heads, cols), "weights"), cols,
        _is(ids, torch.int32, (rows, sel, topk), "ids"), _is(mass, torch.float32, (rows, kv_heads, topk), "mass"),
        None if n_rows is None else _is(n_rows, torch.int32, (batch,), "n_rows"), batch, q_len, kv_heads, sel, topk,
        *_ws(workspace), _stream_ptr(stream))
    _check(st, "msa_cache_accumulate")


def msa_cache_evict(block_table, seq_lens, weights, budget: int, n_sink: int, n_window: int, out_table, out_seq_lens,
                    out_weights, out_freed, out_n_freed, workspace, *, max_model_len: Optional[int] = None,
                    stream=None) -> None:
    """Brings every request to at most ``budget`` blocks, keeping sink, window and the largest summed weights.

    The new table, lengths and weights may be written over the old ones.  See include/msa_attention.h.
    """
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    o_batch, o_cols, o_stride = _requests(out_table, out_seq_lens)
    assert o_batch == batch and o_cols == cols, "out_table, out_seq_lens: like the inputs"
    kv_heads = int(weights.shape[1])
    shape = (batch, kv_heads, cols)
    st = _fn("msa_cache_evict")(
        block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), _is(weights, torch.float32, shape, "weights"), cols,
        batch, kv_heads, MSA_PAGE_TOKENS * cols if max_model_len is None else max_model_len, budget, n_sink, n_window,
        out_table.data_ptr(), o_stride, out_seq_lens.data_ptr(),
        _is(out_weights, torch.float32, shape, "out_weights"), _is(out_freed, torch.int32, (batch, cols), "out_freed"),
        _is(out_n_freed, torch.int32, (batch,), "out_n_freed"), *_ws(workspace), _stream_ptr(stream))
    _check(st, "msa_cache_evict")


def msa_verify_draft(logits, draft_probs, draft_tokens, uniforms, race, out_tokens, out_accepted, workspace, *,
                     temperature=None, n_draft=None, out_logprobs=None, stream=None) -> None:
    """Accepts drafted tokens against softmax(logits / temperature) and draws the next one, from given random numbers.

    ``logits`` fp32 or bf16 [batch, drafts + 1, vocab] (rows of any stride), ``draft_probs`` fp32 [batch, drafts,
    vocab], ``race`` fp32 [batch, vocab] of Exp(1) draws.  See include/msa_attention.h.
    """
    assert logits.dim() == 3 and logits.dtype in (torch.float32, torch.bfloat16) and logits.stride(2) == 1, \
        "logits: fp32 or bf16 [batch, drafts + 1, vocab], rows contiguous"
    batch, rows, vocab = (int(x) for x in logits.shape)
    n = rows - 1
    stride = logits.stride()
    st = _fn("msa_verify_draft")(
        logits.data_ptr(), 1 if logits.dtype == torch.bfloat16 else 0, stride[0] if batch > 1 else rows * vocab,
        stride[1] if rows > 1 else vocab, _is(draft_probs, torch.float32, (batch, n, vocab), "draft_probs"),
        _is(draft_tokens, torch.int32, (batch, n), "draft_tokens"),
        _is(uniforms, torch.float32, (batch, n), "uniforms"), _is(race, torch.float32, (batch, vocab), "race"),
        None if temperature is None else _is(temperature, torch.float32, (batch,), "temperature"),
        None if n_draft is None else _is(n_draft, torch.int32, (batch,), "n_draft"), batch, n, vocab,
        _is(out_tokens, torch.int32, (batch, rows), "out_tokens"),
        _is(out_accepted, torch.int32, (batch,), "out_accepted"), _f32_out(out_logprobs, (batch, rows), "out_logprobs"),
        *_ws(workspace), _stream_ptr(stream))
    _check(st, "msa_verify_draft")


def msa_attention_prefix_workspace_bytes(max_rows: int, heads: int, kv_heads: int, max_prefix_len: int) -> int:
    return int(_fn("msa_attention_prefix_workspace_bytes")(max_rows, heads, kv_heads, max_prefix_len))


def msa_attention_prefix(q, k, v, prefix_table, prefix_len, block_table, seq_lens, out, workspace, *, scale: float,
                         q_len: int = 1, max_prefix_len: Optional[int] = None, max_model_len: Optional[int] = None,
                         out_lse=None, stream=None) -> None:
    """Attention of q [batch * q_len, heads, 128] over a shared prefix and each request's own tokens (bf16 cache).

    ``prefix_table`` int32 [pages], ``prefix_len`` an int32 tensor of one element on the GPU.  See
    include/msa_attention.h.
    """
    ks, vs = _cache(k, False, "k"), _cache(v, False, "v")
    assert k.shape == v.shape, "k and v: one shape"
    pages, kv_heads = int(k.shape[0]), int(k.shape[2])
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    rows = batch * q_len
    heads, q_stride = _queries(q, out, rows)
    assert heads % kv_heads == 0, "q heads: a multiple of kv_heads"
    assert prefix_table.dtype == torch.int32 and prefix_table.dim() == 1 and prefix_table.is_contiguous(), \
        "prefix_table: int32 [pages]"
    assert prefix_len.dtype == torch.int32 and prefix_len.numel() == 1, "prefix_len: int32 [1]"
    bound = MSA_PAGE_TOKENS * int(prefix_table.shape[0])
    assert max_prefix_len is None or max_prefix_len <= bound, "max_prefix_len: within prefix_table"
    st = _fn("msa_attention_prefix")(
        q.data_ptr(), q_stride, k.data_ptr(), ks, v.data_ptr(), vs, pages, prefix_table.data_ptr(),
        prefix_len.data_ptr(), bound if max_prefix_len is None else max_prefix_len, block_table.data_ptr(), bt_stride,
        seq_lens.data_ptr(), batch, q_len, kv_heads, heads // kv_heads,
        MSA_PAGE_TOKENS * cols if max_model_len is None else max_model_len, scale, out.data_ptr(),
        _f32_out(out_lse, (rows, heads), "out_lse"), *_ws(workspace), _stream_ptr(stream))
    _check(st, "msa_attention_prefix")

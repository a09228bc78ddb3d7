"""Binding of the operators declared in include/msa_serving.h (argument marshalling only), in the manner of _attention:
cache append, attention over all of a request's pages, token log probabilities."""

from __future__ import annotations

from typing import Optional

import torch

from . import _attention as _a
from ._attention import (_BF16, _F32, _I32, _P, _Strides, _caches, _f32, _i64, _int, _layout, _length_limit, _one_device,
                         _place, _ptr, _queries, _requests, _shapes, _size, _whole)
from ._binding import MSA_HEAD_DIM, MSA_PAGE_TOKENS, _check

MSA_MAX_ALTERNATIVES = 32
MSA_MAX_GIVEN_TOKENS = 256

SERVING_EXPORTED = (
    "msa_attention_paged",
    "msa_attention_paged_fp8",
    "msa_attention_paged_workspace_bytes",
    "msa_cache_append",
    "msa_cache_append_fp8",
    "msa_token_logprobs",
)

_APPEND = [_P, _i64, _int, _P, _i64, _P, _i64, _P, _i64, _int, _P, _P, _f32, _P, _int, _int, _P]
_APPEND_AT = [_i64, _P, _i64, _P, _P, _i64, _int, _int, _int, _P, _size, _P]
_ARGTYPES = {
    "msa_cache_append": (_APPEND + [_P, _Strides, _P, _Strides] + _APPEND_AT, _int),
    "msa_cache_append_fp8": (_APPEND + [_P, _Strides, _P, _P, _Strides, _P] + _APPEND_AT, _int),
    "msa_attention_paged_workspace_bytes": ([_int, _int, _int], _size),
    "msa_attention_paged": ([_P, _i64, _P, _Strides, _P, _Strides, _i64, _P, _i64, _P, _int, _int, _int, _int, _int, _f32,
                             _P, _P, _P, _size, _P], _int),
    "msa_attention_paged_fp8": ([_P, _i64, _P, _Strides, _P, _P, _Strides, _P, _i64, _P, _i64, _P, _int, _int, _int, _int,
                                 _int, _f32, _P, _P, _P, _size, _P], _int),
    "msa_token_logprobs": ([_P, _int, _i64, _P, _int, _P, _i64, _int, _int, _P, _P, _P, _P, _P, _size, _P], _int),
}
_a._ARGTYPES.update(_ARGTYPES)


def _new_rows(layout, heads: Optional[int], what: str):
    """Rows of new tokens [rows, heads, 128] whose heads are contiguous: (rows, heads, distance of rows)."""
    shape, s, t, _ = layout
    assert t == _BF16 and len(shape) == 3 and shape[2] == MSA_HEAD_DIM, f"{what}: bf16 [rows, heads, 128]"
    rows, n = int(shape[0]), int(shape[1])
    assert heads is None or n == heads, f"{what}: {heads} heads"
    assert s[2] == 1 and (s[1] == MSA_HEAD_DIM or n == 1), f"{what}: heads of a row are contiguous"
    return rows, n, (s[0] if rows > 1 else n * MSA_HEAD_DIM)


@_shapes
def _append_shapes(place, q, out_q, k, v, q_weight, k_weight, inv_freq, positions, k_cache, k_scale, v_cache, v_scale,
                   block_table, seq_lens, cu, q_len, max_model_len, e4m3):
    _one_device(place, q, out_q, k, v, q_weight, k_weight, inv_freq, positions, k_cache, k_scale, v_cache, v_scale,
                block_table, seq_lens, cu)
    assert (v is None) == (v_cache is None) and (q is None) == (out_q is None), "v with v_cache, q with out_q"
    assert not e4m3 or (k_scale is not None and (v is None) == (v_scale is None)), "E4M3: a scale for each cache"
    if v is None:
        ks, vs, pages, kv_heads = _a._cache(k_cache, e4m3, "k_cache"), _Strides(0, 0, 0), int(k_cache[0][0]), int(k_cache[0][2])
    else:
        ks, vs, pages, kv_heads = _caches(k_cache, v_cache, e4m3)
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    rows, _, k_stride = _new_rows(k, kv_heads, "k")
    v_stride = q_heads = q_stride = out_stride = 0
    if v is not None:
        assert v[0] == k[0], "k and v: one shape"
        v_stride = _new_rows(v, kv_heads, "v")[2]
    if q is not None:
        assert q[0] == out_q[0] and q[0][0] == rows, "q, out_q: [rows, heads, 128]"
        _, q_heads, q_stride = _new_rows(q, None, "q")
        out_stride = _new_rows(out_q, q_heads, "out_q")[2]
    if e4m3:
        _whole(k_scale, _F32, (pages, kv_heads, MSA_PAGE_TOKENS), "k_scale")
        if v is not None:
            _whole(v_scale, _F32, (pages, kv_heads, MSA_PAGE_TOKENS), "v_scale")
    _whole(q_weight, _F32, (MSA_HEAD_DIM,), "q_weight", True)
    _whole(k_weight, _F32, (MSA_HEAD_DIM,), "k_weight", True)
    pairs = 0 if inv_freq is None else int(inv_freq[0][0])
    _whole(inv_freq, _F32, (pairs,), "inv_freq", True)
    _whole(positions, _I32, (rows,), "positions", True)
    _whole(cu, _I32, (batch + 1,), "cu_seqlens_q", True)
    assert cu is not None or rows == batch * q_len, "k: batch * q_len rows"
    limit = _length_limit(cols, max_model_len)
    return (q_stride, q_heads, out_stride, k_stride, v_stride, kv_heads, 2 * pairs, ks, vs, pages, bt_stride,
            (rows, batch, q_len, limit))


def _append(name, k, v, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, workspace, q, out_q, q_weight,
            k_weight, eps, inv_freq, interleaved, positions, q_len, cu_seqlens_q, max_model_len, stream):
    e4m3 = name == "msa_cache_append_fp8"
    q_stride, q_heads, out_stride, k_stride, v_stride, kv_heads, rot, ks, vs, pages, bt_stride, sizes = _append_shapes(
        _place(workspace), _layout(q), _layout(out_q), _layout(k), _layout(v), _layout(q_weight), _layout(k_weight),
        _layout(inv_freq), _layout(positions), _layout(k_cache), _layout(k_scale), _layout(v_cache), _layout(v_scale),
        _layout(block_table), _layout(seq_lens), _layout(cu_seqlens_q), q_len, max_model_len, e4m3)
    if e4m3:
        cache = (k_cache.data_ptr(), ks, k_scale.data_ptr(), _ptr(v_cache), vs, _ptr(v_scale))
    else:
        cache = (k_cache.data_ptr(), ks, _ptr(v_cache), vs)
    st = _a._fn(name)(_ptr(q), q_stride, q_heads, _ptr(out_q), out_stride, k.data_ptr(), k_stride, _ptr(v), v_stride, kv_heads,
                      _ptr(q_weight), _ptr(k_weight), eps, _ptr(inv_freq), rot, 1 if interleaved else 0, _ptr(positions),
                      *cache, pages, block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), _ptr(cu_seqlens_q), *sizes,
                      workspace.data_ptr(), workspace.nbytes, _a._stream(stream, k))
    if st:
        _check(st, name)


def msa_cache_append(k, v, k_cache, v_cache, block_table, seq_lens, workspace, *, q=None, out_q=None, q_weight=None,
                     k_weight=None, eps: float = 1e-6, inv_freq=None, interleaved: bool = False, positions=None,
                     q_len: int = 1, cu_seqlens_q=None, max_model_len: Optional[int] = None, stream=None) -> None:
    """Writes the keys (normalised, rotated) and values of new tokens into a bf16 cache, and their queries to out_q.

    ``k``, ``v`` [rows, kv_heads, 128] (any distance of rows: slices of a projection's output), ``q`` and ``out_q``
    [rows, q_heads, 128]; ``k_cache``, ``v_cache`` [pages, 128, kv_heads, 128] in any memory order whose last axis is
    contiguous (an index-K cache [pages, 128, 128] is passed as ``pool.unsqueeze(2)`` with v and v_cache None).
    ``seq_lens`` count the new tokens: each request's last q_len ones, or those of ``cu_seqlens_q``.  ``inv_freq`` fp32
    [rotary_dim / 2].  See include/msa_serving.h.
    """
    _append("msa_cache_append", k, v, k_cache, None, v_cache, None, block_table, seq_lens, workspace, q, out_q, q_weight,
            k_weight, eps, inv_freq, interleaved, positions, q_len, cu_seqlens_q, max_model_len, stream)


def msa_cache_append_fp8(k, v, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, workspace, *, q=None, out_q=None,
                         q_weight=None, k_weight=None, eps: float = 1e-6, inv_freq=None, interleaved: bool = False,
                         positions=None, q_len: int = 1, cu_seqlens_q=None, max_model_len: Optional[int] = None,
                         stream=None) -> None:
    """msa_cache_append into E4M3 codes and fp32 scales [pages, kv_heads, 128]."""
    _append("msa_cache_append_fp8", k, v, k_cache, k_scale, v_cache, v_scale, block_table, seq_lens, workspace, q, out_q,
            q_weight, k_weight, eps, inv_freq, interleaved, positions, q_len, cu_seqlens_q, max_model_len, stream)


def msa_attention_paged_workspace_bytes(max_rows: int, heads: int, kv_heads: int) -> int:
    return int(_a._fn("msa_attention_paged_workspace_bytes")(max_rows, heads, kv_heads))


@_shapes
def _paged_shapes(place, q, k, k_scale, v, v_scale, block_table, seq_lens, out, lse, q_len, max_model_len):
    _one_device(place, q, k, k_scale, v, v_scale, block_table, seq_lens, out, lse)
    e4m3 = k_scale is not None
    ks, vs, pages, kv_heads = _caches(k, v, e4m3)
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    rows = batch * q_len
    heads, q_stride = _queries(q, out, rows, kv_heads)
    if e4m3:
        for scale in (k_scale, v_scale):
            _whole(scale, _F32, (pages, kv_heads, MSA_PAGE_TOKENS), "scales")
    _whole(lse, _F32, (rows, heads), "out_lse", True)
    limit = _length_limit(cols, max_model_len)
    return q_stride, ks, vs, pages, bt_stride, (batch, q_len, kv_heads, heads // kv_heads, limit)


def _paged(name, q, k, k_scale, v, v_scale, block_table, seq_lens, out, workspace, scale, q_len, max_model_len, out_lse,
           stream):
    q_stride, ks, vs, pages, bt_stride, sizes = _paged_shapes(
        _place(workspace), _layout(q), _layout(k), _layout(k_scale), _layout(v), _layout(v_scale), _layout(block_table),
        _layout(seq_lens), _layout(out), _layout(out_lse), q_len, max_model_len)
    if k_scale is None:
        cache = (k.data_ptr(), ks, v.data_ptr(), vs)
    else:
        cache = (k.data_ptr(), ks, k_scale.data_ptr(), v.data_ptr(), vs, v_scale.data_ptr())
    st = _a._fn(name)(q.data_ptr(), q_stride, *cache, pages, block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), *sizes,
                      scale, out.data_ptr(), _ptr(out_lse), workspace.data_ptr(), workspace.nbytes, _a._stream(stream, q))
    if st:
        _check(st, name)


def msa_attention_paged(q, k, v, block_table, seq_lens, out, workspace, *, scale: float, q_len: int = 1,
                        max_model_len: Optional[int] = None, out_lse=None, stream=None) -> None:
    """Attention of q [batch * q_len, heads, 128] over all tokens of each request (bf16 cache).

    ``k`` and ``v`` as msa_attention_sparse takes them; the workspace has msa_attention_paged_workspace_bytes bytes.
    See include/msa_serving.h.
    """
    _paged("msa_attention_paged", q, k, None, v, None, block_table, seq_lens, out, workspace, scale, q_len, max_model_len,
           out_lse, stream)


def msa_attention_paged_fp8(q, k, k_scale, v, v_scale, block_table, seq_lens, out, workspace, *, scale: float,
                            q_len: int = 1, max_model_len: Optional[int] = None, out_lse=None, stream=None) -> None:
    """msa_attention_paged on E4M3 codes with fp32 scales [pages, kv_heads, 128]."""
    _paged("msa_attention_paged_fp8", q, k, k_scale, v, v_scale, block_table, seq_lens, out, workspace, scale, q_len,
           max_model_len, out_lse, stream)


@_shapes
def _logprob_shapes(place, logits, tokens, out, temperature, entropy, ids, top):
    _one_device(place, logits, tokens, out, temperature, entropy, ids, top)
    shape, s, t, _ = logits
    assert len(shape) == 2 and t in (_F32, _BF16) and (s[1] == 1 or shape[1] == 1), \
        "logits: fp32 or bf16 [rows, vocab], rows contiguous"
    rows, vocab = int(shape[0]), int(shape[1])
    given = int(tokens[0][1])
    _whole(tokens, _I32, (rows, given), "tokens")
    _whole(out, _F32, (rows, given), "out_logprobs")
    _whole(temperature, _F32, (rows,), "temperature", True)
    _whole(entropy, _F32, (rows,), "out_entropy", True)
    assert (ids is None) == (top is None), "out_top_ids with out_top_logprobs"
    top_n = 0 if ids is None else int(ids[0][1])
    _whole(ids, _I32, (rows, top_n), "out_top_ids", True)
    _whole(top, _F32, (rows, top_n), "out_top_logprobs", True)
    return 1 if t == _BF16 else 0, (s[0] if rows > 1 else vocab), given, rows, vocab, top_n


def msa_token_logprobs(logits, tokens, out_logprobs, workspace, *, temperature=None, out_entropy=None, out_top_ids=None,
                       out_top_logprobs=None, stream=None) -> None:
    """Log probabilities of tokens [rows, given] under softmax(logits [rows, vocab] / temperature [rows]), the entropy,
    and the largest alternatives (out_top_ids, out_top_logprobs [rows, n]).  See include/msa_serving.h."""
    kind, stride, given, rows, vocab, top_n = _logprob_shapes(
        _place(workspace), _layout(logits), _layout(tokens), _layout(out_logprobs), _layout(temperature),
        _layout(out_entropy), _layout(out_top_ids), _layout(out_top_logprobs))
    st = _a._fn("msa_token_logprobs")(
        logits.data_ptr(), kind, stride, tokens.data_ptr(), given, _ptr(temperature), rows, vocab, top_n,
        out_logprobs.data_ptr(), _ptr(out_entropy), _ptr(out_top_ids), _ptr(out_top_logprobs), workspace.data_ptr(),
        workspace.nbytes, _a._stream(stream, logits))
    if st:
        _check(st, "msa_token_logprobs")

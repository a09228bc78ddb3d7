"""Binding of the serving operators declared in include/msa_attention.h (argument marshalling only).

Like the indexer's calls: each function has the name of the C entry point it calls, takes torch CUDA tensors,
enqueues on the current stream (or ``stream=``) of the current device, which the tensors have to be on, and raises
MsaError on a bad status.  A decode step makes these calls at the same shapes again and again, so what follows from
shapes, strides and types alone (the checks, and the numbers handed to C) is worked out once per combination;
addresses are read on every call.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._binding import MSA_HEAD_DIM, MSA_PAGE_TOKENS, _check, load

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
_F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16
_bound = {}
_shapes = functools.lru_cache(maxsize=1024)  # one entry a combination of shapes, strides and types

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


def _fn(name):
    """The C entry point with its argument types set (once)."""
    f = _bound.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes, f.restype = _ARGTYPES[name]
        _bound[name] = f
    return f


def _layout(t):
    """What a check may look at: (shape, stride, type, device number), or None."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _current_device() -> int:
    return torch._C._cuda_getDevice()


def _place(workspace):
    """Device number of a workspace; one with gaps, or on a device that is not the current one, has none."""
    place = workspace.get_device()
    return place if place >= 0 and workspace.is_contiguous() and place == _current_device() else -1


def _one_device(place, *layouts):
    """All tensors and the workspace on the current CUDA device, where C launches: another's address would be a fault."""
    devices = {x[3] for x in layouts if x is not None}
    assert devices == {place} and place >= 0, \
        "all tensors and a contiguous workspace on one CUDA device, the current one"


def _stream(stream, t):
    """The stream's handle; by default the current stream of t's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _whole(layout, dtype, shape, what: str, optional: bool = False):
    """A contiguous tensor of this type and shape."""
    if layout is None and optional:
        return
    got, stride, t, _ = layout
    want = 1
    for n, s in zip(reversed(got), reversed(stride)):
        assert n <= 1 or s == want or 0 in got, f"{what}: contiguous"
        want *= n
    assert t == dtype and tuple(got) == tuple(shape), f"{what}: {dtype} {list(shape)}, contiguous"


def _cache(layout, e4m3: bool, what: str):
    """Strides (page, token, head) of a cache [pages, 128, kv_heads, 128] in any memory order."""
    shape, s, t, _ = layout
    assert t in (torch.uint8, torch.float8_e4m3fn) if e4m3 else t == _BF16, f"{what}: wrong type"
    assert len(shape) == 4 and shape[1] == MSA_PAGE_TOKENS and shape[3] == MSA_HEAD_DIM, \
        f"{what}: [pages, 128, kv_heads, 128]"
    assert s[3] == 1, f"{what}: the head dimension is contiguous"
    return _Strides(s[0], s[1], s[2])


def _caches(k, v, e4m3: bool):
    assert k[0] == v[0], "k and v: one shape"
    return _cache(k, e4m3, "k"), _cache(v, e4m3, "v"), int(k[0][0]), int(k[0][2])


def _queries(q, out, rows: int, kv_heads: int):
    shape, s, t, _ = q
    assert t == _BF16 and len(shape) == 3 and shape[2] == MSA_HEAD_DIM, "q: bf16 [rows, heads, 128]"
    heads = int(shape[1])
    assert s[2] == 1 and (s[1] == MSA_HEAD_DIM or heads == 1), "q: heads of a row are contiguous"
    assert shape[0] == rows, "q: batch * q_len rows"
    assert heads % kv_heads == 0, "q heads: a multiple of kv_heads"
    _whole(out, _BF16, shape, "out")
    return heads, (s[0] if rows > 1 else heads * MSA_HEAD_DIM)


def _requests(block_table, seq_lens):
    shape, s, t, _ = block_table
    assert t == _I32 and len(shape) == 2 and (s[1] == 1 or shape[1] == 1), "block_table: int32 [batch, blocks]"
    batch, cols = int(shape[0]), int(shape[1])
    _whole(seq_lens, _I32, (batch,), "seq_lens")
    return batch, cols, (s[0] if batch > 1 else cols)


def _length_limit(cols: int, max_model_len: Optional[int]) -> int:
    """Tokens a request may have: a row of the table given ends after its columns, also inside a wider table."""
    tokens = MSA_PAGE_TOKENS * cols
    return tokens if max_model_len is None else min(tokens, max_model_len)


@_shapes
def _sparse_shapes(place, q, k, k_scale, v, v_scale, block_table, seq_lens, ids, out, lse, mass, q_len, max_model_len):
    _one_device(place, q, k, k_scale, v, v_scale, block_table, seq_lens, ids, out, lse, mass)
    e4m3 = k_scale is not None
    ks, vs, pages, kv_heads = _caches(k, v, e4m3)
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    rows = batch * q_len
    heads, q_stride = _queries(q, out, rows, kv_heads)
    assert len(ids[0]) == 3 and ids[0][0] == rows, "ids: int32 [batch * q_len, sel_heads, k]"
    sel, topk = int(ids[0][1]), int(ids[0][2])
    _whole(ids, _I32, (rows, sel, topk), "ids")
    if e4m3:
        for scale in (k_scale, v_scale):
            _whole(scale, _F32, (pages, kv_heads, MSA_PAGE_TOKENS), "scales")
    _whole(lse, _F32, (rows, heads), "out_lse", True)
    _whole(mass, _F32, (rows, kv_heads, topk), "out_mass", True)
    limit = _length_limit(cols, max_model_len)
    return q_stride, ks, vs, pages, bt_stride, (batch, q_len, kv_heads, heads // kv_heads, limit), sel, topk


def _sparse(name, q, k, k_scale, v, v_scale, block_table, seq_lens, ids, out, workspace, scale, q_len, max_model_len,
            out_lse, out_mass, stream):
    q_stride, ks, vs, pages, bt_stride, sizes, sel, topk = _sparse_shapes(
        _place(workspace), _layout(q), _layout(k), _layout(k_scale), _layout(v), _layout(v_scale), _layout(block_table),
        _layout(seq_lens), _layout(ids), _layout(out), _layout(out_lse), _layout(out_mass), q_len, max_model_len)
    if k_scale is None:
        cache = (k.data_ptr(), ks, v.data_ptr(), vs)
    else:
        cache = (k.data_ptr(), ks, k_scale.data_ptr(), v.data_ptr(), vs, v_scale.data_ptr())
    st = _fn(name)(q.data_ptr(), q_stride, *cache, pages, block_table.data_ptr(), bt_stride, seq_lens.data_ptr(),
                   *sizes, ids.data_ptr(), sel, topk, scale, out.data_ptr(), _ptr(out_lse), _ptr(out_mass),
                   workspace.data_ptr(), workspace.nbytes, _stream(stream, q))
    if st:
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


@_shapes
def _accumulate_shapes(place, weights, ids, mass, n_rows, q_len):
    _one_device(place, weights, ids, mass, n_rows)
    batch, kv_heads, cols = (int(x) for x in weights[0])
    rows, sel, topk = (int(x) for x in ids[0])
    assert rows == batch * q_len, "ids: batch * q_len rows"
    _whole(weights, _F32, (batch, kv_heads, cols), "weights")
    _whole(ids, _I32, (rows, sel, topk), "ids")
    _whole(mass, _F32, (rows, kv_heads, topk), "mass")
    _whole(n_rows, _I32, (batch,), "n_rows", True)
    return cols, (batch, q_len, kv_heads, sel, topk)


def msa_cache_accumulate(weights, ids, mass, workspace, *, q_len: int = 1, n_rows=None, stream=None) -> None:
    """Adds the mass of each request's first n_rows positions to weights [batch, kv_heads, blocks], in place.

    ``ids`` [batch * q_len, sel_heads, k] and ``mass`` [batch * q_len, kv_heads, k] as msa_attention_sparse takes and
    gives them.  See include/msa_attention.h.
    """
    cols, sizes = _accumulate_shapes(
        _place(workspace), _layout(weights), _layout(ids), _layout(mass), _layout(n_rows), q_len)
    st = _fn("msa_cache_accumulate")(weights.data_ptr(), cols, ids.data_ptr(), mass.data_ptr(), _ptr(n_rows), *sizes,
                                     workspace.data_ptr(), workspace.nbytes, _stream(stream, weights))
    if st:
        _check(st, "msa_cache_accumulate")


@_shapes
def _evict_shapes(place, block_table, seq_lens, weights, out_table, out_seq_lens, out_weights, out_freed, out_n_freed,
                  max_model_len):
    _one_device(place, block_table, seq_lens, weights, out_table, out_seq_lens, out_weights, out_freed, out_n_freed)
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    o_batch, o_cols, o_stride = _requests(out_table, out_seq_lens)
    assert o_batch == batch and o_cols == cols, "out_table, out_seq_lens: like the inputs"
    shape = (batch, int(weights[0][1]), cols)
    _whole(weights, _F32, shape, "weights")
    _whole(out_weights, _F32, shape, "out_weights")
    _whole(out_freed, _I32, (batch, cols), "out_freed")
    _whole(out_n_freed, _I32, (batch,), "out_n_freed")
    limit = _length_limit(cols, max_model_len)
    return bt_stride, o_stride, (cols, batch, shape[1], limit)


def msa_cache_evict(block_table, seq_lens, weights, budget: int, n_sink: int, n_window: int, out_table, out_seq_lens,
                    out_weights, out_freed, out_n_freed, workspace, *, max_model_len: Optional[int] = None,
                    stream=None) -> None:
    """Brings every request to at most ``budget`` blocks, keeping sink, window and the largest summed weights.

    The new table, lengths and weights may be written over the old ones.  See include/msa_attention.h.
    """
    bt_stride, o_stride, sizes = _evict_shapes(
        _place(workspace),
        _layout(block_table), _layout(seq_lens), _layout(weights), _layout(out_table), _layout(out_seq_lens),
        _layout(out_weights), _layout(out_freed), _layout(out_n_freed), max_model_len)
    st = _fn("msa_cache_evict")(
        block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), weights.data_ptr(), *sizes, budget, n_sink, n_window,
        out_table.data_ptr(), o_stride, out_seq_lens.data_ptr(), out_weights.data_ptr(), out_freed.data_ptr(),
        out_n_freed.data_ptr(), workspace.data_ptr(), workspace.nbytes, _stream(stream, block_table))
    if st:
        _check(st, "msa_cache_evict")


@_shapes
def _verify_shapes(place, logits, draft, tokens, uniforms, race, out, accepted, temperature, n_draft, logprobs):
    _one_device(place, logits, draft, tokens, uniforms, race, out, accepted, temperature, n_draft, logprobs)
    shape, stride, dtype, _ = logits
    assert len(shape) == 3 and dtype in (_F32, _BF16) and stride[2] == 1, \
        "logits: fp32 or bf16 [batch, drafts + 1, vocab], rows contiguous"
    batch, rows, vocab = (int(x) for x in shape)
    n = rows - 1
    _whole(draft, _F32, (batch, n, vocab), "draft_probs")
    _whole(tokens, _I32, (batch, n), "draft_tokens")
    _whole(uniforms, _F32, (batch, n), "uniforms")
    _whole(race, _F32, (batch, vocab), "race")
    _whole(temperature, _F32, (batch,), "temperature", True)
    _whole(n_draft, _I32, (batch,), "n_draft", True)
    _whole(out, _I32, (batch, rows), "out_tokens")
    _whole(accepted, _I32, (batch,), "out_accepted")
    _whole(logprobs, _F32, (batch, rows), "out_logprobs", True)
    return (1 if dtype == _BF16 else 0, stride[0] if batch > 1 else rows * vocab, stride[1] if rows > 1 else vocab), \
        (batch, n, vocab)


def msa_verify_draft(logits, draft_probs, draft_tokens, uniforms, race, out_tokens, out_accepted, workspace, *,
                     temperature=None, n_draft=None, out_logprobs=None, stream=None) -> None:
    """Accepts drafted tokens against softmax(logits / temperature) and draws the next one, from given random numbers.

    ``logits`` fp32 or bf16 [batch, drafts + 1, vocab] (rows of any stride), ``draft_probs`` fp32 [batch, drafts,
    vocab], ``race`` fp32 [batch, vocab] of Exp(1) draws.  See include/msa_attention.h.
    """
    kind, sizes = _verify_shapes(
        _place(workspace),
        _layout(logits), _layout(draft_probs), _layout(draft_tokens), _layout(uniforms), _layout(race),
        _layout(out_tokens), _layout(out_accepted), _layout(temperature), _layout(n_draft), _layout(out_logprobs))
    st = _fn("msa_verify_draft")(
        logits.data_ptr(), *kind, draft_probs.data_ptr(), draft_tokens.data_ptr(), uniforms.data_ptr(),
        race.data_ptr(), _ptr(temperature), _ptr(n_draft), *sizes, out_tokens.data_ptr(), out_accepted.data_ptr(),
        _ptr(out_logprobs), workspace.data_ptr(), workspace.nbytes, _stream(stream, logits))
    if st:
        _check(st, "msa_verify_draft")


def msa_attention_prefix_workspace_bytes(max_rows: int, heads: int, kv_heads: int, max_prefix_len: int) -> int:
    return int(_fn("msa_attention_prefix_workspace_bytes")(max_rows, heads, kv_heads, max_prefix_len))


@_shapes
def _prefix_shapes(place, q, k, v, prefix_table, prefix_len, block_table, seq_lens, out, lse, q_len, max_prefix_len,
                   max_model_len):
    _one_device(place, q, k, v, prefix_table, prefix_len, block_table, seq_lens, out, lse)
    ks, vs, pages, kv_heads = _caches(k, v, False)
    batch, cols, bt_stride = _requests(block_table, seq_lens)
    rows = batch * q_len
    heads, q_stride = _queries(q, out, rows, kv_heads)
    _whole(prefix_table, _I32, (prefix_table[0][0],), "prefix_table")
    _whole(prefix_len, _I32, (1,), "prefix_len")
    bound = MSA_PAGE_TOKENS * int(prefix_table[0][0])
    assert max_prefix_len is None or max_prefix_len <= bound, "max_prefix_len: within prefix_table"
    _whole(lse, _F32, (rows, heads), "out_lse", True)
    limit = _length_limit(cols, max_model_len)
    return (q_stride, ks, vs, pages, bound if max_prefix_len is None else max_prefix_len, bt_stride,
            (batch, q_len, kv_heads, heads // kv_heads, limit))


def msa_attention_prefix(q, k, v, prefix_table, prefix_len, block_table, seq_lens, out, workspace, *, scale: float,
                         q_len: int = 1, max_prefix_len: Optional[int] = None, max_model_len: Optional[int] = None,
                         out_lse=None, stream=None) -> None:
    """Attention of q [batch * q_len, heads, 128] over a shared prefix and each request's own tokens (bf16 cache).

    ``prefix_table`` int32 [pages], ``prefix_len`` an int32 tensor of one element on the GPU.  See
    include/msa_attention.h.
    """
    q_stride, ks, vs, pages, bound, bt_stride, sizes = _prefix_shapes(
        _place(workspace),
        _layout(q), _layout(k), _layout(v), _layout(prefix_table), _layout(prefix_len), _layout(block_table),
        _layout(seq_lens), _layout(out), _layout(out_lse), q_len, max_prefix_len, max_model_len)
    st = _fn("msa_attention_prefix")(
        q.data_ptr(), q_stride, k.data_ptr(), ks, v.data_ptr(), vs, pages, prefix_table.data_ptr(),
        prefix_len.data_ptr(), bound, block_table.data_ptr(), bt_stride, seq_lens.data_ptr(), *sizes, scale,
        out.data_ptr(), _ptr(out_lse), workspace.data_ptr(), workspace.nbytes, _stream(stream, q))
    if st:
        _check(st, "msa_attention_prefix")

"""Operators that bring prompts and trees of drafts into the serving step:
causal attention over packed prompts, pages and slots of the paged KV cache kept
on the GPU, the writing of keys and values to them, attention of a tree of
drafted tokens over the cache and the tree's greedy verification (whose accepted
path :func:`kv_commit` takes).

As in :mod:`.operators` this only marshals arguments: calls are asynchronous on
``stream`` (default: the current stream), allocate only their outputs and, once
per stream, a workspace, may come from any thread, are not recorded by autograd,
and leave data errors to the ``*_error`` functions.
"""

from __future__ import annotations

import collections
import ctypes
import math

import torch

from .operators import (_DTYPES, _INT_MAX, _KV, _P, _SIGNATURES, SV_HEAD_DIM_MAX, _attention_args,
                        _attention_out, _cache_desc, _empty, _error, _f32, _i32, _i64, _launch,
                        _matrix, _sz, _table, _vector)

SV_TREE_MAX_K = 63

Reservation = collections.namedtuple("Reservation",
                                     ["block_table", "held", "free_pages", "free_count"])
Slots = collections.namedtuple("Slots", ["slots", "request", "position", "offsets"])

_SIGNATURES.update({
    "spec_prompt_attention_workspace_size": (_sz, [_i32]),
    "spec_prompt_attention": (ctypes.c_int, [_P, _i64, _i64, _P, _i64, _i64, _P, _i64, _i64, _i32,
                                             _i64, _i32, _i32, _i32, _P, _f32, _i32, _P, _P, _P,
                                             _i32, _P, _sz]),
    "spec_tree_attention_workspace_size": (_sz, [_i32, _i32]),
    "spec_tree_attention": (ctypes.c_int, [_KV, _i32, _i32, _i32, _P, _i64, _i64, _i32, _i64, _P,
                                           _i32, _P, _P, _P, _P, _i32, _f32, _i32, _P, _P, _P,
                                           _i32, _P, _sz]),
    "spec_verify_tree_greedy_workspace_size": (_sz, [_i32]),
    "spec_verify_tree_greedy": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _i32, _i64, _i32,
                                               _P, _sz]),
    "spec_kv_reserve_workspace_size": (_sz, [_i32, _i64]),
    "spec_kv_reserve": (ctypes.c_int, [_P, _P, _i32, _P, _P, _P, _P, _P, _i64, _P, _P, _i32, _P,
                                       _i32, _P, _sz]),
    "spec_kv_slots_workspace_size": (_sz, [_i32, _i64]),
    "spec_kv_slots": (ctypes.c_int, [_P, _i32, _P, _P, _i64, _i32, _P, _P, _P, _P, _P, _i32, _P,
                                     _sz]),
    "spec_kv_write_workspace_size": (_sz, [_i64]),
    "spec_kv_write": (ctypes.c_int, [_KV, _i32, _i32, _P, _i64, _i64, _P, _i64, _i64, _P, _i64, _P,
                                     _P, _sz]),
})


def _heads(t, name, dtype, dev, rows=None):
    """A [rows, heads, D] tensor with contiguous heads; returns its address and strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
        raise TypeError(f"{name} must be a 3-D CUDA tensor")
    if t.dtype is not dtype or t.device != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on {dev}")
    rs, hs, one = t.stride()
    if t.shape[2] > 1 and one != 1:
        raise ValueError(f"the heads of {name} must be contiguous")
    if rows is not None and t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows")
    return t.data_ptr(), rs, hs


def prompt_attention(q, k, v, offsets, *, scale=None, window=0, out=None, out_lse=None,
                     stream=None):
    """Causal attention within each of the sequences that are packed in the rows.

    q: [rows, q_heads, D]; k, v: [rows, kv_heads, D] (bf16, fp16 or fp32; row and
    head strides are free, so that they may be slices of one projection);
    offsets: [B + 1] int32, sequence b having rows offsets[b] .. offsets[b + 1] - 1
    (:func:`kv_slots` gives them).  A token sees its sequence up to itself, with
    ``window`` > 0 only the last ``window`` tokens of that.

    Masked keys and values may be anything.  Infinite and NaN values reach the tokens
    that see them; where the type holds the weight of such a value as 0 (more than 2^126
    below the token's largest, 2^31 in fp16) the result is NaN.  A product of +inf makes
    its row NaN, a position of -inf weighs nothing.

    Returns ``(out [rows, q_heads, D], lse [rows, q_heads] float32)``; rows of no
    sequence are left as they were.  They carry no autograd history."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise TypeError("q must be a 3-D CUDA tensor")
    dtype, dev = q.dtype, q.device
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {dtype}")
    rows, Hq, D = q.shape
    q_args = _heads(q, "q", dtype, dev)
    k_args = _heads(k, "k", dtype, dev, rows)
    v_args = _heads(v, "v", dtype, dev, rows)
    Hk = k.shape[1]
    if k.shape != v.shape or k.shape[2] != D or Hk < 1 or Hq < 1 or Hq % Hk:
        raise ValueError(f"q of {Hq} heads of {D} does not fit k {tuple(k.shape)} and v "
                         f"{tuple(v.shape)}")
    if not 1 <= D <= SV_HEAD_DIM_MAX:
        raise ValueError(f"heads must have 1 to {SV_HEAD_DIM_MAX} elements")
    if window < 0:
        raise ValueError("window must be 0 (off) or positive")
    o_ptr = _vector(offsets, "offsets", torch.int32, 1, dev)
    B = offsets.numel() - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, out_lse = _attention_out(out, out_lse, rows, Hq, D, dtype, dev, stream)
    _launch("prompt_attention", dev, stream, (B if rows else 0,),
            (*q_args, *k_args, *v_args, code, rows, Hq, Hk, D, o_ptr, scale,
             min(window, _INT_MAX), out.data_ptr(), out_lse.data_ptr()), (B,))
    return out, out_lse


def tree_attention(q, cache, layer, kv_len, block_table, k_per_req, parent, spec, *, scale=None,
                   window=0, out=None, out_lse=None, stream=None):
    """Attention of every request's tree of drafted tokens over its paged cache.

    The arguments of :func:`attention`, with up to 63 drafts a request, and
    parent: [rows] int32, for every node (row) the earlier node of its request
    that it hangs from; node 0 is the last emitted token, whose parent is not
    read.  A node lies one position behind its parent, node 0 at kv_len, and sees
    the cached positions, its ancestors and itself, with ``window`` > 0 only the
    last ``window`` of them.  spec: [B, slots, n_layers, 2, E], entry j of node j.
    Where a row sees an infinite value whose weight is 0 in the type, its result may
    be NaN instead of infinite.

    Returns ``(out [rows, q_heads, D], lse [rows, q_heads] float32)``."""
    if spec is None:
        raise ValueError("spec is required")
    dev, dtype, B, rows, Hq, D, args = _attention_args(q, cache, layer, kv_len, block_table,
                                                       k_per_req, spec, scale, window)
    p_ptr = _vector(parent, "parent", torch.int32, rows, dev)
    out, out_lse = _attention_out(out, out_lse, rows, Hq, D, dtype, dev, stream)
    # parent comes behind k_per_req
    _launch("tree_attention", dev, stream, (B, D),
            (*args[:12], p_ptr, *args[12:], out.data_ptr(), out_lse.data_ptr()), (B,))
    return out, out_lse


def verify_tree_greedy(target_argmax, draft_tokens, parent, k_per_req, vocab, *,
                       out_accept_len=None, out_tokens=None, out_path=None, stream=None):
    """Greedy verification of trees of drafts from the target rows' argmax.

    target_argmax, parent: [rows] int32, rows = sum(k_per_req) + B in the layout of
    the verifier's target rows, row t_off[b] + j being node j (:func:`tree_attention`);
    draft_tokens: [rows - B] int32, the tokens of nodes 1 .. k_b; k_per_req: [B]
    int32.  From node 0 on the walk goes to the child whose token is the argmax at
    the node (the lowest such child) until there is none.

    Returns ``(accept_len [B], tokens [rows], path [rows])`` int32: the accepted
    tokens and the argmax at the last node, and the nodes of the walk, both followed
    by -1; accept_len -1 for requests that failed.  :func:`kv_commit` takes the path."""
    if not isinstance(target_argmax, torch.Tensor) or not target_argmax.is_cuda:
        raise TypeError("target_argmax must be a CUDA tensor")
    dev, rows = target_argmax.device, target_argmax.numel()
    B = k_per_req.shape[0]
    if rows < B:
        raise ValueError(f"target_argmax has {rows} rows for {B} requests")
    if not 1 <= vocab <= _INT_MAX:
        raise ValueError("vocab must be positive and below 2^31")
    i32 = torch.int32
    ptrs = [_vector(target_argmax, "target_argmax", i32, rows, dev),
            _vector(draft_tokens, "draft_tokens", i32, rows - B, dev),
            _vector(parent, "parent", i32, rows, dev), _vector(k_per_req, "k_per_req", i32, B, dev)]
    outs = []
    for t, name, n in ((out_accept_len, "out_accept_len", B), (out_tokens, "out_tokens", rows),
                       (out_path, "out_path", rows)):
        if t is None:
            t = _empty((n,), i32, dev, stream)
        outs.append(t)
        ptrs.append(_vector(t, name, i32, n, dev))
    _launch("verify_tree_greedy", dev, stream, (B,), ptrs, (B, rows, vocab))
    return tuple(outs)


def kv_reserve(block_table, held, lengths, free_pages, free_count, page_size, *, out_table=None,
               out_held=None, out_free=None, out_count=None, stream=None):
    """Give every request the pages for ``lengths[b]`` positions and take back what
    it holds beyond them.

    block_table: [B, max_pages] int32; held: [B] int32, the pages each request
    holds (the first entries of its row); lengths: [B] int32; free_pages:
    [capacity] int32, a stack of which the first ``free_count`` ([1] int32) are
    free.  Pages given back go onto the stack in the order of the requests, -1 takes
    their place in the table; requests that need more take pages off its end, one
    request after the other, as long as there are enough for all so far: the first
    request for which there are not, and those behind it that need any, keep what
    they hold (error SV_ERR_DATA_POOL).  A request with a missing page (below 0) among
    those it would give back keeps them all (SV_ERR_DATA_PAGE).  Without outputs
    everything is changed in place; an output of its own gets the whole new contents,
    also where there is no request.

    Returns a :class:`Reservation` (block_table, held, free_pages, free_count)."""
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda:
        raise TypeError("block_table must be a CUDA tensor")
    dev, i32 = block_table.device, torch.int32
    B = held.shape[0]
    if not 1 <= page_size <= _INT_MAX:
        raise ValueError("page_size must be positive and below 2^31")
    t_ptr, cols = _table(block_table, "block_table", B, dev)
    h_ptr = _vector(held, "held", i32, B, dev)
    l_ptr = _vector(lengths, "lengths", i32, B, dev)
    f_ptr = _vector(free_pages, "free_pages", i32, 0, dev)
    c_ptr = _vector(free_count, "free_count", i32, 1, dev)
    P = free_pages.numel()
    got = Reservation(block_table if out_table is None else out_table,
                      held if out_held is None else out_held,
                      free_pages if out_free is None else out_free,
                      free_count if out_count is None else out_count)
    ot_ptr, out_cols = _table(got.block_table, "out_table", B, dev)
    if out_cols != cols:
        raise ValueError(f"out_table must have {cols} columns")
    of_ptr = _vector(got.free_pages, "out_free", i32, P, dev)
    if got.free_pages.numel() != P:
        raise ValueError(f"out_free must have {P} elements")
    oc_ptr = _vector(got.free_count, "out_count", i32, 1, dev)
    # (without requests only a list or count of its own is written)
    work = B or int((f_ptr, c_ptr) != (of_ptr, oc_ptr))
    _launch("kv_reserve", dev, stream, (work, P),
            (t_ptr, ot_ptr, cols, h_ptr, _vector(got.held, "out_held", i32, B, dev), l_ptr, f_ptr,
             of_ptr, P, c_ptr, oc_ptr, page_size), (B,))
    return got


def kv_slots(block_table, start, count, rows, page_size, *, stream=None):
    """Where a step's new tokens go: ``count[b]`` of them to request b, from its
    position ``start[b]`` on, packed request by request.

    block_table: [B, max_pages] int32; start, count: [B] int32; rows: the rows of
    the step, which may be more than its tokens.  Returns :class:`Slots`: slots
    [rows] int64 (page * page_size + position % page_size, for :func:`kv_write`),
    request and position [rows] int32, all -1 behind the last token, and offsets
    [B + 1] int32, for :func:`prompt_attention`."""
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda:
        raise TypeError("block_table must be a CUDA tensor")
    dev, i32 = block_table.device, torch.int32
    B = start.shape[0]
    if not 0 <= rows < _INT_MAX:
        raise ValueError("rows must not be negative and be below 2^31 - 1")
    if not 1 <= page_size <= _INT_MAX:
        raise ValueError("page_size must be positive and below 2^31")
    t_ptr, cols = _table(block_table, "block_table", B, dev)
    s_ptr = _vector(start, "start", i32, B, dev)
    c_ptr = _vector(count, "count", i32, B, dev)
    got = Slots(_empty((rows,), torch.int64, dev, stream), _empty((rows,), i32, dev, stream),
                _empty((rows,), i32, dev, stream), _empty((B + 1,), i32, dev, stream))
    # one size of workspace for many numbers of rows
    _launch("kv_slots", dev, stream, (B, min(-(-rows // 65536) * 65536, _INT_MAX - 1)),
            (t_ptr, cols, s_ptr, c_ptr, rows, page_size, *[x.data_ptr() for x in got]), (B,))
    return got


def kv_write(cache, layer, k, v, slots, *, stream=None):
    """Write rows of keys and values to their slots in one layer of the paged cache.

    cache: [num_pages, n_layers, 2, page_size, kv_heads * D]; k, v: [rows, kv_heads,
    D] of its dtype, row and head strides free; slots: [rows] int64
    (:func:`kv_slots`), -1 for rows that are not written.  No other slot may come
    twice: of two such rows either may stay, in pieces.  Returns ``cache``."""
    desc, shape = _cache_desc(cache)
    dev = cache.device
    k_args = _heads(k, "k", cache.dtype, dev)
    rows, Hk, D = k.shape
    v_args = _heads(v, "v", cache.dtype, dev, rows)
    if k.shape != v.shape or Hk < 1 or Hk * D != shape[4]:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} do not fit a cache entry of "
                         f"{shape[4]} elements")
    if not 0 <= layer < shape[1]:
        raise ValueError(f"layer {layer} of {shape[1]}")
    s_ptr = _vector(slots, "slots", torch.int64, rows, dev)
    # (the workspace does not depend on the rows)
    _launch("kv_write", dev, stream, (1 if rows else 0,),
            (ctypes.byref(desc), layer, Hk, *k_args, *v_args, s_ptr, rows))
    return cache


# --------------------------------------------------------------------- errors
def prompt_attention_error(stream=None, device=None):
    """``(code, request, row)`` of the first failed request of the last
    prompt_attention on this device (code 0: none).  Synchronises."""
    return _error("prompt_attention", stream, device)


def tree_attention_error(stream=None, device=None):
    """The same of the last tree_attention."""
    return _error("tree_attention", stream, device)


def verify_tree_greedy_error(stream=None, device=None):
    """The same of the last verify_tree_greedy."""
    return _error("verify_tree_greedy", stream, device)


def kv_reserve_error(stream=None, device=None):
    """The same of the last kv_reserve."""
    return _error("kv_reserve", stream, device)


def kv_slots_error(stream=None, device=None):
    """The same of the last kv_slots."""
    return _error("kv_slots", stream, device)


def kv_write_error(stream=None, device=None):
    """The same of the last kv_write; ``row`` is the first failed row."""
    return _error("kv_write", stream, device)

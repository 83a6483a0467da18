"""Operators of the serving and drafter-training step around verification:
attention over the paged KV cache that :func:`kv_commit` fills, the accumulated
attention weights, eviction from the cache by them, and log probabilities of
given tokens with their gradient.

Like the rest of the binding this only marshals arguments.  Calls are
asynchronous on ``stream`` (default: the current stream) and allocate only
their outputs and, once per stream, a workspace.  Data errors are found by the
kernels and read back with the ``*_error`` functions.  Calls may come from any
thread.  Nothing here is recorded by autograd, also where an input requires a
gradient: the gradient of :func:`logprobs` is :func:`logprobs_grad`.
"""

from __future__ import annotations

import collections
import ctypes
import math
import threading

import torch

from . import SV_BF16, SV_F32, SV_OK, SpecVerifyError, _KvCache, _Logits, _check, load_library

SV_F16 = 2
SV_LOGPROBS_TOP_MAX = 32
SV_HEAD_DIM_MAX = 256
_INT_MAX = 2 ** 31 - 1

_DTYPES = {torch.float32: SV_F32, torch.bfloat16: SV_BF16, torch.float16: SV_F16}

LogProbs = collections.namedtuple(
    "LogProbs", ["logprob", "entropy", "max", "logsum", "top_tokens", "top_logprobs"])

_P, _i32, _i64, _sz, _f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                             ctypes.c_float)
_KV = ctypes.POINTER(_KvCache)
_SIGNATURES = {
    "spec_attention_workspace_size": (_sz, [_i32, _i32]),
    "spec_attention": (ctypes.c_int, [_KV, _i32, _i32, _i32, _P, _i64, _i64, _i32, _i64, _P, _i32,
                                      _P, _P, _P, _i32, _f32, _i32, _P, _P, _P, _i32, _P, _sz]),
    "spec_attention_weights_workspace_size": (_sz, [_i32]),
    "spec_attention_weights": (ctypes.c_int, [_KV, _i32, _i32, _i32, _P, _i64, _i64, _i32, _i64,
                                              _P, _i32, _P, _P, _P, _i32, _f32, _i32, _P, _P, _P,
                                              _i64, _P, _i64, _i32, _P, _i32, _P, _sz]),
    "spec_kv_evict_workspace_size": (_sz, [_i32, _i32]),
    "spec_kv_evict": (ctypes.c_int, [_KV, _P, _i32, _KV, _P, _i32, _P, _i64, _i32, _P, _i64, _i32,
                                     _P, _P, _i32, _i32, _i32, _P, _P, _i32, _P, _sz]),
    "spec_logprobs_workspace_size": (_sz, [_i64]),
    "spec_logprobs": (ctypes.c_int, [ctypes.POINTER(_Logits), _P, _P, _i32, _P, _P, _P, _P, _P, _P,
                                     _P, _P, _sz]),
    "spec_logprobs_grad": (ctypes.c_int, [ctypes.POINTER(_Logits), _P, _P, _P, _P, _P, _P, _P, _P,
                                          _i64, _P]),
}
_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


# ----------------------------------------------------------- streams, workspaces
# A call's kernels talk through its workspace, which is its stream's: from the
# choice of the workspace to the last launch there is one call at a time, whatever
# thread it comes from (the interpreter's own lock is given away in the C call).
_lock = threading.Lock()
_workspaces = {}   # (kind, device, stream) -> workspace: calls of one stream are in order
_last = {}         # (kind, device) -> (workspace, stream handle) of the last call; the
                   # workspace is None for a call with nothing to do, which wrote none
_sizes = {}        # workspace sizes already asked for


def _stream_of(stream, dev):
    """The handle of ``stream``, or of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _workspace_size(kind, dev, size):
    key = (kind, dev.index, size)
    need = _sizes.get(key)
    if need is None:
        with torch.cuda.device(dev):
            need = int(getattr(_library(), f"spec_{kind}_workspace_size")(*size))
        if need == 0:
            raise SpecVerifyError(1, f"spec_{kind}_workspace_size")
        if len(_sizes) > 4096:
            _sizes.clear()
        _sizes[key] = need
    return need


def _empty(shape, dtype, dev, stream):
    """An output of a call on ``stream``, of that stream's memory."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _scratch(kind, dev, stream, handle, size):
    """A workspace for a call on the stream: one per stream, or one of its own
    while a graph is being captured (the graph may be replayed next to the
    stream's other calls)."""
    need = _workspace_size(kind, dev, size)
    key = (kind, dev.index, handle)
    capturing = torch.cuda.is_current_stream_capturing()
    ws = None if capturing else _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = _empty(max(need, 256), torch.uint8, dev, stream)
        if not capturing:
            _workspaces[key] = ws
    return ws


def _error(kind, stream, device):
    d = torch.device(device or "cuda")
    index = d.index if d.index is not None else torch.cuda.current_device()
    code, req, row = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    with _lock:
        ws, handle = _last[kind, index]
        if ws is None:
            return 0, -1, -1
        rc = _library().spec_verify_get_error(ws.data_ptr(), handle if stream is None else
                                              stream.cuda_stream, ctypes.byref(code),
                                              ctypes.byref(req), ctypes.byref(row))
    if rc != SV_OK:
        raise SpecVerifyError(rc, "spec_verify_get_error")
    return code.value, req.value, row.value


def _call(name, dev, *args):
    f = getattr(_lib or _library(), name)
    if torch.cuda.current_device() == dev.index:
        rc = f(*args)
    else:
        with torch.cuda.device(dev):
            rc = f(*args)
    if rc != SV_OK:
        raise SpecVerifyError(rc, name)


def _launch(kind, dev, stream, size, args, batch=()):
    """spec_<kind> on the stream, with its workspace."""
    handle = _stream_of(stream, dev)
    with _lock:
        ws = _scratch(kind, dev, stream, handle, size)
        _call("spec_" + kind, dev, *args, handle, *batch, ws.data_ptr(), ws.numel())
        # size[0] counts the requests or rows
        _last[kind, dev.index] = ws if size[0] else None, handle


# --------------------------------------------------------------------- checks
def _vector(t, name, dtype, n, dev, optional=False):
    """A contiguous vector of n elements or more; returns its address."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or \
            t.dim() != 1 or not t.is_contiguous():
        _check(t, name, dtype)
        raise ValueError(f"{name} is on {t.device}, not on {dev}")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, {n} are needed")
    return t.data_ptr()


def _matrix(t, name, dtype, shape, dev):
    """A contiguous tensor of this shape; returns its address."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on {dev}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape {tuple(shape)}")
    return t.data_ptr()


def _rows2d(t, name, dtype, rows, dev):
    """A float matrix with contiguous rows; returns its address, row stride and columns."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != dev or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D {dtype} tensor on {dev}")
    n, cols = t.shape
    stride, one = t.stride()
    if n < rows or (cols > 1 and one != 1):
        raise ValueError(f"{name} must have {rows} contiguous rows")
    return t.data_ptr(), stride if n > 1 else cols, cols


def _cache_desc(cache, name="cache"):
    """The cache's descriptor and shape."""
    if not isinstance(cache, torch.Tensor) or not cache.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if cache.dim() != 5 or not cache.is_contiguous():
        raise ValueError(f"{name} must be contiguous [num_pages, n_layers, 2, page_size, E]")
    shape = cache.shape
    pages, layers, two, S, E = shape
    if two != 2:
        raise ValueError(f"{name} must be contiguous [num_pages, n_layers, 2, page_size, E]")
    es = cache.element_size()
    if es not in (2, 4):
        raise TypeError(f"{name} must have a 2- or 4-byte dtype")
    return _KvCache(cache.data_ptr() or None, pages, layers, S, E, es), shape


def _table(t, name, B, dev):
    """A block table; returns its address and columns."""
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 2 or \
            t.device != dev or not t.is_contiguous():
        _check(t, name, torch.int32, ndim=2)
        raise ValueError(f"{name} must be contiguous with {B} rows on {dev}")
    rows, cols = t.shape
    if rows != B:
        raise ValueError(f"{name} must be contiguous with {B} rows on {dev}")
    return t.data_ptr(), cols


def _attention_args(q, cache, layer, kv_len, block_table, k_per_req, spec, scale, window):
    """The checks that both attention calls share; returns their leading arguments."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise TypeError("q must be a 3-D CUDA tensor")
    dtype, dev = q.dtype, q.device
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {dtype}")
    desc, shape = _cache_desc(cache)
    if cache.dtype is not dtype or cache.device != dev:
        raise TypeError("q and cache must share dtype and device")
    rows, Hq, D = q.shape
    _, layers, _, _, E = shape
    if D < 1 or E % D or Hq < 1 or Hq % (E // D):
        raise ValueError(f"{Hq} heads of {D} do not fit a cache entry of {E} elements")
    ts, hs, one = q.stride()
    if D > 1 and one != 1:
        raise ValueError("the heads of q must be contiguous")
    if not 0 <= layer < layers:
        raise ValueError(f"layer {layer} of {layers}")
    if window < 0:
        raise ValueError("window must be 0 (off) or positive")
    B = k_per_req.shape[0]
    k_ptr = _vector(k_per_req, "k_per_req", torch.int32, B, dev)
    n_ptr = _vector(kv_len, "kv_len", torch.int32, B, dev)
    t_ptr, cols = _table(block_table, "block_table", B, dev)
    slots, s_ptr = 0, None
    if spec is not None:
        if not isinstance(spec, torch.Tensor) or spec.dim() != 5 or spec.shape[1] < 1:
            raise ValueError("spec must be [B, slots, n_layers, 2, E]")
        if spec.dtype is not dtype or spec.device != dev:
            raise TypeError("spec must share q's dtype and device")
        slots = spec.shape[1]
        if spec.shape != (B, slots, layers, 2, E) or not spec.is_contiguous():
            raise ValueError("spec must be contiguous [B, slots, n_layers, 2, E] matching the cache")
        s_ptr = spec.data_ptr()
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    return dev, dtype, B, rows, Hq, D, (
        ctypes.byref(desc), code, layer, E // D, q.data_ptr(), ts, hs, Hq, rows, s_ptr, slots,
        k_ptr, n_ptr, t_ptr, cols, scale, min(window, _INT_MAX))   # a wider one hides nothing


# ------------------------------------------------------------------ operators
def attention(q, cache, layer, kv_len, block_table, k_per_req, spec=None, *, scale=None, window=0,
              out=None, out_lse=None, stream=None):
    """Attention of every request's query tokens over its paged cache.

    q: [rows, q_heads, D] (bf16, fp16 or fp32; token and head strides are free),
    request b owning the k_b + 1 rows that it owns among the verifier's target
    rows; cache: [num_pages, n_layers, 2, page_size, kv_heads * D] as in
    :func:`kv_commit`, of which ``layer`` is read; kv_len, k_per_req: [B] int32;
    block_table: [B, max_pages] int32; spec: [B, slots, n_layers, 2, E], the
    entries of the query tokens that :func:`kv_commit` will append (token j then
    sits at position kv_len + j), or None when the cache holds them already
    (token j sits at kv_len - 1 - k + j).  A token sees the positions up to its
    own, with ``window`` > 0 only the last ``window`` of them.

    Returns ``(out [rows, q_heads, D], lse [rows, q_heads] float32)``; a token
    that sees nothing has out 0 and lse -inf.  They carry no autograd history."""
    dev, dtype, B, rows, Hq, D, args = _attention_args(q, cache, layer, kv_len, block_table,
                                                       k_per_req, spec, scale, window)
    if out is None:
        out = _empty((rows, Hq, D), dtype, dev, stream)
    else:
        _matrix(out, "out", dtype, (rows, Hq, D), dev)
    if out_lse is None:
        out_lse = _empty((rows, Hq), torch.float32, dev, stream)
    else:
        _matrix(out_lse, "out_lse", torch.float32, (rows, Hq), dev)
    _launch("attention", dev, stream, (B, D), (*args, out.data_ptr(), out_lse.data_ptr()), (B,))
    return out, out_lse


def attention_weights(q, cache, layer, kv_len, block_table, k_per_req, lse, score, spec=None,
                      accept_len=None, *, scale=None, window=0, out_score=None, stream=None):
    """Add the attention weights of one layer to the positions' running scores.

    The arguments of :func:`attention` and its ``lse``, before :func:`kv_commit`
    moves kv_len; score: [B, cols] float32.  Only the query tokens 0 ..
    accept_len[b] count (all without it; a request with -1 is left alone), so
    rejected drafts leave no trace.  Positions 0 .. kv_len - 1 and, with
    ``spec``, those that the commit will append are written to ``out_score``
    (default: ``score`` itself).  Returns ``out_score``."""
    dev, _, B, rows, Hq, _, args = _attention_args(q, cache, layer, kv_len, block_table,
                                                   k_per_req, spec, scale, window)
    l_ptr = _matrix(lse, "lse", torch.float32, (rows, Hq), dev)
    a_ptr = _vector(accept_len, "accept_len", torch.int32, B, dev, optional=True)
    s_ptr, stride, cols = _rows2d(score, "score", torch.float32, B, dev)
    if out_score is None:
        out_score = score
    o_ptr, out_stride, out_cols = _rows2d(out_score, "out_score", torch.float32, B, dev)
    if out_cols != cols:
        raise ValueError("score and out_score must have the same columns")
    _launch("attention_weights", dev, stream, (B,),
            (*args, l_ptr, a_ptr, s_ptr, stride, o_ptr, out_stride, cols), (B,))
    return out_score


def kv_evict(cache, score, kv_len, block_table, budget, sinks=0, recent=0, *, out_cache=None,
             out_table=None, out_score=None, out_len=None, out_kept=None, with_kept=False,
             stream=None):
    """Keep at most ``budget`` positions of every request, by attention weight.

    A request with more keeps its first ``sinks``, its last ``recent`` and, of
    the others, those of the largest score (lowest position on ties), in their
    order: every layer's K and V move to positions 0 .. budget - 1, scores
    (:func:`attention_weights`) with them, and the length becomes the number
    kept.  Without ``out_table`` the entries move inside the request's own
    pages, which no other request may share; with it they are written to those
    pages of ``out_cache`` (default: the same cache, where they have to be other
    pages, or ``block_table`` itself for in place) and the source stays.
    ``out_score`` and ``out_len`` default to score and kv_len, in place.

    Returns ``(out_len [B] int32, kept [B, budget] int32 or None)``."""
    desc, shape = _cache_desc(cache)
    dev = cache.device
    B = kv_len.shape[0]
    n_ptr = _vector(kv_len, "kv_len", torch.int32, B, dev)
    t_ptr, cols = _table(block_table, "block_table", B, dev)
    if not 1 <= budget <= _INT_MAX or sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("budget must be positive, below 2^31 and hold sinks and recent")
    s_ptr, stride, score_cols = _rows2d(score, "score", torch.float32, B, dev)
    if out_score is None:
        out_score = score
    os_ptr, out_stride, out_cols = _rows2d(out_score, "out_score", torch.float32, B, dev)
    if out_len is None:
        out_len = kv_len
    m_ptr = _vector(out_len, "out_len", torch.int32, B, dev)
    out_desc, ot_ptr, ot_cols = None, None, 0
    if out_table is not None:
        ot_ptr, ot_cols = _table(out_table, "out_table", B, dev)
        dst = cache if out_cache is None else out_cache
        out_desc, out_shape = _cache_desc(dst, "out_cache")
        if dst.dtype is not cache.dtype or dst.device != dev or out_shape[1:] != shape[1:]:
            raise ValueError("out_cache must match the cache in all but its pages")
        out_desc = ctypes.byref(out_desc)
    elif out_cache is not None:
        raise ValueError("out_cache needs out_table")
    if out_kept is None and with_kept:
        out_kept = _empty((B, budget), torch.int32, dev, stream)
    k_ptr = None if out_kept is None else _matrix(out_kept, "out_kept", torch.int32, (B, budget),
                                                  dev)
    _launch("kv_evict", dev, stream, (B, budget),
            (ctypes.byref(desc), t_ptr, cols, out_desc, ot_ptr, ot_cols, s_ptr, stride, score_cols,
             os_ptr, out_stride, out_cols, n_ptr, m_ptr, budget, sinks, recent, k_ptr), (B,))
    return out_len, out_kept


def _rows_desc(x):
    """The descriptor, device, rows and columns of a logit matrix."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dim() != 2:
        raise TypeError("logits must be a 2-D CUDA tensor")
    dtype = x.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError(f"logits must be float32 or bfloat16, got {dtype}")
    R, V = x.shape
    stride, one = x.stride()
    if V > 1 and one != 1:
        raise ValueError("logit rows must be contiguous")
    return _Logits(x.data_ptr() or None, _DTYPES[dtype], V, R, stride if R > 1 else V), x.device, \
        R, V


def logprobs(logits, tokens, temperature=None, n_top=0, *, stream=None):
    """Log probability of each row's token, entropy and the ``n_top`` (at most
    32) most likely tokens, in one pass over the logits.

    logits: [rows, V] float32 or bfloat16, any row stride; tokens: [rows] int32
    (-1: skip the row; None: no log probabilities); temperature: [rows] float32
    or None, 0 standing for 1.  Returns a :class:`LogProbs`: logprob, entropy,
    max, logsum [rows] float32 and top_tokens, top_logprobs [rows, n_top] (None
    without n_top; ties go to the lowest index; -1 and -inf where a row has
    fewer tokens of nonzero probability).

    The results carry no autograd history, also where the logits require a
    gradient: a loss made of them is constant to autograd.  Its gradient is
    :func:`logprobs_grad`, to be handed to ``logits.backward`` (or
    ``torch.autograd.backward`` next to a loss's other terms)."""
    x, dev, R, _ = _rows_desc(logits)
    t_ptr = _vector(tokens, "tokens", torch.int32, R, dev, optional=True)
    T_ptr = _vector(temperature, "temperature", torch.float32, R, dev, optional=True)
    if not 0 <= n_top <= SV_LOGPROBS_TOP_MAX:
        raise ValueError(f"n_top must be in [0, {SV_LOGPROBS_TOP_MAX}]")
    lp, ent, mx, ls = [_empty((R,), torch.float32, dev, stream) for _ in range(4)]
    tok = top = tok_ptr = top_ptr = None
    if n_top:
        tok = _empty((R, n_top), torch.int32, dev, stream)
        top = _empty((R, n_top), torch.float32, dev, stream)
        tok_ptr, top_ptr = tok.data_ptr(), top.data_ptr()
    _launch("logprobs", dev, stream, (R,),
            (ctypes.byref(x), t_ptr, T_ptr, n_top, lp.data_ptr(), ent.data_ptr(), mx.data_ptr(),
             ls.data_ptr(), tok_ptr, top_ptr))
    return LogProbs(lp, ent, mx, ls, tok, top)


def logprobs_grad(logits, tokens, max, logsum, entropy, grad_logprob, grad_entropy=None,
                  temperature=None, *, out=None, stream=None):
    """Gradient of a loss with respect to the logits, from its gradients with
    respect to :func:`logprobs`' logprob and entropy ([rows] float32, either may
    be None) and that call's max, logsum and entropy (needed with grad_entropy).

    Returns ``out`` [rows, V] of the logits' dtype; it may be the logits
    themselves.  Rows with token -1 get 0."""
    x, dev, R, V = _rows_desc(logits)
    t_ptr = _vector(tokens, "tokens", torch.int32, R, dev)
    m_ptr = _vector(max, "max", torch.float32, R, dev)
    l_ptr = _vector(logsum, "logsum", torch.float32, R, dev)
    h_ptr = _vector(entropy, "entropy", torch.float32, R, dev, optional=grad_entropy is None)
    gl_ptr = _vector(grad_logprob, "grad_logprob", torch.float32, R, dev, optional=True)
    gh_ptr = _vector(grad_entropy, "grad_entropy", torch.float32, R, dev, optional=True)
    T_ptr = _vector(temperature, "temperature", torch.float32, R, dev, optional=True)
    if out is None:
        out = _empty((R, V), logits.dtype, dev, stream)
    o_ptr, out_stride, out_cols = _rows2d(out, "out", logits.dtype, R, dev)
    if out_cols != V or out.shape[0] != R:
        raise ValueError(f"out must be {(R, V)}")
    _call("spec_logprobs_grad", dev, ctypes.byref(x), t_ptr, T_ptr, m_ptr, l_ptr, h_ptr, gl_ptr,
          gh_ptr, o_ptr, out_stride, _stream_of(stream, dev))
    return out


# --------------------------------------------------------------------- errors
def attention_error(stream=None, device=None):
    """``(code, request, row)`` of the first failed request of the last
    attention on this device (code 0: none).  Synchronises."""
    return _error("attention", stream, device)


def attention_weights_error(stream=None, device=None):
    """The same of the last attention_weights."""
    return _error("attention_weights", stream, device)


def kv_evict_error(stream=None, device=None):
    """The same of the last kv_evict."""
    return _error("kv_evict", stream, device)


def logprobs_error(stream=None, device=None):
    """The same of the last logprobs; ``row`` is the first failed row."""
    return _error("logprobs", stream, device)

"""Python binding of the language-model operators of libmuon.so (C ABI in
include/muon_lm.h): attention, the norm and rotation of query and key heads,
the embedding, the gated feed-forward block, the norms around a block with its
gate and residual scale, and dropout, each with its gradients.

Argument checks and marshalling only; every step runs in the HIP kernels of
the library.  Calls run on the current stream of the tensors' device and do
not synchronise.  Tensors the library writes are new unless given.  The
workspace comes from torch's allocator for the call unless given (it then is
the caller's to keep apart between streams), so calls can be captured into a
graph.  Same inputs give the same bits every time.

As in ``muon``, nothing here is recorded by autograd: results carry no history,
also where an argument requires a gradient.  ``lm_example`` shows the
``autograd.Function`` around each pair of calls.
"""

import ctypes
import math
import struct

import torch

from . import muon

_lib = muon.lib
_vp, _i64, _sz, _int, _buf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_char_p

for _name, _res, _args in (
        ("muon_attention_workspace_size", _sz, [_buf]),
        ("muon_attention_backward_workspace_size", _sz, [_buf]),
        ("muon_attention", _int, [_buf, _vp, _sz, _vp]),
        ("muon_attention_backward", _int, [_buf, _vp, _sz, _vp]),
        ("muon_qk_norm_rope_backward_workspace_size", _sz, [_buf]),
        ("muon_qk_norm_rope", _int, [_buf, _vp]),
        ("muon_qk_norm_rope_backward", _int, [_buf, _vp, _sz, _vp]),
        ("muon_embedding", _int, [_vp, _int, _vp, _int, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _vp]),
        ("muon_embedding_backward_workspace_size", _sz, [_i64, _i64, _i64]),
        ("muon_embedding_backward", _int, [_vp, _int, _vp, _int, _vp, _int, _i64, _i64, _i64, ctypes.c_float, _vp, _sz,
                                           _vp]),
        ("muon_dropout", _int, [_vp, _vp, _i64, _int, ctypes.c_double, ctypes.c_uint64, ctypes.c_uint64, _vp, _vp]),
        ("muon_residual_norm_backward_workspace_size", _sz, [_buf]),
        ("muon_residual_norm", _int, [_buf, _vp]),
        ("muon_residual_norm_backward", _int, [_buf, _vp, _sz, _vp]),
        ("muon_feed_forward_workspace_size", _sz, [_buf]),
        ("muon_feed_forward_backward_workspace_size", _sz, [_buf]),
        ("muon_feed_forward", _int, [_buf, _vp, _sz, _vp]),
        ("muon_feed_forward_backward", _int, [_buf, _vp, _sz, _vp])):
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args

#: Every symbol include/muon_lm.h declares.
EXPORTS = ("muon_attention_workspace_size", "muon_attention_backward_workspace_size", "muon_attention",
           "muon_attention_backward", "muon_qk_norm_rope_backward_workspace_size", "muon_qk_norm_rope",
           "muon_qk_norm_rope_backward", "muon_embedding", "muon_embedding_backward_workspace_size",
           "muon_embedding_backward", "muon_dropout", "muon_residual_norm_backward_workspace_size",
           "muon_residual_norm", "muon_residual_norm_backward", "muon_feed_forward_workspace_size",
           "muon_feed_forward_backward_workspace_size", "muon_feed_forward", "muon_feed_forward_backward")
#: Largest head sizes (MUON_ATTENTION_MAX_D, MUON_QK_NORM_MAX_D).
ATTENTION_MAX_D = 128
QK_NORM_MAX_D = 512
#: Largest width of residual_norm (MUON_RESIDUAL_NORM_MAX_WIDTH).
RESIDUAL_NORM_MAX_WIDTH = 8192
#: Activations of feed_forward (muon_activation).
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}

_F32, _BF16 = torch.float32, torch.bfloat16
_DTYPE = {_F32: muon.MUON_F32, _BF16: muon.MUON_BF16}
# the argument structures of muon_lm.h: 8-byte fields throughout
_ATTN = struct.Struct("9Q15q2Qq3Q8q2d")
_QK = struct.Struct("10Q12q2qQqQ3qqd")
_RESID = struct.Struct("16Q6q3q2q3q2d3Q")
_FFN = struct.Struct("11Q4q3q2q")


# the current stream of a device as a number (0.1 us; a Stream object for it costs 2)
_raw_stream = torch._C._cuda_getCurrentRawStream


def _tensor(t, name, dtype, dev, dims=None):
    """Checks one tensor; `dtype` is a type or a tuple of types."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.device == dev and (dims is None or t.dim() == dims):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev or dev.type != "cuda":
        raise ValueError(f"{name} must be on {dev if dev.type == 'cuda' else 'a GPU'} (got {t.device})")
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions (got {tuple(t.shape)})")


def _last(t, name):
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _heads(t, name, dev):
    """bfloat16 of 4 dimensions on `dev`, the last one contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.is_cuda and t.device == dev and t.dim() == 4
            and t.stride(3) == 1):
        _tensor(t, name, _BF16, dev, 4)
        _last(t, name)


def _exactly(t, name, dtype, dev, shape):
    """A contiguous tensor of one shape."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.device == dev and t.shape == shape
            and t.is_contiguous()):
        return
    _tensor(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _layout(t):
    """(first byte, past the last one, bytes of a contiguous piece, steps
    between pieces) of a tensor that has elements."""
    size = t.element_size()
    end = piece = size
    steps = []
    for step, n in sorted(zip(t.stride(), t.shape)):
        if n > 1:
            end += (n - 1) * step * size
            if step * size == piece and not steps:
                piece *= n
            elif step:
                steps.append(step * size)
    at = t.data_ptr()
    return at, at + end, piece, steps


def _end(t):
    """Past a tensor's last byte."""
    if t.is_contiguous():
        return t.data_ptr() + t.nbytes
    return _layout(t)[1]


def _overlap(a, b):
    """Whether two tensors may share memory: never False where they do."""
    if a.numel() == 0 or b.numel() == 0:
        return False
    a0, a1, piece, steps = _layout(a)
    if b.data_ptr() >= a1:
        return False
    b0, b1, other, more = _layout(b)
    if b1 <= a0:
        return False
    # interleaved (heads of one projection): pieces begin at multiples of the
    # steps' divisor, those of b `off` past those of a
    step = math.gcd(*steps, *more)
    if step == 0:
        return True
    off = (b0 - a0) % step
    return off < piece or off + other > step


def _repeats(t):
    """Whether elements of a tensor may share memory."""
    end = 1
    for step, n in sorted(zip(t.stride(), t.shape)):
        if n > 1:
            if step < end:
                return True
            end += (n - 1) * step
    return False


def _apart(t, name, *others):
    """Refuses a given output that shares memory with a tensor the kernels read
    beside it; others: (tensor or None, name), and True for one that may be
    the output itself, element for element."""
    first = t.data_ptr()
    end = _end(t)
    for o, other, *itself in others:
        if o is None or o.data_ptr() >= end or _end(o) <= first or not _overlap(t, o):
            continue
        if itself and t.data_ptr() == o.data_ptr() and t.shape == o.shape and all(
                x == y or n == 1 for x, y, n in zip(t.stride(), o.stride(), t.shape)):
            continue
        raise ValueError(f"{name} must not share memory with {other}")


def _ws(workspace, need, dev):
    """(address, bytes) of the caller's workspace or of a new one, and what holds it."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        return workspace.data_ptr(), need, workspace
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _call(dev, fn, *args):
    """Calls fn(*args, stream) with `dev` as the current device."""
    index = dev.index
    if index is not None and index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    else:
        status = fn(*args, _raw_stream(torch.cuda.current_device() if index is None else index))
    if status:
        muon._check(status)


def _attention_args(q, k, v, out, lse, dout, grads, scale, causal, window, softcap, slopes, documents, prefix, lengths,
                    starts):
    """The checked arguments as muon_attention_args, and the tensors it points to."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev = q.device
    _heads(q, "q", dev)
    _heads(k, "k", dev)
    _heads(v, "v", dev)
    b, sq, hq, d = q.shape
    kb, sk, hkv, kd = k.shape
    if kb != b or kd != d or v.shape != k.shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit: (batch, positions, "
                         "heads, head size), k and v alike")
    if hkv == 0 or hq % hkv:
        raise ValueError(f"{hq} query heads over {hkv} key heads")
    if d % 8 or not 0 < d <= ATTENTION_MAX_D:
        raise ValueError(f"the head size must be a multiple of 8 up to {ATTENTION_MAX_D} (got {d})")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    window = 0 if window is None else int(window)
    softcap = 0.0 if softcap is None else float(softcap)
    p_slopes = p_docs = doc_stride = p_prefix = p_lengths = p_starts = 0
    if slopes is not None:
        _exactly(slopes, "slopes", _F32, dev, (hq,))
        p_slopes = slopes.data_ptr()
    if documents is not None:
        _tensor(documents, "documents", torch.int32, dev, 2)
        _last(documents, "documents")
        if documents.shape != (b, sk):
            raise ValueError(f"documents must have shape {(b, sk)} (got {tuple(documents.shape)})")
        p_docs, doc_stride = documents.data_ptr(), documents.stride(0)
    if prefix is not None:
        _exactly(prefix, "prefix", torch.int32, dev, (b,))
        p_prefix = prefix.data_ptr()
    if lengths is not None:
        _exactly(lengths, "lengths", torch.int32, dev, (b,))
        p_lengths = lengths.data_ptr()
    if starts is not None:
        _exactly(starts, "starts", torch.int32, dev, (b,))
        p_starts = starts.data_ptr()
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _heads(out, "out", dev)
        if out.shape != q.shape:
            raise ValueError(f"out must have q's shape {tuple(q.shape)} (got {tuple(out.shape)})")
    if lse is None:
        lse = torch.empty((b, hq, sq), dtype=_F32, device=dev)
    else:
        _exactly(lse, "lse", _F32, dev, (b, hq, sq))
    do_ptr, do_strides = 0, (0, 0, 0)
    if dout is not None:
        do_ptr, do_strides = dout.data_ptr(), dout.stride()[:3]
    args = _ATTN.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), do_ptr, *grads,
                      *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *out.stride()[:3], *do_strides, p_slopes,
                      p_docs, doc_stride, p_prefix, p_lengths, p_starts, b, sq, sk, hq, hkv, d, bool(causal), window,
                      float(scale), softcap)
    return args, out, lse, dev


def attention(q, k, v, scale=None, causal=True, window=0, softcap=0.0, slopes=None, documents=None, prefix=None,
              lengths=None, starts=None, out=None, lse=None, workspace=None):
    """Attention of bfloat16 ``q`` (batch, sq, heads, d) over ``k`` and ``v``
    (batch, sk, kv_heads, d); returns ``(out, lse)``: bfloat16 shaped as q and
    float32 (batch, heads, sq).  d is a multiple of 8 up to 128, heads a
    multiple of kv_heads; strides are free (multiples of 8, the last dimension
    contiguous, 16-byte aligned), so views of one projection's output serve.

    * ``scale``: of the scores (default 1 / sqrt(d)); ``softcap`` c > 0: scores
      become c tanh(score / c); ``slopes`` (heads,) float32: score -= slope
      |position - key|.
    * ``starts`` (batch,) int32: position of the first query (default sk - sq:
      the queries are the last positions).
    * ``causal``: keys up to the query's position; ``window`` w > 0: keys less
      than w away; ``prefix`` (batch,) int32: keys below it are seen by all
      queries nevertheless.
    * ``documents`` (batch, sk) int32: only keys of the query's document, prefix
      or not; ``lengths`` (batch,) int32: positions from there on are padding,
      as keys and as queries, and may hold anything.

    ``out`` may be q itself; else given outputs must not share memory with
    anything (nor may elements of ``out`` among themselves).

    A query that sees no key gets out = 0 and lse = -inf.  Keys and values past
    the last one that any query of the batch sees may hold anything, as the
    rest of a cache does.  A step of generation
    (up to 32 query rows per key head) reads each cached key and value once."""
    given = out, lse
    args, out, lse, dev = _attention_args(q, k, v, out, lse, None, (0, 0, 0), scale, causal, window, softcap, slopes,
                                          documents, prefix, lengths, starts)
    if given[0] is not None or given[1] is not None:
        reads = ((k, "k"), (v, "v"), (slopes, "slopes"), (documents, "documents"), (prefix, "prefix"),
                 (lengths, "lengths"), (starts, "starts"))
        if given[0] is not None:
            if not out.is_contiguous() and _repeats(out):
                raise ValueError("elements of out share memory")
            _apart(out, "out", (q, "q", True), *reads, (given[1], "lse"))
        if given[1] is not None:
            _apart(lse, "lse", (q, "q"), *reads)
    ptr, size, ws = _ws(workspace, _lib.muon_attention_workspace_size(args) or 256, dev)
    _call(dev, _lib.muon_attention, args, ptr, size)
    return out, lse


def attention_backward(dout, q, k, v, out, lse, scale=None, causal=True, window=0, softcap=0.0, slopes=None,
                       documents=None, prefix=None, lengths=None, starts=None, dq=None, dk=None, dv=None,
                       workspace=None):
    """Gradients ``(dq, dk, dv)`` (bfloat16, contiguous) from ``dout``, the
    gradient of ``out``, and the arguments and results of ``attention``.  The
    gradients of a shared key head sum over its query heads.  A given dq may be
    ``out`` itself, dk and dv may be k and v; else given gradients must not
    share memory with q, k, v, dout, the masks or each other, and dq not with
    out or lse either."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    dev = q.device
    _heads(dout, "dout", dev)
    if out is None or lse is None:
        raise TypeError("out and lse of the forward pass are needed")
    if dout.shape != q.shape:
        raise ValueError(f"dout must have q's shape {tuple(q.shape)} (got {tuple(dout.shape)})")
    grads, given = [], (dq, dk, dv)
    for t, like, name in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        if t is None:
            t = torch.empty_like(like, memory_format=torch.contiguous_format)
        else:
            _exactly(t, name, _BF16, dev, like.shape)
        grads.append(t)
    args, out, lse, dev = _attention_args(q, k, v, out, lse, dout, [t.data_ptr() for t in grads], scale, causal,
                                          window, softcap, slopes, documents, prefix, lengths, starts)
    if any(t is not None for t in given):
        # dq is written before q and dout are read for dk and dv, and while k and v are read for it
        dq, dk, dv = given
        reads = ((q, "q"), (dout, "dout"), (slopes, "slopes"), (documents, "documents"), (prefix, "prefix"),
                 (lengths, "lengths"), (starts, "starts"))
        if dq is not None:
            _apart(dq, "dq", *reads, (k, "k"), (v, "v"), (out, "out", True), (lse, "lse"), (dk, "dk"), (dv, "dv"))
        for t, name in ((dk, "dk"), (dv, "dv")):
            if t is not None:
                _apart(t, name, *reads, (k, "k", True), (v, "v", True))
        if dk is not None:
            _apart(dk, "dk", (dv, "dv"))
    ptr, size, ws = _ws(workspace, _lib.muon_attention_backward_workspace_size(args) or 256, dev)
    _call(dev, _lib.muon_attention_backward, args, ptr, size)
    return tuple(grads)


def _qk_args(q, k, table, positions, q_weight, k_weight, eps, outs, dz, dws):
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dev, dtype = q.device, q.dtype
    if dtype not in _DTYPE:
        raise TypeError(f"q must be float32 or bfloat16 (got {dtype})")
    for t, name in ((q, "q"), (k, "k")):
        _tensor(t, name, dtype, dev, 4)
        _last(t, name)
    b, s, hq, d = q.shape
    hkv = k.shape[2]
    if k.shape[0] != b or k.shape[1] != s or k.shape[3] != d:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} differ in more than their heads")
    if d % 2 or not 0 < d <= QK_NORM_MAX_D:
        raise ValueError(f"the head size must be even and up to {QK_NORM_MAX_D} (got {d})")
    _tensor(table, "table", _F32, dev, 3)
    if table.shape[1] != d // 2 or table.shape[2] != 2 or not table.is_contiguous():
        raise ValueError(f"table must be contiguous, (positions, {d // 2}, 2) (got {tuple(table.shape)})")
    ptrs = []
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _exactly(t, name, _F32, dev, (d,))
        ptrs.append(0 if t is None else t.data_ptr())
    p_pos = 0
    if positions is not None:
        _exactly(positions, "positions", torch.int32, dev, (b, s))
        p_pos = positions.data_ptr()
    results = []
    for t, like, name in ((outs[0], q, outs[2] + "q"), (outs[1], k, outs[2] + "k")):
        if t is None:
            t = torch.empty_like(like, memory_format=torch.contiguous_format)
        else:
            _exactly(t, name, dtype, dev, like.shape)
        results.append(t)
    z_ptr, z_str = (0, 0), (0,) * 6
    if dz is not None:
        for t, like, name in ((dz[0], q, "dq"), (dz[1], k, "dk")):
            _tensor(t, name, dtype, dev, 4)
            _last(t, name)
            if t.shape != like.shape:
                raise ValueError(f"{name} must have shape {tuple(like.shape)} (got {tuple(t.shape)})")
        z_ptr = (dz[0].data_ptr(), dz[1].data_ptr())
        z_str = dz[0].stride()[:3] + dz[1].stride()[:3]
    dw_ptr = [0 if t is None else t.data_ptr() for t in dws]
    args = _QK.pack(q.data_ptr(), k.data_ptr(), results[0].data_ptr(), results[1].data_ptr(), *z_ptr, *ptrs, *dw_ptr,
                    *q.stride()[:3], *k.stride()[:3], *z_str, hq, hkv, table.data_ptr(), table.shape[0], p_pos, b, s, d,
                    _DTYPE[dtype], float(eps))
    return args, results, dev


def qk_norm_rope(q, k, table, positions=None, q_weight=None, k_weight=None, eps=1e-6, q_out=None, k_out=None):
    """RMS norm of every head of ``q`` (batch, s, heads, d) and ``k`` (batch, s,
    kv_heads, d), float32 or bfloat16, and their rotation by position, in one
    pass; returns the new (or given) contiguous ``(q, k)``.

    ``table`` (limit, d / 2, 2) float32 holds (cos, sin) of each position and
    pair (i, i + d / 2); ``positions`` (batch, s) int32 (default 0 .. s - 1;
    one outside the table gives NaN); ``q_weight`` and ``k_weight`` (d,)
    float32 scale the norms (default ones).  d is even and up to 512; d a
    multiple of 16 (float32: 8) with 16-byte aligned heads runs fastest.
    ``q_out`` may be q itself and ``k_out`` k; else they must not share memory
    with anything."""
    args, results, dev = _qk_args(q, k, table, positions, q_weight, k_weight, eps, (q_out, k_out, "out of "), None,
                                  (None, None))
    if q_out is not None or k_out is not None:
        reads = ((table, "table"), (positions, "positions"), (q_weight, "q_weight"), (k_weight, "k_weight"))
        if q_out is not None:
            _apart(q_out, "q_out", (q, "q", True), (k, "k"), *reads, (k_out, "k_out"))
        if k_out is not None:
            _apart(k_out, "k_out", (q, "q"), (k, "k", True), *reads)
    _call(dev, _lib.muon_qk_norm_rope, args)
    return results[0], results[1]


def qk_norm_rope_backward(dq, dk, q, k, table, positions=None, q_weight=None, k_weight=None, eps=1e-6, workspace=None):
    """Gradients ``(dq, dk, dq_weight, dk_weight)`` of ``qk_norm_rope`` from the
    gradients of its outputs and its arguments; those of the weights are
    float32, and None for a weight that was not given."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dws = [None if w is None else torch.empty(q.shape[-1], dtype=_F32, device=q.device) for w in (q_weight, k_weight)]
    args, results, dev = _qk_args(q, k, table, positions, q_weight, k_weight, eps, (None, None, "gradient of "),
                                  (dq, dk), dws)
    ptr, size, ws = _ws(workspace, _lib.muon_qk_norm_rope_backward_workspace_size(args) or 256, dev)
    _call(dev, _lib.muon_qk_norm_rope_backward, args, ptr, size)
    return results[0], results[1], dws[0], dws[1]


def _tokens(tokens):
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a torch.Tensor")
    _tensor(tokens, "tokens", (torch.int64, torch.int32), tokens.device)
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens.device, 8 if tokens.dtype is torch.int64 else 4


def _float_type(dtype, name):
    if dtype not in _DTYPE:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {dtype})")


def embedding(tokens, table, scale=1.0, dtype=None, out=None):
    """Rows ``scale * table[tokens]`` of a float32 or bfloat16 table (vocab,
    width), as a new (or given) tensor of shape tokens.shape + (width,) and of
    ``dtype`` (float32 or bfloat16; default the table's).  Tokens are int64 or
    int32; one outside the table gives a row of NaN."""
    dev, token_bytes = _tokens(tokens)
    _tensor(table, "table", (_F32, _BF16), dev, 2)
    if not table.is_contiguous():
        raise ValueError("table must be contiguous")
    shape = (*tokens.shape, table.shape[1])
    if out is None:
        dtype = table.dtype if dtype is None else dtype
        _float_type(dtype, "dtype")
        out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _float_type(out.dtype, "out")
        if dtype is not None and dtype != out.dtype:
            raise TypeError(f"out is {out.dtype}, not {dtype}")
        _exactly(out, "out", out.dtype, dev, shape)
        _apart(out, "out", (tokens, "tokens"), (table, "table"))
    _call(dev, _lib.muon_embedding, tokens.data_ptr(), token_bytes, table.data_ptr(), _DTYPE[table.dtype],
          out.data_ptr(), _DTYPE[out.dtype], tokens.numel(), table.shape[0], table.shape[1], float(scale))
    return out


def embedding_backward(dout, tokens, vocab, scale=1.0, dtype=None, out=None, workspace=None):
    """Gradient (vocab, width) of ``embedding``'s table from ``dout`` (of
    tokens.shape + (width,), float32 or bfloat16, contiguous): for each row the
    sum of its tokens' gradients times ``scale``, in float32 and in one fixed
    order, rounded once to ``dtype`` (default dout's).  Rows of tokens that do
    not occur are zero."""
    dev, token_bytes = _tokens(tokens)
    _tensor(dout, "dout", (_F32, _BF16), dev)
    if dout.dim() != tokens.dim() + 1 or dout.shape[:-1] != tokens.shape:
        raise ValueError(f"dout {tuple(dout.shape)} does not fit tokens {tuple(tokens.shape)}")
    if not dout.is_contiguous():
        raise ValueError("dout must be contiguous")
    vocab, width, n = int(vocab), dout.shape[-1], tokens.numel()
    if out is None:
        dtype = dout.dtype if dtype is None else dtype
        _float_type(dtype, "dtype")
        if vocab <= 0:
            raise ValueError(f"vocab must be positive (got {vocab})")
        out = torch.empty((vocab, width), dtype=dtype, device=dev)
    else:
        _float_type(out.dtype, "out")
        if dtype is not None and dtype != out.dtype:
            raise TypeError(f"out is {out.dtype}, not {dtype}")
        _exactly(out, "out", out.dtype, dev, (vocab, width))
        _apart(out, "out", (tokens, "tokens"), (dout, "dout"))
    ptr, size, ws = _ws(workspace, _lib.muon_embedding_backward_workspace_size(n, vocab, width) or 256, dev)
    _call(dev, _lib.muon_embedding_backward, tokens.data_ptr(), token_bytes, dout.data_ptr(), _DTYPE[dout.dtype],
          out.data_ptr(), _DTYPE[out.dtype], n, vocab, width, float(scale), ptr, size)
    return out


def _rows(t, name):
    """The stride between the rows of the last dimension (any where there is at most one row)."""
    if t.is_contiguous() and t.dim():
        return t.shape[-1]
    if t.dim() == 0:
        raise ValueError(f"{name} must have a last dimension")
    _last(t, name)
    step = count = None
    for n, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step, count = stride, n
        elif stride == step * count:
            count *= n
        else:
            raise ValueError(f"the rows of {name} must be one stride apart (shape {tuple(t.shape)}, strides {t.stride()})")
    return t.shape[-1] if step is None else step


def _drop_args(p, seed, offset, dev):
    """(p, seed, offset, address of the state) of dropout's generator."""
    p = float(p)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be within 0 .. 1 (got {p})")
    offset = int(offset)
    if isinstance(seed, torch.Tensor):
        _exactly(seed, "seed", torch.int64, dev, (2,))
        return p, 0, offset & 0xFFFFFFFFFFFFFFFF, seed.data_ptr()
    return p, int(seed) & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF, 0


def dropout(x, p, seed, offset=0, out=None):
    """Drops elements of ``x`` (float32 or bfloat16, contiguous) with
    probability t / 65536, t = round(65536 p), and multiplies the others by
    65536 / (65536 - t).  Nothing is stored: element i (in memory order) is
    dropped by 16 bits of Philox4x32-10 of ``seed`` and of block ``offset`` + i
    / 8, so the gradient is ``dropout(dout, p, seed, offset)``, and a call uses
    the ``(x.numel() + 7) // 8`` blocks from offset on.

    ``seed`` is an integer, or an int64 tensor (seed, block) on x's device,
    which the kernel reads: the seed, and what is added to ``offset``.  (A
    captured graph whose tensor the program advances drops other elements at
    every replay.)  ``out`` may be x itself; else it must not share memory with
    x or seed."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    _tensor(x, "x", (_F32, _BF16), dev)
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    p, key, first, state = _drop_args(p, seed, offset, dev)
    if out is None:
        out = torch.empty_like(x)
    else:
        _exactly(out, "out", x.dtype, dev, x.shape)
        _apart(out, "out", (x, "x", True), (seed if state else None, "seed"))
    _call(dev, _lib.muon_dropout, x.data_ptr(), out.data_ptr(), x.numel(), _DTYPE[x.dtype], p, key, first, state)
    return out


def _resid_args(x, y, gate, scale, post_weight, pre_weight, post, eps, p, seed, offset, dtype, forward, grads, dev):
    """The checked arguments as muon_residual_norm_args.  x: the stream (or its
    like, backward); forward: (x_out, z) tensors; grads: (dz, dx_out, x_out, x,
    dx, dy, dgate, dscale, dpostw, dprew)."""
    width = x.shape[-1]
    if not 0 < width <= RESIDUAL_NORM_MAX_WIDTH:
        raise ValueError(f"the width must be within 1 .. {RESIDUAL_NORM_MAX_WIDTH} (got {width})")
    rows = x.numel() // width
    batch, s = (x.shape[0], rows // x.shape[0] if x.shape[0] else 0) if x.dim() > 2 else (1, rows)
    kind = g_ptr = g_step = 0
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a torch.Tensor")
        if y is None:
            raise ValueError("a gate without a block's output")
        if gate.shape == x.shape and gate.dim() > 1:
            _tensor(gate, "gate", y.dtype, dev)
            kind, g_step = 3, _rows(gate, "gate")
        elif x.dim() > 2 and gate.dim() == 2:
            _exactly(gate, "gate", _F32, dev, (batch, width))
            kind = 2
        else:
            _exactly(gate, "gate", _F32, dev, (width,))
            kind = 1
        g_ptr = gate.data_ptr()
    ptrs = []
    for t, name in ((scale, "residual_scale"), (post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if t is not None:
            _exactly(t, name, _F32, dev, (width,))
        ptrs.append(0 if t is None else t.data_ptr())
    p, key, first, state = _drop_args(p, seed, offset, dev)
    if y is None:
        post = False
        if p:
            raise ValueError("dropout without a block's output")
    if post_weight is not None and not post:
        raise ValueError("post_weight without the post norm")
    y_ptr, y_step = (0, 0) if y is None else (y.data_ptr(), _rows(y, "y"))
    a = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    r = lambda t, name: 0 if t is None else _rows(t, name)  # noqa: E731
    if forward is not None:
        x_out, z = forward
        return _RESID.pack(x.data_ptr(), y_ptr, g_ptr, *ptrs, a(x_out), a(z), *(0,) * 8, _rows(x, "x"), y_step, g_step,
                           0, 0, 0, batch, s, width, _DTYPE[x.dtype], _DTYPE[dtype], y is not None, bool(post), kind,
                           float(eps), p, key, first, state)
    dz, dx_out, x_out, x_in, dx, dy, dgate, dscale, dpostw, dprew = grads
    return _RESID.pack(a(x_in), y_ptr, g_ptr, *ptrs, x_out.data_ptr(), 0, dz.data_ptr(), a(dx_out), a(dx), a(dy),
                       a(dgate), a(dscale), a(dpostw), a(dprew), r(x_in, "x"), y_step, g_step, _rows(x_out, "x_out"),
                       _rows(dz, "dz"), r(dx_out, "dx_out"), batch, s, width, _DTYPE[x_out.dtype], _DTYPE[dtype],
                       y is not None, bool(post), kind, float(eps), p, key, first, state)


def _resid_types(x, y, dev, name):
    if y is not None and isinstance(y, torch.Tensor) and x.dtype is _BF16 and y.dtype is _BF16 and x.is_cuda and y.device == dev \
            and x.shape == y.shape and x.dim():
        return
    _tensor(x, name, (_F32, _BF16), dev)
    if x.dim() < 1:
        raise ValueError(f"{name} must have a last dimension")
    if y is not None:
        _tensor(y, "y", (_F32, _BF16), dev)
        if y.shape != x.shape:
            raise ValueError(f"y must have the shape of {name}, {tuple(x.shape)} (got {tuple(y.shape)})")
        if y.dtype is _F32 and x.dtype is _BF16:
            raise TypeError("a float32 block on a bfloat16 stream")


def residual_norm(x, y=None, gate=None, residual_scale=None, post_weight=None, pre_weight=None, post=True, eps=1e-6,
                  p=0.0, seed=0, offset=0, dtype=None, x_out=None, z_out=None):
    """The norms before and after a block of a decoder layer, in one pass over
    each row of the residual stream ``x`` (..., width) and the block's output
    ``y`` (shaped as x; both float32 or bfloat16, a float32 y only with a
    float32 x; rows one stride apart):

        n     = y / sqrt(mean(y^2) + eps) post_weight     (``post``; else y)
        n     = dropout(n, p, seed, offset)
        x_out = residual_scale x + gate n
        z     = x_out / sqrt(mean(x_out^2) + eps) pre_weight

    Returns ``(x_out, z)``: the stream, of x's type, and the next block's input,
    of y's.  ``gate`` is a float32 vector (width,), a float32 vector for each
    sequence (x.shape[0], width) of an x of 3 dimensions or more, or a tensor
    of y's shape and type; ``residual_scale`` and the weights are float32
    vectors (width,).  What is None is one.  ``seed`` and ``offset`` as in
    ``dropout``, elements counted in rows of x.

    Without ``y``, as in front of the first block, z is the norm of
    residual_scale x, of type ``dtype`` (default x's).

    Computed in float32, rounded once.  Widths up to 8192; a multiple of 8 with
    rows aligned to 16 bytes runs fastest.  ``x_out`` may be x and ``z_out`` y,
    where those are contiguous; else given outputs must not share memory with
    anything."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    _resid_types(x, y, dev, "x")
    if y is not None:
        if dtype is not None and dtype != y.dtype:
            raise TypeError(f"z has y's type {y.dtype}, not {dtype}")
        dtype = y.dtype
    else:
        dtype = x.dtype if dtype is None else dtype
        _float_type(dtype, "dtype")
        if dtype is _F32 and x.dtype is _BF16:
            raise TypeError("a float32 block on a bfloat16 stream")
    given = x_out, z_out
    if x_out is None:
        x_out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _exactly(x_out, "x_out", x.dtype, dev, x.shape)
    if z_out is None:
        z_out = torch.empty(x.shape, dtype=dtype, device=dev)
    else:
        _exactly(z_out, "z_out", dtype, dev, x.shape)
    args = _resid_args(x, y, gate, residual_scale, post_weight, pre_weight, post, eps, p, seed, offset, dtype,
                       (x_out, z_out), None, dev)
    if given[0] is not None or given[1] is not None:
        reads = ((gate, "gate"), (residual_scale, "residual_scale"), (post_weight, "post_weight"),
                 (pre_weight, "pre_weight"), (seed if isinstance(seed, torch.Tensor) else None, "seed"))
        if given[0] is not None:
            _apart(x_out, "x_out", (x, "x", True), (y, "y"), *reads, (given[1], "z_out"))
        if given[1] is not None:
            _apart(z_out, "z_out", (x, "x"), (y, "y", True), *reads)
    _call(dev, _lib.muon_residual_norm, args)
    return x_out, z_out


def residual_norm_backward(dz, dx_out, x_out, y=None, x=None, gate=None, residual_scale=None, post_weight=None,
                           pre_weight=None, post=True, eps=1e-6, p=0.0, seed=0, offset=0, dx=None, dy=None,
                           workspace=None):
    """Gradients ``(dx, dy, dgate, dresidual_scale, dpost_weight, dpre_weight)``
    of ``residual_norm`` from ``dz`` and ``dx_out`` (None: zeros), the gradients
    of its results, its result ``x_out`` and its arguments; None for what was
    not given.  ``x`` is needed with a residual_scale only.  dx has x_out's
    type, dy and dz y's (without y dz is float32 or bfloat16), dgate is as gate,
    the others are float32; sums over rows are float32, in one order.  A row of a
    padded batch whose dz and dx_out are zeros adds nothing to them if it is
    finite in x, y and x_out (and, with an eps of 0, not all zeros there).  A
    given ``dx`` may be dx_out, and a given ``dy`` dz or y, where those are
    contiguous; else they must not share memory with anything."""
    if not isinstance(x_out, torch.Tensor):
        raise TypeError("x_out must be a torch.Tensor")
    dev = x_out.device
    _resid_types(x_out, y, dev, "x_out")
    _tensor(dz, "dz", (_F32, _BF16) if y is None else y.dtype, dev)
    if dz.dtype is _F32 and x_out.dtype is _BF16:
        raise TypeError("a float32 block on a bfloat16 stream")
    x_in = None
    if residual_scale is not None:
        if x is None:
            raise TypeError("x is needed for the gradient of residual_scale")
        x_in = x
    for t, name in ((dx_out, "dx_out"), (x_in, "x")):
        if t is not None:
            _tensor(t, name, x_out.dtype, dev)
    for t, name in ((dz, "dz"), (dx_out, "dx_out"), (x_in, "x")):
        if t is not None and t.shape != x_out.shape:
            raise ValueError(f"{name} must have x_out's shape {tuple(x_out.shape)} (got {tuple(t.shape)})")
    given = dx, dy
    if dx is None:
        dx = torch.empty_like(x_out, memory_format=torch.contiguous_format)
    else:
        _exactly(dx, "dx", x_out.dtype, dev, x_out.shape)
    if y is None:
        if dy is not None:
            raise ValueError("dy without y")
    elif dy is None:
        dy = torch.empty_like(y, memory_format=torch.contiguous_format)
    else:
        _exactly(dy, "dy", y.dtype, dev, y.shape)
    grads = [None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)
             for t in (gate, residual_scale, post_weight, pre_weight)]
    args = _resid_args(x_out, y, gate, residual_scale, post_weight, pre_weight, post, eps, p, seed, offset, dz.dtype,
                       None, (dz, dx_out, x_out, x_in, dx, dy, *grads), dev)
    if given[0] is not None or given[1] is not None:
        reads = ((x_out, "x_out"), (x_in, "x"), (gate, "gate"), (residual_scale, "residual_scale"),
                 (post_weight, "post_weight"), (pre_weight, "pre_weight"),
                 (seed if isinstance(seed, torch.Tensor) else None, "seed"))
        if given[0] is not None:
            _apart(dx, "dx", (dx_out, "dx_out", True), (dz, "dz"), (y, "y"), *reads, (given[1], "dy"))
        if given[1] is not None:
            _apart(dy, "dy", (dx_out, "dx_out"), (dz, "dz", True), (y, "y", True), *reads)
    ptr, size, ws = _ws(workspace, _lib.muon_residual_norm_backward_workspace_size(args) or 256, dev)
    _call(dev, _lib.muon_residual_norm_backward, args, ptr, size)
    return dx, dy, *grads


def _matrix(t, name, dev, shape=None):
    """The stride between the rows of a bfloat16 tensor on `dev`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.is_cuda and t.device == dev
            and (shape is None or t.shape == shape)):
        _tensor(t, name, _BF16, dev, None if shape is None else len(shape))
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return _rows(t, name)


def _ffn_sizes(x, w_gate, w_up, w_down, activation):
    """Checks the forward pass's arguments: (device, (tokens, width, hidden), row strides of x, gate and up, down)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    x_step = _matrix(x, "x", dev)
    w_step = _matrix(w_gate, "w_gate", dev)
    if w_gate.dim() != 2 or x.shape[-1] != w_gate.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} does not fit w_gate {tuple(w_gate.shape)}")
    hidden, width = w_gate.shape
    if _matrix(w_up, "w_up", dev, w_gate.shape) != w_step:
        raise ValueError("the rows of w_gate and w_up must be the same stride apart")
    down_step = _matrix(w_down, "w_down", dev, (width, hidden))
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)} (got {activation!r})")
    return dev, (x.numel() // width if width else 0, width, hidden), (x_step, w_step, down_step)


def feed_forward(x, w_gate, w_up, w_down, activation="silu", keep=False, out=None, workspace=None):
    """The gated feed-forward block of bfloat16 ``x`` (..., width):

        (activation(x w_gate^T) * (x w_up^T)) w_down^T

    with ``w_gate`` and ``w_up`` (hidden, width) and ``w_down`` (width, hidden),
    bfloat16; returns a new (or given, contiguous) tensor of x's shape.
    ``activation``: "silu", "gelu" (erf), "gelu_tanh" or "relu".  With ``keep``
    it returns ``(out, kept)``: kept (3, tokens, hidden) holds what
    ``feed_forward_backward`` needs, the gate, the up projection and their
    product, rounded to bfloat16.

    width and hidden are multiples of 8; rows are aligned to 16 bytes and one
    stride (a multiple of 8) apart, the same for w_gate and w_up, so the halves
    of one matrix serve.  Sums are float32; the hidden values are rounded once.
    A given ``out`` must not share memory with anything."""
    dev, sizes, steps = _ffn_sizes(x, w_gate, w_up, w_down, activation)
    given = out
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _exactly(out, "out", _BF16, dev, x.shape)
    kept = torch.empty((3, sizes[0], sizes[2]), dtype=_BF16, device=dev) if keep else None
    args = _FFN.pack(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), out.data_ptr(),
                     kept.data_ptr() if keep else 0, 0, 0, 0, 0, 0, *steps, 0, *sizes, ACTIVATIONS[activation],
                     muon.MUON_BF16)
    if given is not None:
        _apart(out, "out", (x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"))
    ptr, size, ws = _ws(workspace, _lib.muon_feed_forward_workspace_size(args) or 256, dev)
    _call(dev, _lib.muon_feed_forward, args, ptr, size)
    return (out, kept) if keep else out


def feed_forward_backward(dout, x, w_gate, w_up, w_down, kept, activation="silu", dtype=_BF16, dx=None,
                          workspace=None):
    """Gradients ``(dx, dw_gate, dw_up, dw_down)`` of ``feed_forward`` from
    ``dout``, its arguments and what it kept.  dx is bfloat16; the matrices'
    gradients are contiguous and of ``dtype`` (bfloat16, or float32: their sums
    as they are).  The gradients of the gate and of the up projection are
    rounded to bfloat16 once on the way.  A token of a padded batch whose dout is
    zero adds nothing to the matrices' gradients if it is finite in x and kept.
    A given ``dx`` must not share memory with anything."""
    dev, sizes, steps = _ffn_sizes(x, w_gate, w_up, w_down, activation)
    dout_step = _matrix(dout, "dout", dev, x.shape)
    _float_type(dtype, "dtype")
    _exactly(kept, "kept", _BF16, dev, (3, sizes[0], sizes[2]))
    given = dx
    if dx is None:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _exactly(dx, "dx", _BF16, dev, x.shape)
    dws = [torch.empty(w.shape, dtype=dtype, device=dev) for w in (w_gate, w_up, w_down)]
    args = _FFN.pack(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), 0, kept.data_ptr(),
                     dout.data_ptr(), dx.data_ptr(), *[t.data_ptr() for t in dws], *steps, dout_step, *sizes,
                     ACTIVATIONS[activation], _DTYPE[dtype])
    if given is not None:
        _apart(dx, "dx", (dout, "dout"), (x, "x"), (w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down"),
               (kept, "kept"))
    ptr, size, ws = _ws(workspace, _lib.muon_feed_forward_backward_workspace_size(args) or 256, dev)
    _call(dev, _lib.muon_feed_forward_backward, args, ptr, size)
    return dx, *dws

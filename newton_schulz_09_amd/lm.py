"""Python binding of the language-model operators of libmuon.so (C ABI in
include/muon_lm.h): attention, the norm and rotation of query and key heads,
and the embedding, each with its gradients.

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
                                           _vp])):
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args

#: Every symbol include/muon_lm.h declares.
EXPORTS = ("muon_attention_workspace_size", "muon_attention_backward_workspace_size", "muon_attention",
           "muon_attention_backward", "muon_qk_norm_rope_backward_workspace_size", "muon_qk_norm_rope",
           "muon_qk_norm_rope_backward", "muon_embedding", "muon_embedding_backward_workspace_size",
           "muon_embedding_backward")
#: Largest head sizes (MUON_ATTENTION_MAX_D, MUON_QK_NORM_MAX_D).
ATTENTION_MAX_D = 128
QK_NORM_MAX_D = 512

_F32, _BF16 = torch.float32, torch.bfloat16
_DTYPE = {_F32: muon.MUON_F32, _BF16: muon.MUON_BF16}
# muon_attention_args and muon_qk_norm_rope_args: 8-byte fields throughout
_ATTN = struct.Struct("9Q15q2Qq3Q8q2d")
_QK = struct.Struct("10Q12q2qQqQ3qqd")


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

"""Serving a model stored in codes: the calls of a token-by-token decode step.

Products of a few rows with int4 weights that carry group scales, an int8
key/value cache with the attention over it, and log probabilities of the
logits with their gradient.  A thin binding like the rest of the package: each
call checks and marshals its arguments and launches the library's kernels on
the current PyTorch stream (or the ``stream`` given, which waits for no other: its
arguments have to be there and to stay; what the call makes is of that stream's
memory).  Activations are
float32, float16 or bfloat16 CUDA tensors whose last dimension is contiguous;
their other strides are free, but for 2-D ones, whose rows must not overlap (an
expanded row is refused).  Data-dependent conditions are OR-ed into
``dstatus`` (an int32 CUDA tensor, or None) as DSTATUS_* bits.  A call given no
``workspace`` uses one of its stream's own, so calls on different streams may
overlap; a graph uses the one of the stream it was captured on (whose buffer is kept
for it when a later call needs a larger one), so graphs that may overlap with one another
or with calls on that stream need workspaces of their own.  There is no
CPU fallback and no autograd: gradients have calls of their own.
"""
from __future__ import annotations

import functools
import struct
from typing import NamedTuple

import torch

import verifiable_quantize_rows_gb300 as _bsg

__all__ = ["Kv8Cache", "wquant_groups", "wgroups_matvec", "wcols_matmul", "kv8_append", "kv8_attend",
           "kv8_attend_window", "kv8_attend_shared", "logprobs", "logprobs_backward", "Logprobs", "MATVEC_MAX_M", "KV8_MAX_T", "MAX_TOP"]

MATVEC_MAX_M = 16
KV8_MAX_T = 16
MAX_TOP = 32

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


# The C structs bsg_kv8_cache and bsg_tokens, packed (a call takes microseconds; a
# ctypes structure would be one of them).
_CACHE = struct.Struct("@PPPPqiii4x")
_TOKENS = struct.Struct("@Pqqq")


class Kv8Cache(NamedTuple):
    """A pool of pages: k, v int8 (pages, heads, page_tokens, dim); k_scale,
    v_scale float32 (pages, heads).  Any tuple of such tensors will do."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, pages: int, heads: int, page_tokens: int, dim: int, device="cuda"):
        """A pool of unwritten pages (nothing has to be cleared)."""
        codes = [torch.empty((pages, heads, page_tokens, dim), dtype=torch.int8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros((pages, heads), dtype=torch.float32, device=device)
                  for _ in range(2)]
        return cls(*codes, *scales)


class Logprobs(NamedTuple):
    """What logprobs() returns: float32 (rows,), (rows,), (rows,), (rows, top)
    and int32 (rows, top)."""
    logprob: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_logprob: torch.Tensor
    top_id: torch.Tensor


# The checks below cost a decode step as much as its small kernels take, so each
# is one condition that a good argument passes; what is wrong is said after.
def _activation(t, dim: int, name: str) -> int:
    """The C dtype of an activation tensor, checked."""
    code = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or not t.is_cuda:
        raise TypeError(f"{name} must be a float32, float16 or bfloat16 CUDA tensor")
    if t.dim() != dim or not t.numel() or (t.stride(-1) != 1 and t.shape[-1] != 1):
        raise ValueError(f"{name} must be a non-empty {dim}-D tensor with a contiguous last dimension")
    return code


def _exact(t, dtype, shape, name: str, device) -> int:
    """The address of a contiguous tensor of this dtype and shape, on `device`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device.index \
            and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be a tensor of dtype {dtype} on {device}")
    raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")


def _rows(t, name: str) -> int:
    """The leading dimension of a 2-D tensor (its row stride; one row has any)."""
    rows, n = t.shape
    if rows == 1:
        return n
    ld = t.stride(0)
    if ld >= n:
        return ld
    raise ValueError(f"the rows of {name} must not overlap: they are {ld} apart and {n} long")


def _made(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    # of `stream`'s memory: what the current stream has freed it may still be using
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _output(out, like, shape, stream):
    """`out`, checked, or a new tensor of `like`'s dtype."""
    if out is None:
        return _made(shape, like.dtype, like.device, stream)
    if not isinstance(out, torch.Tensor) or out.dtype != like.dtype or out.device != like.device:
        raise TypeError(f"out must be a tensor of dtype {like.dtype} on {like.device}")
    if out.shape != shape or (out.stride(-1) != 1 and out.shape[-1] != 1):
        raise ValueError(f"out must have shape {tuple(shape)} and a contiguous last dimension")
    return out


# The current stream's handle: the stream object that torch.cuda.current_stream
# makes takes 2 us.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _stream(stream, device) -> int:
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _status(dstatus, device):
    return None if dstatus is None else _exact(dstatus, torch.int32, (1,), "dstatus", device)


def _lib():
    return _bsg._lib or _bsg.load()


# The default workspaces, one for each stream of a device: calls on different
# streams may overlap.
_default_ws: dict = {}


def _workspace(workspace, need: int, device, stream, handle: int):
    """(address, size) of the workspace given, or of the stream's default one."""
    if workspace is None:
        workspace = _default_ws.get((device.index, handle))
        if workspace is None:
            workspace = _default_ws.setdefault((device.index, handle), _bsg.Workspace(device))
    buf = workspace.buf
    if buf is None or buf.numel() < need or not workspace.captured and (stream is not None or _capturing()):
        with torch.cuda.stream(stream):  # whose memory it is to be (None: the current one's)
            buf = workspace.get(need)
    return buf.data_ptr(), buf.numel()


# ---------------------------------------------------------------------------
def wquant_groups(W, group: int = 64, dstatus=None, stream=None):
    """Store a K x N float32 weight as int4 codes with one scale per `group`
    rows (a multiple of 32; 0: all of them) and column: (Q, scale).  Q: uint8
    (K, ceil(N/2)), two codes per byte, a view of rows padded to 16 bytes;
    scale: float32 (ceil(K/group), N)."""
    if _activation(W, 2, "W") != 0:
        raise TypeError("W must be float32")
    K, N = W.shape
    if group < 0 or group % 32:
        raise ValueError("group must be a multiple of 32, or 0")
    half = (N + 1) // 2
    Q = _made((K, (half + 15) // 16 * 16), torch.uint8, W.device, stream)
    scale = _made(((K + group - 1) // group if group else 1, N), torch.float32, W.device, stream)
    _bsg._check(_lib().bsg_wquant_groups(
        W.data_ptr(), K, N, _rows(W, "W"), group, Q.data_ptr(), Q.shape[1], scale.data_ptr(), N,
        _status(dstatus, W.device), _stream(stream, W.device)), "bsg_wquant_groups")
    return Q[:, :half], scale


@functools.lru_cache(maxsize=1024)
def _matvec_bytes(M: int, N: int, K: int) -> int:
    return _lib().bsg_wgroups_matvec_workspace_size(M, N, K)


def wgroups_matvec(X, Q, scale, group: int = 64, relu: bool = False, out=None, dstatus=None,
                   stream=None, workspace=None):
    """Y = X . W_hat (+ReLU) for up to MATVEC_MAX_M rows of X (M x K) and a
    weight stored by wquant_groups -- or by wquant_cols with bits=4, with
    group=0 and scale viewed as (1, N).  Y: M x N of X's dtype; `out` must not
    share X's memory."""
    code = _activation(X, 2, "X")
    dev = X.device
    M, K = X.shape
    if M > MATVEC_MAX_M:
        raise ValueError(f"at most {MATVEC_MAX_M} rows a call: X has {M}")
    if group < 0 or group % 32:
        raise ValueError("group must be a multiple of 32, or 0")
    if not isinstance(scale, torch.Tensor) or scale.dtype is not torch.float32 or scale.get_device() != dev.index:
        raise TypeError(f"scale must be a float32 tensor on {dev}")
    if scale.dim() != 2 or scale.stride(1) != 1 and scale.shape[1] != 1 \
            or scale.shape[0] != ((K + group - 1) // group if group else 1):
        raise ValueError("scale must be (groups, N), one row per group of rows of the weight")
    N = scale.shape[1]
    if not isinstance(Q, torch.Tensor) or Q.dtype is not torch.uint8 or Q.get_device() != dev.index:
        raise TypeError(f"Q must be a uint8 tensor on {dev}")
    if Q.shape != (K, (N + 1) // 2) or Q.stride(1) != 1 and Q.shape[1] != 1:
        raise ValueError("Q must be (K, ceil(N/2)) with contiguous rows")
    Y = _output(out, X, (M, N), stream)
    if Y.data_ptr() == X.data_ptr():  # one CTA's columns of Y would be another's X
        raise ValueError("out must not share X's memory")
    need = _matvec_bytes(M, N, K)
    on = _stream(stream, dev)
    wp, wn = _workspace(workspace, need, dev, stream, on) if need else (None, 0)
    _bsg._check(_lib().bsg_wgroups_matvec(
        X.data_ptr(), code, _rows(X, "X"), Q.data_ptr(), _rows(Q, "Q"), scale.data_ptr(), _rows(scale, "scale"),
        group, M, N, K, bool(relu), Y.data_ptr(), _rows(Y, "out"), wp, wn, _status(dstatus, dev), on),
        "bsg_wgroups_matvec")
    return Y


@functools.lru_cache(maxsize=1024)
def _matmul_bytes(M: int, N: int, K: int) -> int:
    return _lib().bsg_wcols_matmul_workspace_size(M, N, K)


def wcols_matmul(X, Q, scale, relu: bool = False, out=None, dstatus=None, stream=None, workspace=None):
    """Y = X . W_hat (+ReLU) in 8-bit integers for any number of rows of X (M x K)
    and a weight stored by wquant_cols with bits=8: Q int8 (K, N), scale float32
    (N,).  Each row of X is quantized by itself, by quantize_rows' rule; the sums of
    code products are exact.  Y: M x N of X's dtype; `out` must not share X's
    memory."""
    code = _activation(X, 2, "X")
    dev = X.device
    M, K = X.shape
    if not isinstance(Q, torch.Tensor) or Q.dtype is not torch.int8 or Q.get_device() != dev.index:
        raise TypeError(f"Q must be an int8 tensor on {dev}")
    if Q.dim() != 2 or Q.shape[0] != K or not Q.shape[1] or Q.stride(1) != 1 and Q.shape[1] != 1:
        raise ValueError("Q must be (K, N) with contiguous rows")
    if K > _bsg.MAX_K:
        raise ValueError(f"at most {_bsg.MAX_K} columns of X")
    N = Q.shape[1]
    sp = _exact(scale, torch.float32, (N,), "scale", dev)
    Y = _output(out, X, (M, N), stream)
    if Y.data_ptr() == X.data_ptr():
        raise ValueError("out must not share X's memory")
    need = _matmul_bytes(M, N, K)
    on = _stream(stream, dev)
    wp, wn = _workspace(workspace, need, dev, stream, on) if need else (None, 0)
    _bsg._check(_lib().bsg_wcols_matmul(
        X.data_ptr(), code, _rows(X, "X"), Q.data_ptr(), _rows(Q, "Q"), sp, M, N, K, bool(relu), Y.data_ptr(),
        _rows(Y, "out"), wp, wn, _status(dstatus, dev), on), "bsg_wcols_matmul")
    return Y


# ---------------------------------------------------------------------------
def _cache(cache, device):
    """(bsg_kv8_cache, heads, page_tokens, dim), checked."""
    k, v, ks, vs = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("the cache's k must be (pages, heads, page_tokens, dim)")
    pages, heads, page_tokens, dim = shape = k.shape
    per_page = (pages, heads)
    packed = _CACHE.pack(_exact(k, torch.int8, shape, "k", device), _exact(v, torch.int8, shape, "v", device),
                         _exact(ks, torch.float32, per_page, "k_scale", device),
                         _exact(vs, torch.float32, per_page, "v_scale", device), pages, heads, page_tokens, dim)
    return packed, heads, page_tokens, dim


def _tokens(t):
    s = t.stride()
    return _TOKENS.pack(t.data_ptr(), s[0], s[1], s[2])


def _table(table, B: int, device):
    if not isinstance(table, torch.Tensor) or table.dim() != 2 or table.shape[0] != B:
        raise ValueError("table must be (batch, pages of a sequence)")
    return _exact(table, torch.int32, table.shape, "table", device)


def kv8_append(k, v, cache, table, starts, counts=None, dstatus=None, stream=None):
    """Append k and v (batch, tokens, heads, dim) to the cache's pages: token t
    of sequence b at position starts[b] + t, for t < counts[b] (all of them
    where counts is None).  table: int32 (batch, pages of a sequence); starts,
    counts: int32 (batch,).  The cache is updated in place."""
    code = _activation(k, 4, "k")
    dev = k.device
    if _activation(v, 4, "v") != code or v.shape != k.shape or v.device != dev:
        raise ValueError("k and v must have the same shape, dtype and device")
    B, T, H, D = k.shape
    c, heads, _, dim = _cache(cache, dev)
    if H != heads or D != dim:
        raise ValueError(f"the cache has {heads} heads of {dim}")
    _bsg._check(_lib().bsg_kv8_append(
        c, _table(table, B, dev), table.shape[1], _exact(starts, torch.int32, (B,), "starts", dev),
        None if counts is None else _exact(counts, torch.int32, (B,), "counts", dev), _tokens(k),
        _tokens(v), code, B, T, _status(dstatus, dev), _stream(stream, dev)), "bsg_kv8_append")


@functools.lru_cache(maxsize=1024)
def _attend_bytes(pages: int, heads: int, page_tokens: int, dim: int, width: int, B: int, T: int, H: int) -> int:
    anything = _CACHE.pack(256, 256, 256, 256, pages, heads, page_tokens, dim)  # its addresses do not matter
    return _lib().bsg_kv8_attend_workspace_size(anything, width, B, T, H)


def kv8_attend(q, cache, table, lens, scale: float | None = None, out=None, lse=None,
               dstatus=None, stream=None, workspace=None):
    """Attention of the newest T tokens (at most KV8_MAX_T) of each sequence
    over the cache.  q: (batch, T, heads, dim), heads a multiple of the
    cache's; lens: int32 (batch,), tokens cached with the new ones; scale:
    dim ** -0.5 by default.  Returns out, of q's shape and dtype; a query that
    sees no position gives zeros.  lse: float32 (batch, T, heads) to be filled,
    or None."""
    code = _activation(q, 4, "q")
    dev = q.device
    B, T, H, D = q.shape
    c, heads, page_tokens, dim = _cache(cache, dev)
    if D != dim or H % heads:
        raise ValueError(f"the cache has {heads} heads of {dim}")
    if T > KV8_MAX_T:
        raise ValueError(f"at most {KV8_MAX_T} tokens a sequence: q has {T}")
    O = _output(out, q, q.shape, stream)
    tp, width = _table(table, B, dev), table.shape[1]
    on = _stream(stream, dev)
    wp, wn = _workspace(workspace, _attend_bytes(cache[0].shape[0], heads, page_tokens, dim, width, B, T, H), dev,
                        stream, on)
    _bsg._check(_lib().bsg_kv8_attend(
        c, tp, width, _exact(lens, torch.int32, (B,), "lens", dev), _tokens(q), _tokens(O), code, B, T, H,
        D ** -0.5 if scale is None else scale,
        None if lse is None else _exact(lse, torch.float32, (B, T, H), "lse", dev), wp, wn,
        _status(dstatus, dev), on), "bsg_kv8_attend")
    return O


@functools.lru_cache(maxsize=1024)
def _window_bytes(pages: int, heads: int, page_tokens: int, dim: int, width: int, B: int, T: int, H: int,
                  window: int, sinks: int) -> int:
    anything = _CACHE.pack(256, 256, 256, 256, pages, heads, page_tokens, dim)
    return _lib().bsg_kv8_attend_window_workspace_size(anything, width, B, T, H, window, sinks)


def _apart(O, q):
    if O.data_ptr() == q.data_ptr():
        raise ValueError("out must not share q's memory")


def kv8_attend_window(q, cache, table, lens, window: int = 0, sinks: int = 0, counts=None,
                      scale: float | None = None, out=None, lse=None, dstatus=None, stream=None,
                      workspace=None):
    """Attention of any number of new tokens of each sequence over the cache: a
    query at position i sees the positions j <= i with j > i - window or j < sinks
    (window 0: all of them).  q: (batch, T, heads, dim), heads a multiple of the
    cache's; counts: int32 (batch,), how many of the T tokens of each sequence are
    there (None: all); lens: int32 (batch,), tokens cached with the new ones.
    Returns out, of q's shape and dtype (not q's memory), in which tokens past a
    sequence's count are left as they were; a query that sees no position gives
    zeros.  lse: float32 (batch, T, heads) to be filled, or None."""
    code = _activation(q, 4, "q")
    dev = q.device
    B, T, H, D = q.shape
    c, heads, page_tokens, dim = _cache(cache, dev)
    if D != dim or H % heads:
        raise ValueError(f"the cache has {heads} heads of {dim}")
    if not (0 <= window < 1 << 31 and 0 <= sinks < 1 << 31):
        raise ValueError("window and sinks must be 0 or more, and below 2^31")
    O = _output(out, q, q.shape, stream)
    _apart(O, q)
    tp, width = _table(table, B, dev), table.shape[1]
    on = _stream(stream, dev)
    wp, wn = _workspace(workspace, _window_bytes(cache[0].shape[0], heads, page_tokens, dim, width, B, T, H,
                                                 window, sinks), dev, stream, on)
    _bsg._check(_lib().bsg_kv8_attend_window(
        c, tp, width, _exact(lens, torch.int32, (B,), "lens", dev),
        None if counts is None else _exact(counts, torch.int32, (B,), "counts", dev), _tokens(q), _tokens(O),
        code, B, T, H, window, sinks, D ** -0.5 if scale is None else scale,
        None if lse is None else _exact(lse, torch.float32, (B, T, H), "lse", dev), wp, wn,
        _status(dstatus, dev), on), "bsg_kv8_attend_window")
    return O


@functools.lru_cache(maxsize=1024)
def _shared_bytes(pages: int, heads: int, page_tokens: int, dim: int, prefix: int, width: int, B: int, T: int,
                  H: int) -> int:
    anything = _CACHE.pack(256, 256, 256, 256, pages, heads, page_tokens, dim)
    return _lib().bsg_kv8_attend_shared_workspace_size(anything, prefix, width, B, T, H)


def kv8_attend_shared(q, cache, prefix, prefix_len, table, lens, scale: float | None = None, out=None,
                      lse=None, dstatus=None, stream=None, workspace=None):
    """kv8_attend for sequences that begin with the same tokens, whose part of the
    cache is read once for all of them.  prefix: int32 (pages,), the pages of the
    common tokens; prefix_len: int32 (1,), how many there are.  table, lens: each
    sequence's own tokens behind them, which begin a page of their own; lens counts
    these alone, with the new ones.  A query sees the whole prefix and its own
    sequence up to itself; one before its sequence's first own token (lens below T; a
    slot of length 0 is idle) gives zeros.  q, out (not q's memory) and lse are
    kv8_attend's."""
    code = _activation(q, 4, "q")
    dev = q.device
    B, T, H, D = q.shape
    c, heads, page_tokens, dim = _cache(cache, dev)
    if D != dim or H % heads:
        raise ValueError(f"the cache has {heads} heads of {dim}")
    if T > KV8_MAX_T:
        raise ValueError(f"at most {KV8_MAX_T} tokens a sequence: q has {T}")
    if not isinstance(prefix, torch.Tensor) or prefix.dim() != 1 or not prefix.numel():
        raise ValueError("prefix must be (pages of the prefix,), one page at least")
    O = _output(out, q, q.shape, stream)
    _apart(O, q)
    tp, width, pages = _table(table, B, dev), table.shape[1], prefix.shape[0]
    on = _stream(stream, dev)
    wp, wn = _workspace(workspace, _shared_bytes(cache[0].shape[0], heads, page_tokens, dim, pages, width, B, T, H),
                        dev, stream, on)
    _bsg._check(_lib().bsg_kv8_attend_shared(
        c, _exact(prefix, torch.int32, (pages,), "prefix", dev), pages,
        _exact(prefix_len, torch.int32, (1,), "prefix_len", dev), tp, width,
        _exact(lens, torch.int32, (B,), "lens", dev), _tokens(q), _tokens(O), code, B, T, H,
        D ** -0.5 if scale is None else scale,
        None if lse is None else _exact(lse, torch.float32, (B, T, H), "lse", dev), wp, wn,
        _status(dstatus, dev), on), "bsg_kv8_attend_shared")
    return O


# ---------------------------------------------------------------------------
def logprobs(logits, target=None, top: int = 0, dstatus=None, stream=None) -> Logprobs:
    """Per row of logits (rows, vocab): the log probability of the row's target
    (int64 (rows,); negative or None: no token given, 0), the entropy, the log
    of the softmax's denominator, and the `top` largest log probabilities with
    their tokens, the lowest token first among equals."""
    code = _activation(logits, 2, "logits")
    dev = logits.device
    M, V = logits.shape
    if not 0 <= top <= min(MAX_TOP, V):
        raise ValueError(f"top must be 0 to {min(MAX_TOP, V)}")
    tp = None if target is None else _exact(target, torch.int64, (M,), "target", dev)
    lp, ent, lse = _made((3, M), torch.float32, dev, stream).unbind()
    tl = _made((M, top), torch.float32, dev, stream)
    ti = _made((M, top), torch.int32, dev, stream)
    _bsg._check(_lib().bsg_logprobs(
        logits.data_ptr(), code, M, V, _rows(logits, "logits"), tp, top, lp.data_ptr(), ent.data_ptr(),
        lse.data_ptr(), tl.data_ptr(), ti.data_ptr(), _status(dstatus, dev),
        _stream(stream, dev)), "bsg_logprobs")
    return Logprobs(lp, ent, lse, tl, ti)


def logprobs_backward(logits, target, lse, entropy=None, g_logprob=None, g_entropy=None, out=None,
                      dstatus=None, stream=None):
    """The gradient of the log probabilities and entropies that logprobs() gave
    for these logits, with respect to them: g_logprob, g_entropy (float32
    (rows,), or None for zeros) come in, a tensor like logits goes out.  `out`
    may be the logits themselves."""
    code = _activation(logits, 2, "logits")
    dev = logits.device
    M, V = logits.shape
    if g_entropy is not None and entropy is None:
        raise ValueError("g_entropy needs the entropy that logprobs() gave")
    per_row = [None if t is None else _exact(t, torch.float32, (M,), name, dev)
               for t, name in ((lse, "lse"), (entropy, "entropy"), (g_logprob, "g_logprob"),
                               (g_entropy, "g_entropy"))]
    tp = None if target is None else _exact(target, torch.int64, (M,), "target", dev)
    D = _output(out, logits, (M, V), stream)
    _bsg._check(_lib().bsg_logprobs_backward(
        logits.data_ptr(), code, M, V, _rows(logits, "logits"), tp, *per_row, D.data_ptr(), _rows(D, "out"),
        _status(dstatus, dev), _stream(stream, dev)), "bsg_logprobs_backward")
    return D

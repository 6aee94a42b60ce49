"""Serving a model stored in codes: the calls of a token-by-token decode step.

Products of a few rows with int4 weights that carry group scales, an int8
key/value cache with the attention over it, and log probabilities of the
logits with their gradient.  A thin binding like the rest of the package: each
call checks and marshals its arguments and launches the library's kernels on
the current PyTorch stream (or the ``stream`` given).  Activations are
float32, float16 or bfloat16 CUDA tensors whose last dimension is contiguous;
their other strides are free.  Data-dependent conditions are OR-ed into
``dstatus`` (an int32 CUDA tensor, or None) as DSTATUS_* bits.  There is no
CPU fallback and no autograd: gradients have calls of their own.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

import verifiable_quantize_rows_gb300 as _bsg

__all__ = ["Kv8Cache", "wquant_groups", "wgroups_matvec", "kv8_append", "kv8_attend", "logprobs",
           "logprobs_backward", "Logprobs", "MATVEC_MAX_M", "KV8_MAX_T", "MAX_TOP"]

MATVEC_MAX_M = 16
KV8_MAX_T = 16
MAX_TOP = 32

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class _CacheStruct(ctypes.Structure):
    """The C struct bsg_kv8_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("dim", ctypes.c_int)]


class _TokensStruct(ctypes.Structure):
    """The C struct bsg_tokens."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


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


def _activation(t, dim: int, name: str) -> int:
    """The C dtype of an activation tensor, checked."""
    code = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None or not t.is_cuda:
        raise TypeError(f"{name} must be a float32, float16 or bfloat16 CUDA tensor")
    if t.dim() != dim or t.numel() == 0 or (t.stride(-1) != 1 and t.shape[-1] != 1):
        raise ValueError(f"{name} must be a non-empty {dim}-D tensor with a contiguous last dimension")
    return code


def _exact(t, dtype, shape, name: str, device) -> int:
    """The address of a contiguous tensor of this dtype and shape, on `device`."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device:
        raise TypeError(f"{name} must be a tensor of dtype {dtype} on {device}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _rows(t) -> int:
    """The leading dimension of a 2-D tensor (its row stride; one row has any)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _made(shape, dtype, device, stream):
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def _output(out, shape, dtype, device, stream):
    """`out`, checked, or a new tensor."""
    if out is None:
        return _made(shape, dtype, device, stream)
    if not isinstance(out, torch.Tensor) or out.dtype != dtype or out.device != device:
        raise TypeError(f"out must be a tensor of dtype {dtype} on {device}")
    if out.shape != shape or (out.stride(-1) != 1 and out.shape[-1] != 1):
        raise ValueError(f"out must have shape {tuple(shape)} and a contiguous last dimension")
    return out


def _stream(stream, device) -> int:
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


def _status(dstatus, device):
    return None if dstatus is None else _exact(dstatus, torch.int32, (1,), "dstatus", device)


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
    _bsg._check(_bsg.load().bsg_wquant_groups(
        W.data_ptr(), K, N, _rows(W), group, Q.data_ptr(), Q.shape[1], scale.data_ptr(), N,
        _status(dstatus, W.device), _stream(stream, W.device)), "bsg_wquant_groups")
    return Q[:, :half], scale


def wgroups_matvec(X, Q, scale, group: int = 64, relu: bool = False, out=None, dstatus=None,
                   stream=None, workspace=None):
    """Y = X . W_hat (+ReLU) for up to MATVEC_MAX_M rows of X (M x K) and a
    weight stored by wquant_groups -- or by wquant_cols with bits=4, with
    group=0 and scale viewed as (1, N).  Y: M x N of X's dtype."""
    code = _activation(X, 2, "X")
    dev = X.device
    M, K = X.shape
    if M > MATVEC_MAX_M:
        raise ValueError(f"at most {MATVEC_MAX_M} rows: X has {M} (use bsgemm_i8 for more)")
    if group < 0 or group % 32:
        raise ValueError("group must be a multiple of 32, or 0")
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32 or scale.device != dev:
        raise TypeError(f"scale must be a float32 tensor on {dev}")
    if scale.dim() != 2 or scale.stride(1) != 1 and scale.shape[1] != 1 \
            or scale.shape[0] != ((K + group - 1) // group if group else 1):
        raise ValueError("scale must be (groups, N), one row per group of rows of the weight")
    N = scale.shape[1]
    if not isinstance(Q, torch.Tensor) or Q.dtype != torch.uint8 or Q.device != dev:
        raise TypeError(f"Q must be a uint8 tensor on {dev}")
    if Q.shape != (K, (N + 1) // 2) or Q.stride(1) != 1 and Q.shape[1] != 1:
        raise ValueError("Q must be (K, ceil(N/2)) with contiguous rows")
    Y = _output(out, (M, N), X.dtype, dev, stream)
    lib = _bsg.load()
    wp, wn = _bsg._ws(workspace, lib.bsg_wgroups_matvec_workspace_size(M, N, K))
    _bsg._check(lib.bsg_wgroups_matvec(
        X.data_ptr(), code, _rows(X), Q.data_ptr(), _rows(Q), scale.data_ptr(), _rows(scale),
        group, M, N, K, bool(relu), Y.data_ptr(), _rows(Y), wp, wn, _status(dstatus, dev),
        _stream(stream, dev)), "bsg_wgroups_matvec")
    return Y


# ---------------------------------------------------------------------------
def _cache_struct(cache, device):
    k, v, ks, vs = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("the cache's k must be (pages, heads, page_tokens, dim)")
    pages, heads, page_tokens, dim = shape = k.shape
    return _CacheStruct(_exact(k, torch.int8, shape, "k", device),
                        _exact(v, torch.int8, shape, "v", device),
                        _exact(ks, torch.float32, shape[:2], "k_scale", device),
                        _exact(vs, torch.float32, shape[:2], "v_scale", device),
                        pages, heads, page_tokens, dim)


def _tokens_struct(t):
    s = t.stride()
    return _TokensStruct(t.data_ptr(), s[0], s[1], s[2])


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
    c = _cache_struct(cache, dev)
    if (H, D) != (c.heads, c.dim):
        raise ValueError(f"the cache has {c.heads} heads of {c.dim}")
    _bsg._check(_bsg.load().bsg_kv8_append(
        ctypes.byref(c), _table(table, B, dev), table.shape[1],
        _exact(starts, torch.int32, (B,), "starts", dev),
        None if counts is None else _exact(counts, torch.int32, (B,), "counts", dev),
        ctypes.byref(_tokens_struct(k)), ctypes.byref(_tokens_struct(v)), code, B, T,
        _status(dstatus, dev), _stream(stream, dev)), "bsg_kv8_append")


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
    c = _cache_struct(cache, dev)
    if D != c.dim or H % c.heads:
        raise ValueError(f"the cache has {c.heads} heads of {c.dim}")
    if T > KV8_MAX_T:
        raise ValueError(f"at most {KV8_MAX_T} tokens a sequence: q has {T}")
    O = _output(out, q.shape, q.dtype, dev, stream)
    lib = _bsg.load()
    tp, width = _table(table, B, dev), table.shape[1]
    need = lib.bsg_kv8_attend_workspace_size(ctypes.byref(c), width, B, T, H)
    wp, wn = _bsg._ws(workspace, need)
    _bsg._check(lib.bsg_kv8_attend(
        ctypes.byref(c), tp, width, _exact(lens, torch.int32, (B,), "lens", dev),
        ctypes.byref(_tokens_struct(q)), ctypes.byref(_tokens_struct(O)), code, B, T, H,
        D ** -0.5 if scale is None else scale,
        None if lse is None else _exact(lse, torch.float32, (B, T, H), "lse", dev), wp, wn,
        _status(dstatus, dev), _stream(stream, dev)), "bsg_kv8_attend")
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
    lp, ent, lse = (_made((M,), torch.float32, dev, stream) for _ in range(3))
    tl = _made((M, top), torch.float32, dev, stream)
    ti = _made((M, top), torch.int32, dev, stream)
    _bsg._check(_bsg.load().bsg_logprobs(
        logits.data_ptr(), code, M, V, _rows(logits), tp, top, lp.data_ptr(), ent.data_ptr(),
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
    D = _output(out, (M, V), logits.dtype, dev, stream)
    _bsg._check(_bsg.load().bsg_logprobs_backward(
        logits.data_ptr(), code, M, V, _rows(logits), tp, *per_row, D.data_ptr(), _rows(D),
        _status(dstatus, dev), _stream(stream, dev)), "bsg_logprobs_backward")
    return D

"""The target's side of a step: what of its forward depends on the step itself.

Between a schedule and a verification the target runs over the scheduled tokens.  Their keys and
values go into a paged cache (``cache_append``, which also normalises and rotates queries and
keys), the tokens, a chain or a tree, attend to it (``tree_attention``), ``tree_verify`` verifies
them against the target's probabilities from given uniform numbers, and ``cache_keep`` moves the
accepted ones' keys and values together.

Rows of tokens are padded, [B, N, ...] with ``counts`` [B] int32 (None: all N), as the step's own
calls have them, or packed, [rows, ...] with ``starts`` [B + 1] int32 (request b's are rows
starts[b] .. starts[b + 1] - 1) and ``nodes``, the most tokens of a request.  ``parents`` [B, N]
or [rows] int32 names each token's parent by its place in the request (-1 for the first); None: a
chain.  A tree has at most 64 tokens.  ``pages`` [B, max_pages] and ``lengths`` [B] int32 say where
a request's tokens are cached and how many were before the step.  ``stream`` is the stream the
kernels run on (default: the current one); outputs that a call allocates belong to it, and the
caller orders it after what produced the inputs.  A call raises ValueError for tensors of the
wrong type, shape, layout or device, and DSparkError for what the library refuses; nothing is
launched in either case.  What only the device sees (counts, lengths, pages, parents out of range)
is reported by ``ws.status()``.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import warnings
from typing import Dict, Optional

from . import DSparkError, Workspace, _build, lib
from .rows import _NOTHING, _device, _done, _on, _rows, _types, _vector


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("layers", ctypes.c_int),
                ("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("layer_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class PagedCache:
    """Keys and values in pages: ``k`` and ``v`` [pages, page_size, heads, head_dim], or with a
    leading dimension of layers, bf16 or fp16, of equal strides (any whose last is 1 and whose
    others are multiples of 8).  The handle holds on to both tensors and writes into them."""

    def __init__(self, k, v):
        torch, codes = _types()
        if k.dtype is not torch.bfloat16 and k.dtype is not torch.float16:
            raise ValueError(f"k: dtype {k.dtype} is not bfloat16 or float16")
        if k.dim() not in (4, 5) or not k.is_cuda or k.numel() == 0:
            raise ValueError(f"k: a CUDA tensor [(layers,) pages, page_size, heads, head_dim] is needed, not "
                             f"{tuple(k.shape)} on {k.device}")
        if v.dtype is not k.dtype or v.shape != k.shape or v.stride() != k.stride() or v.device != k.device:
            raise ValueError("k and v have one type, shape, device and strides")
        shape, stride = tuple(k.shape), k.stride()
        if stride[-1] != 1:
            raise ValueError(f"k: its last dimension is not contiguous (strides {tuple(stride)})")
        if len(shape) == 4:
            shape, stride = (1,) + shape, (0,) + tuple(stride)
        # (a dimension of one has no stride of its own)
        stride = [0 if size == 1 else step for size, step in zip(shape, stride)]
        self.k, self.v = k, v
        self.layers, self.n_pages, self.page_size, self.heads, self.head_dim = shape
        self.dtype, self.device, self.index = k.dtype, k.device, k.get_device()
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), codes[k.dtype], *shape, *stride[:4])
        self._ptr = ctypes.addressof(self._struct)
        self._key = (self._ptr, self.dtype, self.index, self.heads, self.head_dim)


class _Unchecked:
    """In the place of the module: every call is left to the checks below."""
    append = attend = verify = keep = staticmethod(lambda *args: None)


def _module():
    """The module of calls.cpp; None where it was not built for this interpreter."""
    if not os.path.exists(_build.CALLS):
        return None
    loader = importlib.machinery.ExtensionFileLoader("_dspark_calls", _build.CALLS)
    try:
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_dspark_calls", loader))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"{_build.CALLS} cannot be loaded, calls are checked in Python: {e}", RuntimeWarning)
        return None
    return module


@functools.lru_cache(maxsize=None)
def _calls():
    """What checks and makes a well-formed call in C (calls.cpp): for a single token the checks
    below take longer than the kernel.  Its functions return a status, or None where a check failed
    or an output is to be made: then the checks below are made, which say what is wrong."""
    torch, _ = _types()
    L = lib()
    module = _module()
    if module is None:
        return _Unchecked
    module.setup(*(ctypes.cast(getattr(L, "dspark_" + name), ctypes.c_void_p).value
                   for name in ("cache_append", "tree_attention", "tree_verify", "cache_keep")),
                 torch.float32, torch.bfloat16, torch.float16, torch.int32, torch._C._cuda_getDevice,
                 torch._C._cuda_getCurrentRawStream)
    return module


def _begin(like, ws, stream):
    """(device index, stream handle, context in which outputs are allocated for it)."""
    torch, _ = _types()
    dev = like.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or ws.buf.get_device() != dev:
        _device(like, ws)
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev), _NOTHING
    return (dev, *_on(stream, like))


def _flat(t, name, n, dtype, like, dev, k=1):
    """Pointer of a contiguous input or output of n x k entries; None stays None."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n * k and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _vector(t, name, n, dtype, like, None if k == 1 else k)


def _tokens(lead, starts, counts, nodes, like, dev, i32):
    """(B, N, rows, starts, counts) of rows with the leading dimensions ``lead``."""
    if starts is None:
        if len(lead) != 2:
            raise ValueError(f"rows [B, N, ...] are needed where starts is not given, not {tuple(lead)}")
        B, N = lead
        return B, N, B * N, None, _flat(counts, "counts", B, i32, like, dev)
    if len(lead) != 1 or counts is not None or nodes is None:
        raise ValueError("packed rows have one leading dimension, starts and nodes, and no counts")
    B = starts.numel() - 1
    if B < 0:
        raise ValueError("starts: [B + 1] entries are needed")
    return B, nodes, lead[0], _flat(starts, "starts", B + 1, i32, like, dev), None


def _slots(pages, lengths, B, like, dev, i32):
    if pages.dim() != 2:
        raise ValueError(f"pages: a table [B, max_pages] is needed, not {tuple(pages.shape)}")
    most = pages.shape[1]
    return _flat(pages, "pages", B, i32, like, dev, most), most, _flat(lengths, "lengths", B, i32, like, dev)


def _heads(t, name, lead, dim, cache):
    """(pointer, row stride, head stride, heads) of rows of heads."""
    if t.dtype is not cache.dtype or t.get_device() != cache.index:
        raise ValueError(f"{name}: {cache.dtype} on {cache.device} is needed, not {t.dtype} on {t.device}")
    shape, stride = t.shape, t.stride()
    if len(shape) != len(lead) + 2 or shape[:-2] != lead or shape[-1] != dim:
        raise ValueError(f"{name}: {tuple(lead)} rows of heads of {dim} are needed, not {tuple(shape)}")
    if stride[-1] != 1:
        raise ValueError(f"{name}: its last dimension is not contiguous (strides {tuple(stride)})")
    heads, n, row = shape[-2], lead[0], stride[0]
    if len(lead) == 2:
        N = lead[1]
        if N != 1:
            row = stride[1]
            if n > 1 and stride[0] != N * row:
                raise ValueError(f"{name}: its leading dimensions do not flatten into rows of one stride "
                                 f"(shape {tuple(shape)}, strides {tuple(stride)})")
        n *= N
    return t.data_ptr(), row if n > 1 else 0, stride[-2] if heads > 1 else 0, heads


def cache_append(cache: PagedCache, k, v, pages, lengths, ws: Workspace, q=None, q_out=None, starts=None,
                 counts=None, nodes: Optional[int] = None, parents=None, inv_freq=None, interleaved: bool = False,
                 q_weight=None, k_weight=None, eps: float = 1e-6, layer: int = 0, stream=None):
    """Appends ``k`` and ``v`` [..., heads, head_dim] of the step's tokens to the cache, and
    returns ``q`` [..., q_heads, head_dim] normalised and rotated like the keys (in ``q_out``,
    which may be ``q``; None without ``q``).

    Token i of request b has slot lengths[b] + i.  ``q_weight`` and ``k_weight`` [head_dim] fp32:
    each head is divided by its root mean square (``eps`` added to the mean) and multiplied by the
    weight.  ``inv_freq`` [R / 2] fp32: the first R elements of each head are rotated by position
    times frequency, in pairs (j, j + R / 2), or (2 j, 2 j + 1) with ``interleaved``; the position is
    lengths[b] plus the token's depth in its tree.  A chain may be of any length (a prompt)."""
    if stream is None:
        code = _calls().append(cache, k, v, pages, lengths, ws, q, q_out, starts, counts, nodes, parents, inv_freq,
                               interleaved, q_weight, k_weight, eps, layer)
        if code is not None:
            _done("dspark_cache_append", code)
            return q_out
    torch, _ = _types()
    i32, f32 = torch.int32, torch.float32
    dev, handle, allocate = _begin(k, ws, stream)
    D = cache.head_dim
    lead = k.shape[:-2]
    B, N, rows, s, c = _tokens(lead, starts, counts, nodes, k, dev, i32)
    k_p, k_row, k_head, heads = _heads(k, "k", lead, D, cache)
    v_p, v_row, v_head, v_heads = _heads(v, "v", lead, D, cache)
    if heads != cache.heads or v_heads != heads:
        raise ValueError(f"k and v: {cache.heads} heads are needed, not {heads} and {v_heads}")
    q_p = q_row = q_head = q_heads = o_p = o_row = o_head = 0
    if q is not None:
        q_p, q_row, q_head, q_heads = _heads(q, "q", lead, D, cache)
        if q_out is None:
            with allocate:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        o_p, o_row, o_head, o_heads = _heads(q_out, "q_out", lead, D, cache)
        if o_heads != q_heads:
            raise ValueError(f"q_out: {q_heads} heads are needed, not {o_heads}")
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    rotated = 0 if inv_freq is None else 2 * inv_freq.numel()
    table, most, used = _slots(pages, lengths, B, k, dev, i32)
    _done("dspark_cache_append", lib().dspark_cache_append(
        cache._ptr, layer, s, c, _flat(parents, "parents", rows, i32, k, dev), B, N, rows, table, most, used,
        k_p, k_row, k_head, v_p, v_row, v_head, q_p or None, q_row, q_head, q_heads, o_p or None, o_row, o_head,
        _flat(inv_freq, "inv_freq", rotated // 2, f32, k, dev), rotated, interleaved,
        _flat(q_weight, "q_weight", D, f32, k, dev), _flat(k_weight, "k_weight", D, f32, k, dev), eps,
        ws.ptr, ws.nbytes, handle))
    return q_out


def tree_attention_workspace_bytes(B: int, nodes: int, q_heads: int, heads: int, head_dim: int) -> int:
    """Bytes of the workspace that ``tree_attention`` needs for B requests of up to ``nodes`` tokens."""
    nbytes = lib().dspark_tree_attention_workspace_bytes(B, nodes, q_heads, heads, head_dim)
    if nbytes == 0:
        raise ValueError(f"unsupported shapes B={B} nodes={nodes} q_heads={q_heads} heads={heads} head_dim={head_dim}")
    return int(nbytes)


def tree_attention(q, cache: PagedCache, pages, lengths, ws: Workspace, starts=None, counts=None,
                   nodes: Optional[int] = None, parents=None, scale: Optional[float] = None, out=None, lse=None,
                   layer: int = 0, stream=None):
    """Attention of the step's tokens ``q`` [..., q_heads, head_dim] over the cache, to which their
    keys and values have been appended: each sees the slots before the step, its ancestors and
    itself.  ``scale`` (default head_dim ** -0.5) multiplies the scores.  Returns ``out`` like
    ``q``; ``lse`` [..., q_heads] fp32, if given, gets the logarithms of the softmax's sums.
    head_dim is 64 or 128, and a request has at most 64 tokens."""
    if stream is None:
        code = _calls().attend(q, cache, pages, lengths, ws, starts, counts, nodes, parents,
                               cache.head_dim ** -0.5 if scale is None else scale, out, lse, layer)
        if code is not None:
            _done("dspark_tree_attention", code)
            return out
    torch, _ = _types()
    i32 = torch.int32
    dev, handle, allocate = _begin(q, ws, stream)
    lead, D = q.shape[:-2], cache.head_dim
    B, N, rows, s, c = _tokens(lead, starts, counts, nodes, q, dev, i32)
    q_p, q_row, q_head, q_heads = _heads(q, "q", lead, D, cache)
    if out is None:
        with allocate:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    o_p, o_row, o_head, o_heads = _heads(out, "out", lead, D, cache)
    if o_heads != q_heads:
        raise ValueError(f"out: {q_heads} heads are needed, not {o_heads}")
    table, most, used = _slots(pages, lengths, B, q, dev, i32)
    _done("dspark_tree_attention", lib().dspark_tree_attention(
        cache._ptr, layer, s, c, _flat(parents, "parents", rows, i32, q, dev), B, N, rows, table, most, used,
        q_p, q_row, q_head, q_heads, D ** -0.5 if scale is None else scale, o_p, o_row, o_head,
        _flat(lse, "lse", rows, torch.float32, q, dev, q_heads), ws.ptr, ws.nbytes, handle))
    return out


def tree_verify(p, tokens, uniforms, ws: Workspace, q=None, starts=None, counts=None, nodes: Optional[int] = None,
                parents=None, out: Optional[Dict] = None, stream=None) -> Dict:
    """Verification of the step's tokens against the target's probabilities ``p`` [..., V] (fp32, bf16
    or fp16; p's row of a token is the distribution after it).

    ``tokens`` [...] int32 (a request's first is its last committed token), ``uniforms`` [...] fp32 in
    [0, 1): the first token's is the last draw's, the others' decide their token.  ``q`` [..., V]: the
    distribution from which a token's children were drawn, each independently; None: children
    that the draft names without chance (greedy drafts, its most probable tokens).  Returns a dict
    of int32 tensors: ``accept_len`` [B], ``path`` [B, N] the accepted tokens' places, ``out_tokens``
    [B, N] their ids and the last token, ``n_out`` [B]; -1 behind them.  It is ``out`` if that is
    given: entries that it holds are written, those that it lacks are made."""
    if stream is None and out is not None:
        code = _calls().verify(p, tokens, uniforms, ws, q, starts, counts, nodes, parents, out.get("accept_len"),
                               out.get("path"), out.get("out_tokens"), out.get("n_out"))
        if code is not None:
            _done("dspark_tree_verify", code)
            return out
    torch, _ = _types()
    i32 = torch.int32
    code, n, V, ld = _rows(p, "p")
    dev, handle, allocate = _begin(p, ws, stream)
    B, N, rows, s, c = _tokens(p.shape[:-1], starts, counts, nodes, p, dev, i32)
    ld_q, q_p = ld, None
    if q is not None:
        code_q, n_q, V_q, ld_q = _rows(q, "q")
        if (code_q, n_q, V_q) != (code, n, V) or q.get_device() != dev:
            raise ValueError(f"q: {n} x {V} {p.dtype} on {p.device} are needed, not {tuple(q.shape)} {q.dtype}")
        q_p = q.data_ptr()
    if out is None:
        out = {}
    for key, shape in (("accept_len", (B,)), ("path", (B, N)), ("out_tokens", (B, N)), ("n_out", (B,))):
        if out.get(key) is None:
            with allocate:
                out[key] = torch.empty(shape, dtype=i32, device=p.device)
    _done("dspark_tree_verify", lib().dspark_tree_verify(
        p.data_ptr(), ld, q_p, ld_q, code, V, _flat(tokens, "tokens", rows, i32, p, dev),
        _flat(uniforms, "uniforms", rows, torch.float32, p, dev), s, c, _flat(parents, "parents", rows, i32, p, dev),
        B, N, rows, _flat(out["accept_len"], "accept_len", B, i32, p, dev), _flat(out["path"], "path", B, i32, p, dev, N),
        _flat(out["out_tokens"], "out_tokens", B, i32, p, dev, N), _flat(out["n_out"], "n_out", B, i32, p, dev),
        ws.ptr, ws.nbytes, handle))
    return out


def cache_keep(cache: PagedCache, pages, lengths, path, accept_len, ws: Workspace, stream=None) -> None:
    """Moves the accepted tokens' keys and values together in every layer: token path[b, j] of
    request b to slot lengths[b] + 1 + j, for j < accept_len[b] (``path`` [B, N], ``accept_len`` [B] as
    ``tree_verify`` returns them).  After it lengths[b] + 1 + accept_len[b] slots are used; the
    caller updates ``lengths``."""
    if stream is None:
        code = _calls().keep(cache, pages, lengths, path, accept_len, ws)
        if code is not None:
            return _done("dspark_cache_keep", code)
    torch, _ = _types()
    if path.dim() != 2:
        raise ValueError(f"path: [B, N] is needed, not {tuple(path.shape)}")
    i32, k = torch.int32, cache.k
    dev, handle, _ = _begin(k, ws, stream)
    B, N = path.shape
    table, most, used = _slots(pages, lengths, B, k, dev, i32)
    _done("dspark_cache_keep", lib().dspark_cache_keep(
        cache._ptr, B, N, table, most, used, _flat(path, "path", B, i32, k, dev, N),
        _flat(accept_len, "accept_len", B, i32, k, dev), ws.ptr, ws.nbytes, handle))

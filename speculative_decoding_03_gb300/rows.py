"""Calls on rows of logits and of tables (fp32, bf16 or fp16): what trains the draft head
and reports on the tokens a step answers with.

The target's rows give a teacher's top logits (``token_logprobs``), the student's logits the
loss and its gradient (``distill_loss_grad``), and the gradient of looked-up rows of W1 is
summed into the table's (``embed``, ``embed_grad``).  Matrices may have leading dimensions
that flatten into rows of one stride; their last dimension is contiguous.  ``stream`` is the
stream the kernels run on (default: the current one); outputs that a call allocates belong to
it, and the caller orders it after what produced the inputs.  A call raises ValueError for
tensors of the wrong type, shape, layout or device, and DSparkError for what the library
refuses; nothing is launched in either case.
"""
from __future__ import annotations

import contextlib
import functools
import math
from typing import Dict, Optional

from . import DSparkError, Workspace, lib


@functools.lru_cache(maxsize=None)
def _types():
    import torch
    if not torch.cuda.is_available():
        raise RuntimeError("the DSpark kernels need a CUDA device; there is no CPU fallback")
    return torch, {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _rows(t, name: str):
    """(dtype code, rows, length, leading dimension) of a matrix, its leading dimensions
    flattened."""
    torch, codes = _types()
    code = codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype} is not float32, bfloat16 or float16")
    if t.dim() < 1 or not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor of at least one dimension is needed")
    shape = t.shape
    length = shape[-1]
    if t.is_contiguous():
        return code, t.numel() // length if length else math.prod(shape[:-1]), length, length
    stride = t.stride()
    if length > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: its last dimension is not contiguous (strides {tuple(stride)})")
    n, ld = 1, length
    for size, step in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if size == 1:
            continue
        if n == 1:
            ld = step
        elif step != n * ld:
            raise ValueError(f"{name}: its leading dimensions do not flatten into rows of one stride "
                             f"(shape {tuple(shape)}, strides {tuple(stride)})")
        n *= size
    return code, n, length, ld


def _vector(t, name: str, n: int, dtype, like, k: Optional[int] = None):
    """Pointer of a contiguous input or output of n (or n x k) entries; None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != (n if k is None else n * k) or not t.is_contiguous() \
            or t.get_device() != like.get_device():
        want = f"{n}" if k is None else f"{n} x {k}"
        raise ValueError(f"{name}: {want} contiguous {dtype} on {like.device} are needed, not "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return t.data_ptr()


def _device(like, ws: Workspace):
    torch, _ = _types()
    if like.device.index != torch.cuda.current_device() or ws.buf.device != like.device:
        raise ValueError(f"tensors on {like.device}, workspace on {ws.buf.device}: both must be on "
                         f"the current device (cuda:{torch.cuda.current_device()})")


_NOTHING = contextlib.nullcontext()


def _on(stream, like):
    """(stream handle, context in which outputs are allocated for it)."""
    torch, _ = _types()
    if stream is None:
        # (the handle alone: a Stream object takes 3 us to make)
        return torch._C._cuda_getCurrentRawStream(like.device.index), _NOTHING
    return stream.cuda_stream, torch.cuda.stream(stream)


def _done(call: str, code: int):
    if code != 0:
        raise DSparkError(call, code)


def token_logprobs(logits, tokens, top: int, ws: Workspace, out: Optional[Dict] = None,
                   stream=None) -> Dict:
    """Log probabilities of given tokens with entropy, rank and the ``top`` alternatives.

    ``logits`` [..., V] and ``tokens`` [...] int32, e.g. a step's target rows and its
    ``out_tokens``: a row whose token is -1 is not read.  ``tokens`` None uses every row
    (then no ``logprob`` and no ``rank``).  Returns (or fills ``out``) a dict of tensors of
    the rows' shape: ``logprob``, ``entropy``, ``rank`` (1 for the largest logit),
    ``row_max``, ``row_sumexp``, and with ``top`` > 0 ``top_ids`` and ``top_logprobs``
    [..., top], largest first.  ``out`` says what is written: it holds ``logprob`` and ``rank``
    just where tokens are given, ``top_ids`` and ``top_logprobs`` where ``top`` > 0 (with 0 they
    stay as they are), and may lack the others."""
    torch, _ = _types()
    code, n, V, ld = _rows(logits, "logits")
    _device(logits, ws)
    handle, allocate = _on(stream, logits)
    tok = _vector(tokens, "tokens", n, torch.int32, logits)
    f32, i32 = torch.float32, torch.int32
    if out is None:
        lead, d = tuple(logits.shape[:-1]), logits.device
        with allocate:
            out = {k: torch.empty(lead, dtype=f32, device=d) for k in ("entropy", "row_max", "row_sumexp")}
            if tokens is not None:
                out["logprob"] = torch.empty(lead, dtype=f32, device=d)
                out["rank"] = torch.empty(lead, dtype=i32, device=d)
            if top > 0:
                out["top_ids"] = torch.empty(lead + (top,), dtype=i32, device=d)
                out["top_logprobs"] = torch.empty(lead + (top,), dtype=f32, device=d)
    v = lambda key, dtype, k=None: _vector(out.get(key), key, n, dtype, logits, k)  # noqa: E731
    _done("dspark_token_logprobs", lib().dspark_token_logprobs(
        logits.data_ptr(), code, ld, tok, n, V, top, v("logprob", f32), v("entropy", f32),
        v("rank", i32), v("row_max", f32), v("row_sumexp", f32),
        v("top_ids", i32, top) if top > 0 else None, v("top_logprobs", f32, top) if top > 0 else None,
        ws.ptr, ws.nbytes, handle))
    return out


def token_logprobs_grad(logits, tokens, row_max, row_sumexp, entropy, d_logprob, d_entropy,
                        ws: Workspace, out=None, stream=None):
    """Gradient of ``token_logprobs``'s log probabilities and entropies with respect to the
    logits, for the upstream gradients ``d_logprob`` and ``d_entropy`` (either may be None).
    ``row_max``, ``row_sumexp`` and ``entropy`` are that call's.  ``out``: a tensor of the
    logits' type and shape, or the logits themselves."""
    torch, _ = _types()
    code, n, V, ld = _rows(logits, "logits")
    _device(logits, ws)
    handle, allocate = _on(stream, logits)
    out, ld_d = _like_logits(out, logits, code, n, V, allocate)
    f32 = torch.float32
    v = lambda t, name, dtype=f32: _vector(t, name, n, dtype, logits)  # noqa: E731
    _done("dspark_token_logprobs_grad", lib().dspark_token_logprobs_grad(
        logits.data_ptr(), code, ld, v(tokens, "tokens", torch.int32), n, V, v(row_max, "row_max"),
        v(row_sumexp, "row_sumexp"), v(entropy, "entropy"), v(d_logprob, "d_logprob"),
        v(d_entropy, "d_entropy"), out.data_ptr(), ld_d, ws.ptr, ws.nbytes, handle))
    return out


def _like_logits(out, logits, code, n, V, allocate):
    torch, _ = _types()
    if out is None:
        with allocate:
            out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    code_d, n_d, V_d, ld_d = _rows(out, "the logits' gradient")
    if (code_d, n_d, V_d) != (code, n, V) or out.device != logits.device:
        raise ValueError(f"the logits' gradient: {n} x {V} {logits.dtype} on {logits.device} are needed, "
                         f"not {tuple(out.shape)} {out.dtype} on {out.device}")
    return out, ld_d


def _distill(grad: bool, logits, teacher_ids, teacher_logits, ws, labels, weights, d_loss, temperature,
             kl, tv, ce, out, stream):
    torch, _ = _types()
    code, n, V, ld = _rows(logits, "logits")
    _device(logits, ws)
    handle, allocate = _on(stream, logits)
    f32, i32 = torch.float32, torch.int32
    K = 0 if teacher_ids is None else teacher_ids.shape[-1]
    lead, d = tuple(logits.shape[:-1]), logits.device
    if out is None:
        out = {}
    for key in ("loss", "accept"):
        if out.get(key) is None:
            with allocate:
                out[key] = torch.empty(lead, dtype=f32, device=d)
    v = lambda t, name, dtype=f32, k=None: _vector(t, name, n, dtype, logits, k)  # noqa: E731
    args = [logits.data_ptr(), code, ld, v(teacher_ids, "teacher_ids", i32, K),
            v(teacher_logits, "teacher_logits", f32, K), v(labels, "labels", i32), v(weights, "weights")]
    shape = [n, V, K, temperature, kl, tv, ce, v(out["loss"], "loss"), v(out["accept"], "accept")]
    if not grad:
        _done("dspark_distill_loss", lib().dspark_distill_loss(*args, *shape, ws.ptr, ws.nbytes, handle))
        return out
    out["d_logits"], ld_d = _like_logits(out.get("d_logits"), logits, code, n, V, allocate)
    _done("dspark_distill_loss_grad", lib().dspark_distill_loss_grad(
        *args, v(d_loss, "d_loss"), *shape, out["d_logits"].data_ptr(), ld_d, ws.ptr, ws.nbytes, handle))
    return out


def distill_loss(logits, teacher_ids, teacher_logits, ws: Workspace, labels=None, weights=None,
                 temperature: float = 1.0, kl: float = 1.0, tv: float = 0.0, ce: float = 0.0,
                 out: Optional[Dict] = None, stream=None) -> Dict:
    """Distillation loss of the student's ``logits`` [..., V] from a teacher's top logits.

    ``teacher_ids`` [..., K] int32 (-1: no entry) and ``teacher_logits`` [..., K] fp32 (logits
    or log probabilities, as ``token_logprobs`` returns them), ``labels`` [...] int32 (-1:
    none), ``weights`` [...] fp32 (0: the row is not read).  Per row, with p and q the
    teacher's and the student's softmax at ``temperature``: ``loss`` = weight (kl KL(p || q) +
    tv TV(p, q) - ce log q[label]) and ``accept`` = sum min(p, q), the probability that a
    token drafted from q is accepted by a target cut to the entries (p sums to 1 over them).  By
    the whole target it differs from that by at most the probability that the entries leave out:
    1 - exp(teacher_logits).sum(-1) for ``token_logprobs``'s at temperature 1.  Returns a dict of both, ``out`` if it is given: entries
    that it holds are written, those that it lacks are made."""
    return _distill(False, logits, teacher_ids, teacher_logits, ws, labels, weights, None, temperature, kl,
                    tv, ce, out, stream)


def distill_loss_grad(logits, teacher_ids, teacher_logits, ws: Workspace, labels=None, weights=None,
                      d_loss=None, temperature: float = 1.0, kl: float = 1.0, tv: float = 0.0,
                      ce: float = 0.0, out: Optional[Dict] = None, stream=None) -> Dict:
    """``distill_loss`` and, from the same read of the logits, ``d_logits``: the gradient of
    sum(d_loss * loss) (``d_loss`` [...] fp32, None: all 1).  ``out={"d_logits": logits}`` writes
    it over the logits."""
    return _distill(True, logits, teacher_ids, teacher_logits, ws, labels, weights, d_loss, temperature, kl,
                    tv, ce, out, stream)


def embed(W, ids, ws: Workspace, scale: float = 1.0, out=None, dtype=None, stream=None):
    """``scale`` times the rows ``ids`` [...] int32 (-1: a zero row) of the table ``W`` [V, D],
    as [..., D] of ``dtype`` (W's, or float32)."""
    torch, _ = _types()
    if W.dim() != 2:
        raise ValueError(f"W: a table [V, D] is needed, not {tuple(W.shape)}")
    code, V, D, ld = _rows(W, "W")
    _device(W, ws)
    handle, allocate = _on(stream, W)
    n = ids.numel()
    if out is None:
        with allocate:
            out = torch.empty(tuple(ids.shape) + (D,), dtype=dtype or W.dtype, device=W.device)
    code_o, n_o, D_o, ld_o = _rows(out, "out")
    if (n_o, D_o) != (n, D) or out.device != W.device or (dtype is not None and out.dtype is not dtype):
        raise ValueError(f"out: {n} x {D} on {W.device} are needed, not {tuple(out.shape)} {out.dtype}")
    _done("dspark_embed", lib().dspark_embed(
        W.data_ptr(), code, ld, _vector(ids, "ids", n, torch.int32, W), n, V, D, scale, out.data_ptr(),
        code_o, ld_o, ws.ptr, ws.nbytes, handle))
    return out


def embed_grad_workspace_bytes(n: int, V: int, D: int) -> int:
    """Bytes of the workspace that ``embed_grad`` needs for n positions of a table [V, D]."""
    nbytes = lib().dspark_embed_grad_workspace_bytes(n, V, D)
    if nbytes == 0:
        raise ValueError(f"unsupported shapes n={n} V={V} D={D}")
    return int(nbytes)


def embed_grad(d_out, ids, V: int, ws: Workspace, scale: float = 1.0, out=None, accumulate: bool = False,
               dtype=None, stream=None):
    """Gradient of ``embed`` with respect to its table: [V, D] of ``dtype`` (d_out's, or
    float32) with row v the sum of ``scale * d_out[n]`` over the positions n of token v.  With
    ``accumulate`` it is added to ``out``.  Equal inputs give equal bits."""
    torch, _ = _types()
    code, n, D, ld = _rows(d_out, "d_out")
    _device(d_out, ws)
    handle, allocate = _on(stream, d_out)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out, the table to add to")
        with allocate:
            out = torch.empty((V, D), dtype=dtype or d_out.dtype, device=d_out.device)
    code_o, V_o, D_o, ld_o = _rows(out, "out")
    if out.dim() != 2 or (V_o, D_o) != (V, D) or out.device != d_out.device \
            or (dtype is not None and out.dtype is not dtype):
        raise ValueError(f"out: {V} x {D} on {d_out.device} are needed, not {tuple(out.shape)} {out.dtype}")
    _done("dspark_embed_grad", lib().dspark_embed_grad(
        d_out.data_ptr(), code, ld, _vector(ids, "ids", n, torch.int32, d_out), n, V, D, scale,
        int(accumulate), out.data_ptr(), code_o, ld_o, ws.ptr, ws.nbytes, handle))
    return out

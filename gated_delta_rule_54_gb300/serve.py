"""Serving operators: the 8-bit paged cache, the attention that reads it, and beam search.

Argument marshalling only (``include/gdn_qdq.h`` has the definitions).  A layer's cache is
``codes`` uint8 [2, pages, heads, page, dim] (0: K, 1: V) and ``scales`` f32 [2, pages, heads],
one scale per page of tokens and head; a pool over layers has a leading [layers].  Rows find
their pages in ``table`` int32 [rows, columns]; ``refs`` int32 [pages] counts the holders of a
page.  Everything runs on the current stream and nothing waits for the host.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from ._lib import (DTYPES, QDQ_MODES, GdnBeamProblem, GdnError, GdnKv8Pool, GdnKv8Problem, check,
                   load)
from .api import _ptr, _stream

_i32 = torch.int32
_byref = ctypes.byref


def _need(cond, text):
    if not cond:
        raise ValueError(text)


def _flat(name, t, dtype, device):
    _need(isinstance(t, torch.Tensor) and t.is_cuda and t.device == device,
          "%s must be a CUDA tensor on %s" % (name, device))
    _need(t.dtype == dtype, "%s must be %s" % (name, dtype))
    _need(t.is_contiguous(), "%s must be contiguous" % name)


def kv8_pool(layers, pages, heads, dim, page=64, device="cuda"):
    """An empty pool: (codes, scales) of zeros."""
    return (torch.zeros(layers, 2, pages, heads, page, dim, dtype=torch.uint8, device=device),
            torch.zeros(layers, 2, pages, heads, dtype=torch.float32, device=device))


def _strides(x):
    """(row, token, head) strides in elements of [rows, tokens, heads, dim] or [total, heads, dim]."""
    s, n = x.stride(), x.shape
    _need(s[-1] == 1 or n[-1] == 1, "the last dim must be contiguous")
    s = [a if b > 1 else 0 for a, b in zip(s, n)]
    return (s[0], s[1], s[2]) if x.dim() == 4 else (0, s[0], s[1])


def _problem(x, v, codes, scales, table, lengths, cu_seqlens, max_seqlen, mode, scale, causal,
             window) -> GdnKv8Problem:
    dev = codes.device
    _flat("codes", codes, torch.uint8, dev)
    _flat("scales", scales, torch.float32, dev)
    _flat("table", table, _i32, dev)
    _flat("lengths", lengths, _i32, dev)
    _need(codes.dim() == 5 and codes.shape[0] == 2, "codes must be [2, pages, heads, page, dim]")
    _, pages, heads, page, dim = codes.shape
    _need(scales.shape == codes.shape[:3], "scales must be [2, pages, heads]")
    _need(table.dim() == 2 and lengths.shape == (table.shape[0],),
          "table must be [rows, columns] and lengths [rows]")
    _need(x.is_cuda and x.device == dev, "q, k, v must be on %s" % dev)
    _need(mode in QDQ_MODES, "mode must be one of %s, got %r" % (sorted(QDQ_MODES), mode))
    p = GdnKv8Problem()
    p.pages, p.rows, p.cols = pages, table.shape[0], table.shape[1]
    p.heads, p.dim, p.page = heads, dim, page
    if cu_seqlens is None:
        _need(x.dim() == 4 and x.shape[0] == p.rows, "expected [rows, tokens, heads, dim]")
        p.total, p.tokens = x.shape[0] * x.shape[1], x.shape[1]
    else:
        _flat("cu_seqlens", cu_seqlens, _i32, dev)
        _need(x.dim() == 3, "expected packed [total, heads, dim]")
        _need(cu_seqlens.shape == (p.rows + 1,), "cu_seqlens must be [rows + 1]")
        p.total = x.shape[0]
        p.tokens = min(x.shape[0], x.shape[0] if max_seqlen is None else int(max_seqlen))
        p.cu_seqlens = cu_seqlens.data_ptr()
    _need(x.shape[-1] == dim, "head dim %d is not the cache's %d" % (x.shape[-1], dim))
    _need(heads > 0 and x.shape[-2] % heads == 0 and x.shape[-2] > 0,
          "%d heads cannot share %d K/V heads" % (x.shape[-2], heads))
    p.group = x.shape[-2] // heads
    p.mode = QDQ_MODES[mode]
    p.dtype = DTYPES.get({torch.bfloat16: "bf16", torch.float16: "fp16",
                          torch.float32: "fp32"}.get(x.dtype), 99)
    p.causal, p.window, p.scale = int(bool(causal)), int(window), scale
    p.x_row, p.x_token, p.x_head = _strides(x)
    if v is not None:
        _need(v.is_cuda and v.device == dev and v.dtype == x.dtype and v.shape == x.shape,
              "k and v must have the same shape, type and device")
        _need(p.group == 1, "k and v must have the cache's heads")
        p.v_row, p.v_token, p.v_head = _strides(v)
    return p


def kv8_append(k, v, codes, scales, table, start, cu_seqlens=None, max_seqlen=None, mode="e4m3"):
    """New tokens go to the cache, in place: row r's at positions start[r] onwards.

    k, v bf16 [rows, tokens, heads, dim], or packed [total, heads, dim] with ``cu_seqlens``
    int32 [rows + 1] (``max_seqlen``: an upper bound of a row's tokens); any strides that are
    multiples of 8, last dim contiguous.  codes, scales: one layer's cache.  A page's scale is
    max |x| / 448 (E4M3) or / 127 (INT8) over its tokens so far; where a new token raises it,
    the page's older codes are rounded again."""
    p = _problem(k, v, codes, scales, table, start, cu_seqlens, max_seqlen, mode, 1.0, True, 0)
    check("gdn_kv8_append", load().gdn_kv8_append(
        _byref(p), k.data_ptr(), v.data_ptr(), codes.data_ptr(), scales.data_ptr(),
        table.data_ptr(), start.data_ptr(), _stream(codes.device)))


def kv8_attention(q, codes, scales, table, lengths, cu_seqlens=None, max_seqlen=None, mode="e4m3",
                  scale: Optional[float] = None, causal=True, window=0, need_lse=False,
                  workspace=None, out=None):
    """Attention of q over the cache: softmax(scale q K^T) V, query head h reading K/V head
    h // (query heads / heads).

    q bf16 [rows, tokens, query heads, dim], or packed [total, query heads, dim] with
    ``cu_seqlens`` (``max_seqlen``: an upper bound of a row's tokens).  Row r's queries are
    the last of its lengths[r] tokens, which are all in the cache; a query sees the keys up to
    its own position (``causal``), and with ``window`` > 0 only the last ``window`` of them.
    scale defaults to dim ** -0.5.  Returns o bf16 like q and, with ``need_lse``, the log of
    the sum of exponentials f32 [..., query heads]; a query that sees nothing gets 0 and -inf."""
    dev = codes.device
    p = _problem(q, None, codes, scales, table, lengths, cu_seqlens, max_seqlen, mode,
                 codes.shape[-1] ** -0.5 if scale is None else float(scale), causal, window)
    lib = load()
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    else:
        _flat("out", out, torch.bfloat16, dev)
        _need(out.shape == q.shape, "out must have q's shape")
    lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev) if need_lse else None
    need = lib.gdn_kv8_workspace_bytes(_byref(p))
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    check("gdn_kv8_attention", lib.gdn_kv8_attention(
        _byref(p), q.data_ptr(), codes.data_ptr(), scales.data_ptr(), table.data_ptr(),
        lengths.data_ptr(), out.data_ptr(), lse.data_ptr() if need_lse else None,
        _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream(dev)))
    return (out, lse) if need_lse else out


def kv8_workspace_bytes(q, codes, scales, table, lengths, cu_seqlens=None, max_seqlen=None,
                        mode="e4m3", window=0) -> int:
    """Bytes of the workspace that kv8_attention takes for these arguments."""
    p = _problem(q, None, codes, scales, table, lengths, cu_seqlens, max_seqlen, mode, 1.0, True,
                 window)
    return int(load().gdn_kv8_workspace_bytes(_byref(p)))


def _pool_problem(codes, scales, table, lengths, refs) -> GdnKv8Pool:
    dev = codes.device
    _flat("codes", codes, torch.uint8, dev)
    _flat("scales", scales, torch.float32, dev)
    _need(codes.dim() == 6 and codes.shape[1] == 2,
          "codes must be [layers, 2, pages, heads, page, dim]")
    _need(scales.shape == codes.shape[:4], "scales must be [layers, 2, pages, heads]")
    p = GdnKv8Pool()
    p.planes, p.pages, p.heads, p.page, p.dim = 2 * codes.shape[0], *codes.shape[2:]
    p.rows, p.cols = 1, 0
    if table is not None:
        _flat("table", table, _i32, dev)
        _flat("lengths", lengths, _i32, dev)
        _flat("refs", refs, _i32, dev)
        _need(table.dim() == 2 and lengths.shape == (table.shape[0],),
              "table must be [rows, columns] and lengths [rows]")
        _need(refs.shape == (p.pages,), "refs must be [pages]")
        p.rows, p.cols = table.shape
    return p


def _pool_workspace(p, workspace, device):
    if workspace is None:
        workspace = torch.empty(load().gdn_kv8_pool_workspace_bytes(_byref(p)), dtype=torch.uint8,
                                device=device)
    return workspace


def kv8_copy_pages(codes, scales, src, dst):
    """Page src[i] is copied to page dst[i], in every layer: codes and scales, in place.  The
    pages of dst are distinct and none of them is in src.  src, dst int32 [n] on the device."""
    dev = codes.device
    p = _pool_problem(codes, scales, None, None, None)
    _flat("src", src, _i32, dev)
    _flat("dst", dst, _i32, dev)
    _need(src.dim() == 1 and src.shape == dst.shape, "src and dst must be [n]")
    check("gdn_kv8_copy_pages", load().gdn_kv8_copy_pages(
        _byref(p), codes.data_ptr(), scales.data_ptr(), src.data_ptr(), dst.data_ptr(),
        src.numel(), _stream(dev)))


def _fork(codes, scales, table, lengths, parents, drop, refs, workspace):
    dev = codes.device
    p = _pool_problem(codes, scales, table, lengths, refs)
    ws = _pool_workspace(p, workspace, dev)
    out = torch.empty_like(table), torch.empty_like(lengths), torch.empty_like(refs)
    missing = torch.empty(1, dtype=_i32, device=dev)
    check("gdn_kv8_fork", load().gdn_kv8_fork(
        _byref(p), codes.data_ptr(), scales.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        refs.data_ptr(), _ptr(parents), _ptr(drop), out[0].data_ptr(), out[1].data_ptr(),
        out[2].data_ptr(), missing.data_ptr(), ws.data_ptr(), ws.numel(), _stream(dev)))
    return (*out, missing)


def kv8_fork(codes, scales, table, lengths, parents, refs, workspace=None):
    """New row r takes the sequence of old row parents[r] (int32 [rows]; -1: it becomes empty).

    Whole pages are shared; the partly filled last page stays with the lowest row that takes
    the sequence and is copied, in every layer, to the lowest free pages for the others.
    Sequences that no row takes are released.  Returns new (table, lengths, refs, missing):
    missing int32 [1] counts the copies there was no free page for."""
    _flat("parents", parents, _i32, codes.device)
    _need(parents.shape == lengths.shape, "parents must be [rows]")
    return _fork(codes, scales, table, lengths, parents, None, refs, workspace)


def kv8_free(codes, scales, table, lengths, rows, refs, workspace=None):
    """Releases the sequences of the rows where ``rows`` (bool [rows]) holds.  Returns new
    (table, lengths, refs)."""
    _flat("rows", rows, torch.bool, codes.device)
    _need(rows.shape == lengths.shape, "rows must be bool [rows]")
    return _fork(codes, scales, table, lengths, None, rows, refs, workspace)[:3]


def kv8_reserve(codes, scales, table, lengths, extra, refs, workspace=None):
    """Room for extra[r] (int32 [rows]) more tokens of each row: the lowest free pages, in row
    order.  Returns new (table, lengths, refs, missing) with lengths + extra; the tokens are
    then written by kv8_append at the old lengths."""
    dev = codes.device
    p = _pool_problem(codes, scales, table, lengths, refs)
    _flat("extra", extra, _i32, dev)
    _need(extra.shape == lengths.shape, "extra must be [rows]")
    ws = _pool_workspace(p, workspace, dev)
    out = torch.empty_like(table), torch.empty_like(lengths), torch.empty_like(refs)
    missing = torch.empty(1, dtype=_i32, device=dev)
    check("gdn_kv8_reserve", load().gdn_kv8_reserve(
        _byref(p), table.data_ptr(), lengths.data_ptr(), refs.data_ptr(), extra.data_ptr(),
        out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), missing.data_ptr(),
        ws.data_ptr(), ws.numel(), _stream(dev)))
    return (*out, missing)


def kv8_compact(codes, scales, table, lengths, refs, workspace=None):
    """Live pages move to the start of the pool, in every layer: with n of them, the i-th
    lowest at or above n goes to the i-th lowest free page below n.  Returns new
    (table, refs, live) with live int32 [1] = n.  Page ids held elsewhere become stale."""
    dev = codes.device
    p = _pool_problem(codes, scales, table, lengths, refs)
    ws = _pool_workspace(p, workspace, dev)
    out = torch.empty_like(table), torch.empty_like(refs), torch.empty(1, dtype=_i32, device=dev)
    check("gdn_kv8_compact", load().gdn_kv8_compact(
        _byref(p), codes.data_ptr(), scales.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        refs.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(),
        ws.numel(), _stream(dev)))
    return out


def beam_select(logits, scores, finished=None, k: Optional[int] = None, eos=-1, workspace=None):
    """The k best continuations of each batch item's beams (k defaults to the beams).

    logits bf16 or f32 [batch, beams, vocab] (last dim contiguous, rows evenly spaced);
    scores f32 [batch, beams] running log probabilities; finished bool [batch, beams] or None.
    A candidate scores scores + log_softmax(logits); a finished beam has one, itself with token
    ``eos``.  Order: score, then beam, then logit, then token.  Returns (scores f32, parents
    int32 = batch * beams + beam, tokens int32, finished bool), each [batch, k]."""
    dev = logits.device
    _need(logits.is_cuda and logits.dim() == 3, "logits must be [batch, beams, vocab] on CUDA")
    b, w, v = logits.shape
    s = logits.stride()
    _need(v == 1 or s[2] == 1, "the vocabulary must be contiguous")
    row = s[1] if w > 1 else s[0] if b > 1 else v
    _need(w == 1 or b == 1 or s[0] == w * s[1], "rows of logits must be evenly spaced")
    _flat("scores", scores, torch.float32, dev)
    _need(scores.shape == (b, w), "scores must be [batch, beams]")
    if finished is not None:
        _flat("finished", finished, torch.bool, dev)
        _need(finished.shape == (b, w), "finished must be [batch, beams]")
    p = GdnBeamProblem()
    p.batch, p.stride, p.beams, p.vocab = b, row, w, v
    p.k = w if k is None else int(k)
    p.dtype = DTYPES.get({torch.bfloat16: "bf16", torch.float16: "fp16",
                          torch.float32: "fp32"}.get(logits.dtype), 99)
    p.eos = int(eos)
    lib = load()
    check("gdn_beam_validate", lib.gdn_beam_validate(_byref(p)))
    out = torch.empty(3, b, p.k, dtype=_i32, device=dev)
    done = torch.empty(b, p.k, dtype=torch.bool, device=dev)
    if workspace is None:
        workspace = torch.empty(lib.gdn_beam_workspace_bytes(_byref(p)), dtype=torch.uint8,
                                device=dev)
    best, parents, tokens = out.unbind(0)
    best = best.view(torch.float32)
    check("gdn_beam_select", lib.gdn_beam_select(
        _byref(p), logits.data_ptr(), scores.data_ptr(), _ptr(finished), best.data_ptr(),
        parents.data_ptr(), tokens.data_ptr(), done.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream(dev)))
    return best, parents, tokens, done


def beam_reorder(states: Sequence[torch.Tensor], parents, beams: int, out=None):
    """Row r of every state [rows, ...] becomes row parents[r] (int32, any shape of rows
    elements; -1: zeros).  In place by default: parents then stay within groups of ``beams``
    consecutive rows, and a row that keeps itself is not touched.  ``out`` gives other buffers
    of the same shapes, one per state (any parents).  Rows are a multiple of 16 bytes.
    Returns the states that were written."""
    dst = list(states if out is None else out)
    if not states:
        return dst
    dev, rows = states[0].device, states[0].shape[0]
    _flat("parents", parents, _i32, dev)
    _need(parents.numel() == rows, "parents must have one entry per row")
    _need(len(dst) == len(states), "out must have one buffer per state")
    n = len(dst)
    a, b, size = (ctypes.c_void_p * n)(), (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)()
    for i, (x, y) in enumerate(zip(states, dst)):
        _need(x.is_cuda and x.device == dev and x.is_contiguous() and x.shape[0] == rows,
              "states must be contiguous [rows, ...] on one device")
        _need(y is x or (y.shape == x.shape and y.dtype == x.dtype and y.device == dev
                         and y.is_contiguous()), "out must match the states")
        a[i], b[i] = x.data_ptr(), y.data_ptr()
        size[i] = x.numel() // rows * x.element_size() if rows else 0
    check("gdn_beam_reorder", load().gdn_beam_reorder(n, a, b, size, parents.data_ptr(), rows,
                                                      int(beams), _stream(dev)))
    return dst


__all__ = ["beam_reorder", "beam_select", "kv8_append", "kv8_attention", "kv8_compact",
           "kv8_copy_pages", "kv8_fork", "kv8_free", "kv8_pool", "kv8_reserve",
           "kv8_workspace_bytes", "GdnError"]

"""Serving operators: the 8-bit paged cache, the attention that reads it, and beam search.

Argument marshalling only (``include/gdn_qdq.h`` has the definitions).  A layer's cache is
``codes`` uint8 [2, pages, heads, page, dim] (0: K, 1: V) and ``scales`` f32 [2, pages, heads],
one scale per page of tokens and head; a pool over layers has a leading [layers].  Rows find
their pages in ``table`` int32 [rows, columns]; ``refs`` int32 [pages] counts the holders of a
page.  Everything runs on the current stream and nothing waits for the host.  A ``workspace`` is any
contiguous tensor with enough bytes, on the same device.
"""
from __future__ import annotations

import struct
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import DTYPES, QDQ_MODES, GdnError, load

_i32, _u8, _f32, _bf16 = torch.int32, torch.uint8, torch.float32, torch.bfloat16
_raw_stream = torch._C._cuda_getCurrentRawStream
_MODES = {k: v for k, v in QDQ_MODES.items() if v}
_XTYPES = {torch.bfloat16: DTYPES["bf16"], torch.float16: DTYPES["fp16"], torch.float32: DTYPES["fp32"]}


def _structure(layout):
    """Packs a problem as the C compiler lays it out."""
    pack = struct.Struct(layout).pack

    def packed(*fields):
        try:
            return pack(*fields)
        except struct.error as e:
            raise ValueError("a size or number of the call does not fit its C structure: %s" % e) from None
    return packed


_KV8 = _structure("@3q10ifP6q")
_POOL = _structure("@2q5i0q")
_BEAM = _structure("@2q5i0q")
_ROTARY = _structure("@4q2i")
_LOGITS = _structure("@4q3i0q")
_TOO_SMALL = -5  # GDN_ERR_WORKSPACE_TOO_SMALL
_contiguous = torch.contiguous_format
_shared_bytes = {}  # of the workspace, by the problem's sizes


def _fns():
    return _lib._lib or load()


def _raise(fn, status):
    raise GdnError(fn, status)


def _launch(dev, fn, *args):
    """fn(*args, the current stream of device dev), with that device current."""
    if torch._C._cuda_getDevice() == dev:
        return fn(*args, _raw_stream(dev))
    with torch.cuda.device(dev):
        return fn(*args, _raw_stream(dev))


def _need(cond, text):
    if not cond:
        raise ValueError(text)


def _plain(t, dtype, dev):
    """t is a contiguous tensor of this type on CUDA device number dev."""
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _say(dev, *named):
    """Raises for the first of (name, tensor, dtype) that is not plain."""
    for name, t, dtype in named:
        _need(isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == dev,
              "%s must be a CUDA tensor on cuda:%d" % (name, dev))
        _need(t.dtype == dtype, "%s must be %s" % (name, dtype))
        _need(t.is_contiguous(), "%s must be contiguous" % name)


def _room(workspace, dev):
    """Address and bytes of a workspace."""
    _need(isinstance(workspace, torch.Tensor) and workspace.get_device() == dev and workspace.is_contiguous(),
          "workspace must be a contiguous tensor on cuda:%d" % dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kv8_pool(layers, pages, heads, dim, page=64, device="cuda"):
    """An empty pool: (codes, scales) of zeros."""
    return (torch.zeros(layers, 2, pages, heads, page, dim, dtype=torch.uint8, device=device),
            torch.zeros(layers, 2, pages, heads, dtype=torch.float32, device=device))


def _strides(x, shape):
    """(row, token, head) strides in elements of [rows, tokens, heads, dim] or [total, heads, dim]."""
    s = x.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError("the last dim must be contiguous")
    if len(shape) == 4:
        a, b, c = s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0
        return a, b, c
    return 0, s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0


def _bad_problem(x, v, codes, scales, table, lengths, cu_seqlens, mode):
    """Says what _problem does not take."""
    dev = codes.get_device()
    _need(dev >= 0, "codes must be a CUDA tensor")
    _say(dev, ("codes", codes, _u8), ("scales", scales, _f32), ("table", table, _i32),
         ("lengths", lengths, _i32))
    _need(codes.dim() == 5 and codes.shape[0] == 2, "codes must be [2, pages, heads, page, dim]")
    _need(scales.shape == codes.shape[:3], "scales must be [2, pages, heads]")
    _need(table.dim() == 2 and lengths.shape == table.shape[:1],
          "table must be [rows, columns] and lengths [rows]")
    _need(x.get_device() == dev, "q, k, v must be on cuda:%d" % dev)
    _need(mode in _MODES, "mode must be one of %s, got %r" % (sorted(_MODES), mode))
    rows, heads, dim = table.shape[0], codes.shape[2], codes.shape[4]
    if cu_seqlens is None:
        _need(x.dim() == 4 and x.shape[0] == rows, "expected [rows, tokens, heads, dim]")
    else:
        _say(dev, ("cu_seqlens", cu_seqlens, _i32))
        _need(x.dim() == 3, "expected packed [total, heads, dim]")
        _need(cu_seqlens.shape == (rows + 1,), "cu_seqlens must be [rows + 1]")
    _need(x.shape[-1] == dim, "head dim %d is not the cache's %d" % (x.shape[-1], dim))
    _need(heads > 0 and x.shape[-2] > 0 and x.shape[-2] % heads == 0,
          "%d heads cannot share %d K/V heads" % (x.shape[-2], heads))
    if v is not None:
        _need(v.get_device() == dev and v.dtype is x.dtype and v.shape == x.shape,
              "k and v must have the same shape, type and device")
        _need(x.shape[-2] == heads, "k and v must have the cache's heads")
    raise ValueError("arguments do not fit together")


def _problem(x, v, codes, scales, table, lengths, cu_seqlens, max_seqlen, mode, scale, causal,
             window, group=0):
    """The packed gdn_kv8_problem (``group`` where x has the K/V heads).  (Texts are made only for what is refused: this is on the
    way of every token.)"""
    dev = codes.get_device()
    cs, shape, m = codes.shape, x.shape, _MODES.get(mode)
    if not (dev >= 0 and codes.dtype is _u8 and codes.is_contiguous() and _plain(scales, _f32, dev)
            and _plain(table, _i32, dev) and _plain(lengths, _i32, dev) and x.get_device() == dev
            and len(cs) == 5 and cs[0] == 2 and scales.shape == cs[:3] and table.dim() == 2
            and lengths.shape == table.shape[:1] and m is not None):
        _bad_problem(x, v, codes, scales, table, lengths, cu_seqlens, mode)
    _, pages, heads, page, dim = cs
    rows, cols = table.shape
    if len(shape) != (4 if cu_seqlens is None else 3):
        _bad_problem(x, v, codes, scales, table, lengths, cu_seqlens, mode)
    if cu_seqlens is None:
        fits = shape[0] == rows
        tokens, cu = shape[1], 0
        total = rows * tokens
    else:
        fits = _plain(cu_seqlens, _i32, dev) and cu_seqlens.shape == (rows + 1,)
        total = tokens = shape[0]
        if max_seqlen is not None and max_seqlen < tokens:
            tokens = int(max_seqlen)
        cu = cu_seqlens.data_ptr()
    xh = shape[-2]
    if not (fits and shape[-1] == dim and heads > 0 and xh > 0 and xh % heads == 0 and (
            v is None or (xh == heads and v.shape == shape and v.dtype is x.dtype and v.get_device() == dev))):
        _bad_problem(x, v, codes, scales, table, lengths, cu_seqlens, mode)
    strides = _strides(x, shape)
    more = strides if v is None else _strides(v, shape)
    return _KV8(pages, rows, total, tokens, cols, heads, group or xh // heads, dim, page, m,
                _XTYPES.get(x.dtype, 99), causal, window, scale, cu, *strides, *more)


def kv8_append(k, v, codes, scales, table, start, cu_seqlens=None, max_seqlen=None, mode="e4m3"):
    """New tokens go to the cache, in place: row r's at positions start[r] onwards.

    k, v bf16 [rows, tokens, heads, dim], or packed [total, heads, dim] with ``cu_seqlens``
    int32 [rows + 1] (``max_seqlen``: an upper bound of a row's tokens, further ones are not
    written; without it the call is laid out for one row with all of them); any strides that are
    multiples of 8, last dim contiguous.  codes, scales: one layer's cache.  A page's scale is
    max |x| / 448 (E4M3) or / 127 (INT8) over its tokens so far; where a new token raises it,
    the page's older codes are rounded again.  A NaN or an infinity in a token makes the scale one."""
    p = _problem(k, v, codes, scales, table, start, cu_seqlens, max_seqlen, mode, 1.0, 1, 0)
    st = _fns().gdn_kv8_append(p, k.data_ptr(), v.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                               table.data_ptr(), start.data_ptr(), _raw_stream(codes.get_device()))
    if st:
        _raise("gdn_kv8_append", st)


def _bad_rotary(q, k, cos, sin, dev):
    """Says what kv8_append_rotary does not take of its queries and angles."""
    _need(q.get_device() == dev and q.dtype is k.dtype, "q must have k's type and device")
    _need(q.dim() == k.dim() and q.dim() >= 3 and q.shape[:-2] == k.shape[:-2] and q.shape[-1] == k.shape[-1],
          "q must be like k but for the heads")
    _need(q.shape[-2] > 0 and q.shape[-2] % k.shape[-2] == 0,
          "%d heads cannot share %d K/V heads" % (q.shape[-2], k.shape[-2]))
    _say(dev, ("cos", cos, _f32), ("sin", sin, _f32))
    raise ValueError("cos and sin must be [positions, pairs]")


def kv8_append_rotary(q, k, v, codes, scales, table, start, cos, sin, interleaved=False, cu_seqlens=None,
                      max_seqlen=None, mode="e4m3"):
    """New tokens go to the cache with their keys turned by position, in place; returns the queries,
    turned as well, bf16 contiguous like q.

    k, v and the cache as for kv8_append; q bf16 [rows, tokens, query heads, dim], or packed
    [total, query heads, dim].  cos, sin f32 [positions, pairs]: the angles of row t are those of
    position t, pairs a multiple of 8 and at most dim / 2.  The first 2 * pairs dims of a head
    turn, dim j with dim pairs + j, or, ``interleaved``, dim 2 j with dim 2 j + 1.  The keys are
    quantized from the fp32 numbers that this gives.  The dims of a query that turn are NaN at positions
    that cos does not have, and so are the scales of key blocks written there; queries are 0 for packed
    tokens of no row, and NaN for a packed row with more than ``max_seqlen`` tokens."""
    dev, qs, ks, cs = codes.get_device(), q.shape, k.shape, cos.shape
    n = len(ks)
    heads, xh = (ks[-2], qs[-2]) if n >= 3 and len(qs) == n else (0, 0)
    if not (heads > 0 and xh > 0 and xh % heads == 0 and qs[0] == ks[0] and qs[-1] == ks[-1] and (n == 3 or qs[1] == ks[1])
            and q.dtype is k.dtype and q.get_device() == dev and cos.dtype is _f32 and sin.dtype is _f32
            and cos.get_device() == dev and sin.get_device() == dev and cos.is_contiguous() and sin.is_contiguous()
            and len(cs) == 2 and sin.shape == cs):
        _need(n >= 3 and ks[-2] > 0, "expected k of [rows, tokens, heads, dim] or [total, heads, dim]")
        _bad_rotary(q, k, cos, sin, dev)
    p = _problem(k, v, codes, scales, table, start, cu_seqlens, max_seqlen, mode, 1.0, 1, 0, xh // heads)
    w = _ROTARY(cs[0], *_strides(q, qs), 2 * cs[1], 1 if interleaved else 0)
    out = torch.empty_like(q, dtype=_bf16, memory_format=_contiguous)
    st = _launch(
        dev, _fns().gdn_kv8_append_rotary, p, w, q.data_ptr(), k.data_ptr(), v.data_ptr(), cos.data_ptr(), sin.data_ptr(),
        codes.data_ptr(), scales.data_ptr(), table.data_ptr(), start.data_ptr(), out.data_ptr())
    if st:
        _raise("gdn_kv8_append_rotary", st)
    return out


def kv8_attention(q, codes, scales, table, lengths, cu_seqlens=None, max_seqlen=None, mode="e4m3",
                  scale: Optional[float] = None, causal=True, window=0, need_lse=False,
                  workspace=None, out=None):
    """Attention of q over the cache: softmax(scale q K^T) V, query head h reading K/V head
    h // (query heads / heads).

    q bf16 [rows, tokens, query heads, dim], or packed [total, query heads, dim] with
    ``cu_seqlens`` (``max_seqlen``: an upper bound of a row's tokens, which a row with more gets
    NaN for; without it the call is laid out for one row with all of them, which costs time, most
    where rows have few).  Tokens of no row get 0 and -inf.  Row r's queries are
    the last of its lengths[r] tokens, which are all in the cache; a query sees the keys up to
    its own position (``causal``), and with ``window`` > 0 only the last ``window`` of them.
    scale defaults to dim ** -0.5.  Returns o bf16 like q and, with ``need_lse``, the log of
    the sum of exponentials f32 [..., query heads]; a query that sees nothing gets 0 and -inf, and
    one that is not finite or sees a key of a block whose scale is not gets NaN in both."""
    p = _problem(q, None, codes, scales, table, lengths, cu_seqlens, max_seqlen, mode,
                 codes.shape[-1] ** -0.5 if scale is None else scale, 1 if causal else 0, window)
    dev = codes.get_device()
    if out is None:
        out = torch.empty(q.shape, dtype=_bf16, device=codes.device)
    else:
        _say(dev, ("out", out, _bf16))
        _need(out.shape == q.shape, "out must have q's shape")
    lse = torch.empty(q.shape[:-1], dtype=_f32, device=codes.device) if need_lse else None
    lib = _fns()

    def call(ws):
        return lib.gdn_kv8_attention(
            p, q.data_ptr(), codes.data_ptr(), scales.data_ptr(), table.data_ptr(),
            lengths.data_ptr(), out.data_ptr(), lse.data_ptr() if need_lse else None,
            *((None, 0) if ws is None else _room(ws, dev)), _raw_stream(dev))

    st = call(workspace)
    if st == _TOO_SMALL and workspace is None:
        st = call(torch.empty(lib.gdn_kv8_workspace_bytes(p), dtype=_u8, device=codes.device))
    if st:
        _raise("gdn_kv8_attention", st)
    return (out, lse) if need_lse else out


def kv8_attention_shared(q, codes, scales, table, lengths, shared, beams, mode="e4m3",
                         scale: Optional[float] = None, causal=True, need_lse=False, workspace=None,
                         out=None):
    """kv8_attention for rows that have their first tokens in common, which are read once.

    Rows form groups of ``beams`` consecutive ones; shared int32 [rows / beams] counts the tokens
    that a group has in common (the prompt of its beams: with kv8_fork its whole pages; all rows'
    system prompt with beams = rows).  Positions below it are looked up in the table row of the
    group's first row (which has no more of them in common than it has), the others in the row's
    own, so the result is kv8_attention's, up to roundings, where the rows hold the same tokens there.
    q bf16 [rows, tokens, query heads, dim], for a few tokens each: whole prompts gain nothing from
    sharing, nor do groups with little in common, nor a few rows with many tokens of their own, which one
    CTA goes through for each row and K/V head (4 rows x 4 heads with 8000 own tokens behind 1024: 177 us,
    kv8_attention 21; with 500: 12 and 14).  A row's bits do not depend on what its group's other
    rows hold, nor on its place among them while beams * tokens * query heads / K/V heads <= 64.  The
    rest as for kv8_attention."""
    p = _problem(q, None, codes, scales, table, lengths, None, None, mode,
                 codes.shape[-1] ** -0.5 if scale is None else scale, 1 if causal else 0, 0)
    dev, beams = codes.get_device(), int(beams)
    if not _plain(shared, _i32, dev):
        _say(dev, ("shared", shared, _i32))
    _need(beams > 0 and q.shape[0] % beams == 0 and shared.shape == (q.shape[0] // beams,),
          "rows must be a multiple of beams, and shared [rows / beams]")
    if out is None:
        out = torch.empty_like(q, dtype=_bf16, memory_format=_contiguous)
    else:
        _say(dev, ("out", out, _bf16))
        _need(out.shape == q.shape, "out must have q's shape")
    lse = torch.empty(*q.shape[:-1], dtype=_f32, device=codes.device) if need_lse else None
    lib = _fns()
    if workspace is None:
        need = _shared_bytes.get((p, beams))
        if need is None:
            if len(_shared_bytes) >= 256:
                _shared_bytes.clear()
            need = _shared_bytes[p, beams] = lib.gdn_kv8_shared_workspace_bytes(p, beams)
        if need:
            workspace = torch.empty(need, dtype=_u8, device=codes.device)
    st = _launch(
        dev, lib.gdn_kv8_attention_shared, p, beams, q.data_ptr(), codes.data_ptr(), scales.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        shared.data_ptr(), out.data_ptr(), lse.data_ptr() if need_lse else None,
        *((None, 0) if workspace is None else _room(workspace, dev)))
    if st:
        _raise("gdn_kv8_attention_shared", st)
    return (out, lse) if need_lse else out


def kv8_shared_workspace_bytes(q, codes, scales, table, lengths, beams, mode="e4m3") -> int:
    """Bytes of the workspace that kv8_attention_shared takes for these arguments."""
    return int(_fns().gdn_kv8_shared_workspace_bytes(
        _problem(q, None, codes, scales, table, lengths, None, None, mode, 1.0, 1, 0), int(beams)))


def kv8_workspace_bytes(q, codes, scales, table, lengths, cu_seqlens=None, max_seqlen=None,
                        mode="e4m3", window=0) -> int:
    """Bytes of the workspace that kv8_attention takes for these arguments."""
    return int(_fns().gdn_kv8_workspace_bytes(
        _problem(q, None, codes, scales, table, lengths, cu_seqlens, max_seqlen, mode, 1.0, 1,
                 window)))


def _pool_problem(codes, scales, table=None, lengths=None, refs=None):
    """The packed gdn_kv8_pool."""
    dev = codes.get_device()
    if not (_plain(codes, _u8, dev) and _plain(scales, _f32, dev) and dev >= 0):
        _need(dev >= 0, "codes must be a CUDA tensor")
        _say(dev, ("codes", codes, _u8), ("scales", scales, _f32))
    cs = codes.shape
    _need(len(cs) == 6 and cs[1] == 2, "codes must be [layers, 2, pages, heads, page, dim]")
    _need(scales.shape == cs[:4], "scales must be [layers, 2, pages, heads]")
    rows, cols = 1, 0
    if table is not None:
        if not (_plain(table, _i32, dev) and _plain(lengths, _i32, dev) and _plain(refs, _i32, dev)):
            _say(dev, ("table", table, _i32), ("lengths", lengths, _i32), ("refs", refs, _i32))
        rows, cols = table.shape if table.dim() == 2 else (-1, -1)
        _need(rows >= 0 and lengths.shape == (rows,),
              "table must be [rows, columns] and lengths [rows]")
        _need(refs.shape == (cs[2],), "refs must be [pages]")
    return _POOL(cs[2], rows, cols, cs[4], 2 * cs[0], cs[3], cs[5])


def _pool_workspace(p, workspace, device):
    if workspace is None:
        workspace = torch.empty(_fns().gdn_kv8_pool_workspace_bytes(p), dtype=_u8, device=device)
    return workspace


def kv8_copy_pages(codes, scales, src, dst):
    """Page src[i] is copied to page dst[i], in every layer: codes and scales, in place.  The
    pages of dst are distinct and none of them is in src.  src, dst int32 [n] on the device."""
    p, dev = _pool_problem(codes, scales), codes.get_device()
    _say(dev, ("src", src, _i32), ("dst", dst, _i32))
    _need(src.dim() == 1 and src.shape == dst.shape, "src and dst must be [n]")
    st = _fns().gdn_kv8_copy_pages(p, codes.data_ptr(), scales.data_ptr(), src.data_ptr(),
                                   dst.data_ptr(), src.numel(), _raw_stream(dev))
    if st:
        _raise("gdn_kv8_copy_pages", st)


def _fork(codes, scales, table, lengths, parents, drop, refs, workspace):
    p = _pool_problem(codes, scales, table, lengths, refs)
    which, dtype = (parents, _i32) if drop is None else (drop, torch.bool)
    dev = codes.get_device()
    if not (_plain(which, dtype, dev) and which.shape == lengths.shape):
        _say(dev, ("parents" if drop is None else "rows", which, dtype))
        _need(False, "parents (rows) must have one entry per row")
    ws = _pool_workspace(p, workspace, codes.device)
    t, n, r = torch.empty_like(table), torch.empty_like(lengths), torch.empty_like(refs)
    missing = torch.empty(1, dtype=_i32, device=codes.device)
    st = _fns().gdn_kv8_fork(
        p, codes.data_ptr(), scales.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        refs.data_ptr(), parents.data_ptr() if drop is None else None,
        None if drop is None else drop.data_ptr(), t.data_ptr(), n.data_ptr(), r.data_ptr(),
        missing.data_ptr(), *_room(ws, dev), _raw_stream(dev))
    if st:
        _raise("gdn_kv8_fork", st)
    return t, n, r, missing


def kv8_fork(codes, scales, table, lengths, parents, refs, workspace=None):
    """New row r takes the sequence of old row parents[r] (int32 [rows]; -1: it becomes empty).

    Whole pages are shared; the partly filled last page stays with the lowest row that takes
    the sequence and is copied, in every layer, to the lowest free pages for the others.
    Sequences that no row takes are released.  Returns new (table, lengths, refs, missing):
    missing int32 [1] counts the copies there was no free page for."""
    return _fork(codes, scales, table, lengths, parents, None, refs, workspace)


def kv8_free(codes, scales, table, lengths, rows, refs, workspace=None):
    """Releases the sequences of the rows where ``rows`` (bool [rows]) holds.  Returns new
    (table, lengths, refs)."""
    return _fork(codes, scales, table, lengths, None, rows, refs, workspace)[:3]


def kv8_reserve(codes, scales, table, lengths, extra, refs, workspace=None):
    """Room for extra[r] (int32 [rows]) more tokens of each row: the lowest free pages, in row
    order.  Returns new (table, lengths, refs, missing) with lengths + extra; the tokens are
    then written by kv8_append at the old lengths."""
    p = _pool_problem(codes, scales, table, lengths, refs)
    dev = codes.get_device()
    _say(dev, ("extra", extra, _i32))
    _need(extra.shape == lengths.shape, "extra must be [rows]")
    ws = _pool_workspace(p, workspace, codes.device)
    t, n, r = torch.empty_like(table), torch.empty_like(lengths), torch.empty_like(refs)
    missing = torch.empty(1, dtype=_i32, device=codes.device)
    st = _fns().gdn_kv8_reserve(
        p, table.data_ptr(), lengths.data_ptr(), refs.data_ptr(), extra.data_ptr(), t.data_ptr(),
        n.data_ptr(), r.data_ptr(), missing.data_ptr(), *_room(ws, dev),
        _raw_stream(dev))
    if st:
        _raise("gdn_kv8_reserve", st)
    return t, n, r, missing


def kv8_compact(codes, scales, table, lengths, refs, workspace=None):
    """Live pages move to the start of the pool, in every layer: with n of them, the i-th
    lowest at or above n goes to the i-th lowest free page below n.  Returns new
    (table, refs, live) with live int32 [1] = n.  Page ids held elsewhere become stale."""
    p = _pool_problem(codes, scales, table, lengths, refs)
    dev = codes.get_device()
    ws = _pool_workspace(p, workspace, codes.device)
    t, r = torch.empty_like(table), torch.empty_like(refs)
    live = torch.empty(1, dtype=_i32, device=codes.device)
    st = _fns().gdn_kv8_compact(
        p, codes.data_ptr(), scales.data_ptr(), table.data_ptr(), lengths.data_ptr(),
        refs.data_ptr(), t.data_ptr(), r.data_ptr(), live.data_ptr(), *_room(ws, dev),
        _raw_stream(dev))
    if st:
        _raise("gdn_kv8_compact", st)
    return t, r, live


def _per_row(name, t, lead, width, dev, dtype):
    """Address of t, and elements from one row's to the next (0: one for all): t is [width], or
    [batch, beams, width] with rows evenly spaced or the same."""
    if t is None:
        return None, 0
    _need(isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype,
          "%s must be %s on cuda:%d" % (name, dtype, dev))
    shape, st = t.shape, t.stride()
    _need(len(shape) > 0 and shape[-1] >= width and (shape[-1] == 1 or st[-1] == 1) and (
        len(shape) == 1 or tuple(shape[:-1]) == lead),
          "%s must be [%d] or [batch, beams, %d], the last dim contiguous" % (name, width, width))
    if len(shape) == 1:
        return t.data_ptr(), 0
    row = st[1] if lead[1] > 1 else st[0] if lead[0] > 1 else 0
    _need(lead[0] <= 1 or lead[1] <= 1 or st[0] == lead[1] * row, "rows of %s must be evenly spaced" % name)
    return t.data_ptr(), row


def beam_logits(logits, tokens=None, lengths=None, repetition=None, frequency=None, presence=None,
                bias=None, mask=None, out=None):
    """Logits as beam_select then takes them: penalties for repeated tokens, a bias, a grammar's mask.

    logits bf16 or f32 [batch, beams, vocab] (last dim contiguous, rows evenly spaced).  tokens
    int32 [batch, beams, columns] with lengths int32 [batch, beams] (or all columns): what each row
    has said; ids outside the vocabulary (-1) count nowhere.  repetition, frequency, presence f32
    [batch, beams]: a token that is there n > 0 times has its logit divided by ``repetition`` if
    above 0, else multiplied by it, then less ``frequency`` * n and ``presence``.  bias f32
    [vocab] or [batch, beams, vocab] is added.  mask int32 [words] or [batch, beams, words]: token
    v is allowed where bit v % 32 of word v // 32 is set, the others get -inf.  All in fp32,
    rounded once.  The three penalties have one history: where repetition is to see more than the others
    do (the prompt as well), it takes a call of its own before theirs, and bf16 logits are rounded
    by both.  Returns logits like those given, contiguous; ``out`` may be the logits themselves."""
    dev = logits.get_device()
    _need(dev >= 0 and logits.dim() == 3, "logits must be [batch, beams, vocab] on CUDA")
    (b, w, v), s = logits.shape, logits.stride()
    lead = (b, w)
    _need(v == 1 or s[2] == 1, "the vocabulary must be contiguous")
    row = s[1] if w > 1 else s[0] if b > 1 else v
    _need(w <= 1 or b <= 1 or s[0] == w * row, "rows of logits must be evenly spaced")
    cols = 0
    if tokens is None:
        _need(repetition is None and frequency is None and presence is None and lengths is None,
              "penalties need tokens")
    else:
        if not _plain(tokens, _i32, dev):
            _say(dev, ("tokens", tokens, _i32))
        ts = tokens.shape
        _need(len(ts) == 3 and ts[0] == b and ts[1] == w, "tokens must be [batch, beams, columns]")
        cols = ts[2]
        for name, t, dtype in (("lengths", lengths, _i32), ("repetition", repetition, _f32),
                               ("frequency", frequency, _f32), ("presence", presence, _f32)):
            if t is not None:
                if not _plain(t, dtype, dev):
                    _say(dev, (name, t, dtype))
                _need(t.shape == lead, "%s must be [batch, beams]" % name)
    bias_at, bias_row = _per_row("bias", bias, lead, v, dev, _f32)
    mask_at, mask_row = _per_row("mask", mask, lead, (v + 31) // 32, dev, _i32)
    if out is None:
        out = torch.empty_like(logits, memory_format=_contiguous)
    else:
        _say(dev, ("out", out, logits.dtype))
        _need(out.shape == logits.shape, "out must have the logits' shape")
    st = _launch(
        dev, _fns().gdn_beam_logits, _LOGITS(b * w, row, bias_row, mask_row, v, cols, _XTYPES.get(logits.dtype, 99)), logits.data_ptr(),
        None if tokens is None else tokens.data_ptr(), None if lengths is None else lengths.data_ptr(),
        None if repetition is None else repetition.data_ptr(), None if frequency is None else frequency.data_ptr(),
        None if presence is None else presence.data_ptr(), bias_at, mask_at, out.data_ptr())
    if st:
        _raise("gdn_beam_logits", st)
    return out


def beam_select(logits, scores, finished=None, k: Optional[int] = None, eos=-1, workspace=None):
    """The k best continuations of each batch item's beams (k defaults to the beams).

    logits bf16 or f32 [batch, beams, vocab] (last dim contiguous, rows evenly spaced);
    scores f32 [batch, beams] running log probabilities; finished bool [batch, beams] or None.
    A candidate scores scores + log_softmax(logits); a finished beam has one, itself with token
    ``eos``.  Order: score, then beam, then logit, then token.  Returns (scores f32, parents
    int32 = batch * beams + beam, tokens int32, finished bool), each [batch, k]."""
    dev = logits.get_device()
    _need(dev >= 0 and logits.dim() == 3, "logits must be [batch, beams, vocab] on CUDA")
    b, w, v = logits.shape
    s = logits.stride()
    _need(v == 1 or s[2] == 1, "the vocabulary must be contiguous")
    row = s[1] if w > 1 else s[0] if b > 1 else v
    _need(w == 1 or b == 1 or s[0] == w * row, "rows of logits must be evenly spaced")
    if not _plain(scores, _f32, dev):
        _say(dev, ("scores", scores, _f32))
    _need(scores.shape == (b, w), "scores must be [batch, beams]")
    if finished is not None:
        if not _plain(finished, torch.bool, dev):
            _say(dev, ("finished", finished, torch.bool))
        _need(finished.shape == (b, w), "finished must be [batch, beams]")
    k = w if k is None else int(k)
    p = _BEAM(b, row, w, v, k, _XTYPES.get(logits.dtype, 99), int(eos))
    lib = _fns()
    st = lib.gdn_beam_validate(p)
    if st:
        _raise("gdn_beam_validate", st)
    on = logits.device
    best = torch.empty(b, k, dtype=_f32, device=on)
    parents = torch.empty(b, k, dtype=_i32, device=on)
    tokens = torch.empty(b, k, dtype=_i32, device=on)
    done = torch.empty(b, k, dtype=torch.bool, device=on)
    if workspace is None:
        workspace = torch.empty(lib.gdn_beam_workspace_bytes(p), dtype=_u8, device=on)
    st = lib.gdn_beam_select(
        p, logits.data_ptr(), scores.data_ptr(),
        None if finished is None else finished.data_ptr(), best.data_ptr(), parents.data_ptr(),
        tokens.data_ptr(), done.data_ptr(), *_room(workspace, dev),
        _raw_stream(dev))
    if st:
        _raise("gdn_beam_select", st)
    return best, parents, tokens, done


def beam_reorder(states: Sequence[torch.Tensor], parents, beams: int, out=None):
    """Row r of every state [rows, ...] becomes row parents[r] (int32, any shape of rows
    elements; -1: zeros).  In place by default: parents then stay within groups of ``beams``
    consecutive rows, and a row that keeps itself is not touched.  ``out`` gives other buffers
    of the same shapes, one per state (any parents); a buffer that is written may not overlap
    any other state or buffer.  Rows are a multiple of 16 bytes.
    Returns the states that were written."""
    dst = list(states if out is None else out)
    if not states:
        return dst
    _need(states[0].dim() > 0, "states must be [rows, ...]")
    dev, rows = states[0].get_device(), states[0].shape[0]
    if not _plain(parents, _i32, dev):
        _say(dev, ("parents", parents, _i32))
    _need(parents.numel() == rows, "parents must have one entry per row")
    _need(len(dst) == len(states), "out must have one buffer per state")
    n, src, to, size = len(dst), [], [], []
    for x, y in zip(states, dst):
        _need(x.get_device() == dev and dev >= 0 and x.is_contiguous() and x.dim() > 0 and x.shape[0] == rows,
              "states must be contiguous [rows, ...] on one CUDA device")
        _need(y is x or (y.shape == x.shape and y.dtype is x.dtype and y.get_device() == dev
                         and y.is_contiguous()), "out must match the states")
        src.append(x.data_ptr())
        to.append(y.data_ptr())
        size.append(x.numel() // rows * x.element_size() if rows else 0)
    pack = struct.Struct("%dQ" % n).pack
    st = _fns().gdn_beam_reorder(n, pack(*src), pack(*to), pack(*size), parents.data_ptr(), rows,
                                 int(beams), _raw_stream(dev))
    if st:
        _raise("gdn_beam_reorder", st)
    return dst


__all__ = ["beam_logits", "beam_reorder", "beam_select", "kv8_append", "kv8_append_rotary",
           "kv8_attention", "kv8_attention_shared", "kv8_compact", "kv8_copy_pages", "kv8_fork",
           "kv8_free", "kv8_pool", "kv8_reserve", "kv8_shared_workspace_bytes",
           "kv8_workspace_bytes", "GdnError"]

"""Serving oracle: the 8-bit paged cache, attention over it, its pages, and beam search — numpy.

TEST INFRASTRUCTURE ONLY.  Quantization follows the fp32 definition bit for bit (scale, its
rounded reciprocal, one rounding per product); attention and log-softmax are fp64; pages and
beams are plain loops over Python integers.
"""
from __future__ import annotations

import numpy as np

CODE_MAX = {"e4m3": 448.0, "int8": 127.0}
f32 = np.float32


def _e4m3_values():
    v = np.zeros(256)
    for b in range(256):
        e, f = (b >> 3) & 15, b & 7
        v[b] = (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)) * (-1 if b & 128 else 1)
    return v


_GRID = _e4m3_values()


def decode_codes(codes, mode):
    """Values of code bytes, fp64 (a byte that is no E4M3 number reads as the next on the grid)."""
    return codes.view(np.int8).astype(np.float64) if mode == "int8" else _GRID[codes]


def encode(u, mode):
    """Code bytes of fp32 numbers: nearest, ties to even, clamped."""
    u = np.asarray(u, f32)
    if mode == "int8":
        return np.clip(np.rint(u), -127, 127).astype(np.int8).view(np.uint8)
    a = np.minimum(np.abs(u.astype(np.float64)), 448.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    q = np.rint(a / 2.0 ** (e - 3)) * 2.0 ** (e - 3)   # may step up to the next binade: still exact
    e = np.where(q >= 2.0 ** -6, np.floor(np.log2(np.maximum(q, 2.0 ** -6))), -7)
    frac = np.where(e < -6, q / 2.0 ** -9, (q / 2.0 ** np.maximum(e, -6) - 1) * 8)
    code = (np.maximum(e + 7, 0) * 8 + frac).astype(np.uint8)
    return np.where(np.signbit(u), code | 128, code).astype(np.uint8)


def append(k, v, codes, scales, table, start, counts, mode):
    """k, v: one [n_r, heads, dim] fp32 array per row; codes, scales changed in place."""
    page = codes.shape[3]
    for r, (kr, vr) in enumerate(zip(k, v)):
        n, st = counts[r], int(start[r])
        for b in range(st // page, (st + n - 1) // page + 1 if n else 0):
            lo, hi = max(st, b * page), min(st + n, (b + 1) * page)
            if b >= table.shape[1] or not 0 <= table[r, b] < codes.shape[1]:
                continue
            pg, old = table[r, b], lo - b * page
            for i, x in ((0, kr), (1, vr)):
                for h in range(codes.shape[2]):
                    new = x[lo - st:hi - st, h].astype(f32)
                    was = scales[i, pg, h] if old else f32(0)
                    now = max(was, f32(np.abs(new).max()) / f32(CODE_MAX[mode]))
                    with np.errstate(divide="ignore", over="ignore"):
                        rcp = f32(1) / f32(now)
                    if np.isinf(rcp):
                        now = rcp = f32(0)
                    tile = codes[i, pg, h]
                    if now > was:
                        val = decode_codes(tile[:old], mode).astype(f32) * was
                        tile[:old] = encode(val * rcp, mode)
                    tile[old:old + hi - lo] = encode(new * rcp, mode)
                    scales[i, pg, h] = now


def attention(q, codes, scales, table, length, mode, scale, causal=True, window=0):
    """One row: q [n, query heads, dim] fp64, table [columns].  Returns o, lse fp64 and, for tolerances, per
    output the sum of weight * |v|, the largest weight * V scale * code maximum, and per
    query the largest sum of |scale q k|."""
    _, pages, heads, page, dim = codes.shape
    n, hq = q.shape[:2]
    end = max(0, min(length, len(table) * page))
    o, lse = np.zeros((n, hq, dim)), np.full((n, hq), -np.inf)
    absum, top, dots = np.zeros((n, hq, dim)), np.zeros((n, hq)), np.zeros((n, hq))
    ids = np.array([table[r] for r in range(-(-end // page))], dtype=np.int64)
    there = (ids >= 0) & (ids < pages)
    ids = np.where(there, ids, 0)
    exists = np.repeat(there, page)[:end]
    for h in range(heads):
        kk, vv = ((decode_codes(codes[i][ids, h], mode) * scales[i][ids, h].astype(np.float64)[:, None, None])
                  .reshape(-1, dim)[:end] for i in (0, 1))
        vs = np.repeat(scales[1][ids, h].astype(np.float64), page)[:end]
        for i in range(n):
            pos = length - n + i
            j = np.arange(end)
            ok = exists & ((j <= pos) if causal else (pos >= 0)) & ((j > pos - window) if window else True)
            if not ok.any():
                continue
            for g in range(hq // heads):
                x = h * (hq // heads) + g
                s = scale * (kk[ok] @ q[i, x])
                m = s.max()
                w = np.exp(s - m)
                z = w.sum()
                o[i, x], lse[i, x] = w @ vv[ok] / z, m + np.log(z)
                absum[i, x] = w @ np.abs(vv[ok]) / z
                top[i, x] = (w * vs[ok]).max() / z * CODE_MAX[mode]
                dots[i, x] = (np.abs(scale * kk[ok]) @ np.abs(q[i, x])).max()
    return o, lse, absum, top, dots


def turn(x, positions, cos, sin, interleaved):
    """x [n, heads, dim] fp32 turned by the angles of ``positions``; products and sums rounded to fp32."""
    y, half = np.array(x, f32), cos.shape[1]
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    for i, t in enumerate(positions):
        ok = 0 <= t < len(cos)
        c, s = (cos[t], sin[t]) if ok else (f32(np.nan), f32(np.nan))
        a, b = y[i][:, one].copy(), y[i][:, two].copy()
        y[i][:, one] = (a * c).astype(f32) - (b * s).astype(f32)
        y[i][:, two] = (b * c).astype(f32) + (a * s).astype(f32)
    return y


def attention_shared(q, codes, scales, first, own, shared, length, mode, scale, causal=True):
    """One row whose positions below ``shared`` are in the pages ``first``, the others in ``own``."""
    page = codes.shape[3]
    end = max(0, min(length, len(own) * page))
    j = np.arange(end)
    ids = np.array([(first if t < shared else own)[t // page] for t in j], dtype=np.int64)
    there = (ids >= 0) & (ids < codes.shape[1])
    at = np.where(there, ids, 0)
    # a cache with a page for each of the row's tokens
    one = codes[:, at, :, j % page, :]                 # [keys, 2, heads, dim]
    one = np.moveaxis(one, 0, 1)[:, :, :, None, :] if end else np.zeros((2, 0, codes.shape[2], 1, codes.shape[4]), np.uint8)
    table = np.where(there, j, -1)
    table = np.concatenate([table, np.full(max(len(own) * page - end, 0), -1, np.int64)])
    return attention(q, one, scales[:, at], table, length, mode, scale, causal)


def beam_logits(logits, tokens, lengths, repetition, frequency, presence, bias, mask):
    """fp64, [rows, vocab]; tokens a list of lists, mask bool [rows, vocab] (True: allowed) or None."""
    out = logits.astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for r in range(len(out)):
            count = {}
            for t in tokens[r][:max(int(lengths[r]), 0)] if tokens is not None else ():
                if 0 <= t < out.shape[1]:
                    count[int(t)] = count.get(int(t), 0) + 1
            for t, n in count.items():
                x = out[r, t]
                if repetition is not None:
                    rep = np.float64(repetition[r])
                    x = x / rep if x > 0 else x * rep
                out[r, t] = x - (frequency[r] * n if frequency is not None else 0) - (presence[r] if presence is not None else 0)
            if bias is not None:
                out[r] += bias[r]
            if mask is not None:
                out[r][~mask[r]] = -np.inf
    return out


def _own(table, lengths, page):
    return [[int(table[r][c]) for c in range(min(-(-max(int(n), 0) // page), len(table[r])))]
            for r, n in enumerate(lengths)]


def fork(table, lengths, refs, parents, page):
    """New (table, lengths, refs), the copies (source, destination), and the pages missed."""
    rows, cols = table.shape
    refs, out, lens = [int(x) for x in refs], np.full_like(table, -1), []
    own = _own(table, lengths, page)
    for pages in own:
        for p in pages:
            refs[p] -= 1
    first, want = {}, []
    for r in range(rows):
        p = int(parents[r])
        n = int(lengths[p]) if p >= 0 else 0
        lens.append(n)
        for c, pg in enumerate(own[p] if p >= 0 else []):
            if (c + 1) * page > n and first.setdefault(p, r) != r:
                want.append((r, c, pg))
            else:
                out[r, c] = pg
                refs[pg] += 1
    free = [i for i, x in enumerate(refs) if x == 0]
    moves = []
    for (r, c, pg), to in zip(want, free):
        out[r, c] = to
        refs[to] = 1
        moves.append((pg, to))
    return out, np.array(lens, np.int32), np.array(refs, np.int32), moves, len(want) - len(moves)


def reserve(table, lengths, refs, extra, page):
    rows, cols = table.shape
    refs, out, missing = [int(x) for x in refs], np.full_like(table, -1), 0
    free = iter([i for i, x in enumerate(refs) if x == 0])
    lens = []
    for r, own in enumerate(_own(table, lengths, page)):
        out[r, :len(own)] = own
        n = int(lengths[r])
        want = n + max(int(extra[r]), 0)
        lens.append(max(n, min(want, cols * page)))
        for c in range(-(-n // page), -(-want // page)):
            pg = next(free, -1) if c < cols else -1
            if pg < 0:
                missing += 1
                continue
            out[r, c] = pg
            refs[pg] = 1
    return out, np.array(lens, np.int32), np.array(refs, np.int32), missing


def compact(table, lengths, refs, page):
    n = int((refs > 0).sum())
    moves = list(zip([p for p in range(n, len(refs)) if refs[p] > 0], [p for p in range(n) if refs[p] <= 0]))
    to, new = dict(moves), np.where(np.arange(len(refs)) < n, refs, 0)
    for a, b in moves:
        new[b] = refs[a]
    out = np.full_like(table, -1)
    for r, own in enumerate(_own(table, lengths, page)):
        out[r, :len(own)] = [to.get(p, p) for p in own]
    return out, new.astype(np.int32), moves, n


def beam_select(logits, scores, finished, k, eos):
    """fp64; NaN counts as -inf.  Also the candidates' scores around the k-th, for ties."""
    batch, beams, vocab = logits.shape
    best, parents, tokens, done = [], [], [], []
    for b in range(batch):
        cand = []
        for w in range(beams):
            if finished[b, w]:
                cand += [(-float(scores[b, w]) if i == 0 else np.inf, w, i, eos) for i in range(k)]
                continue
            x = np.where(np.isnan(logits[b, w]), -np.inf, logits[b, w].astype(np.float64))
            order = np.argsort(-x, kind="stable")[:k]
            m = x.max()
            for i in range(k):
                if i >= len(order):
                    cand.append((np.inf, w, i, 0))
                    continue
                lp = -np.inf if m == -np.inf else x[order[i]] - m - np.log(np.exp(x - m).sum())
                cand.append((-(float(scores[b, w]) + lp), w, i, int(order[i])))
        cand.sort(key=lambda c: c[:3])
        top = cand[:k]
        best.append([-c[0] for c in top])
        parents.append([b * beams + c[1] for c in top])
        tokens.append([c[3] for c in top])
        done.append([bool(finished[b, c[1]]) or (eos >= 0 and c[3] == eos) for c in top])
    return np.array(best), np.array(parents), np.array(tokens), np.array(done)

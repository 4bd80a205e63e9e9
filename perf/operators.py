"""Cases of the serving operators: an 8-bit paged cache (append, attention, pages) and beam search.

A hybrid stack of gated-delta-rule and attention layers answers with a recurrent state per GDN layer and a
cache of K and V per attention layer.  The cache is held in 8 bits (E4M3 or INT8) with one scale per page of
tokens and head:

  codes   uint8 [2, pages, heads, page, dim]   (0: K, 1: V); a pool over layers has a leading [layers]
  scales  f32   [2, pages, heads]              value = code * scale
  table   int32 [rows, columns]                page of each block of a row's tokens, -1 where there is none
  lengths int32 [rows], refs int32 [pages]     tokens of a row; rows (and other holders) of a page

``run`` computes a case in its plain form, or, with ``own``, by the package's entry points.
"""
import math
import random

import torch

own = False

CODE_MAX = {"e4m3": 448.0, "int8": 127.0}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user, one token, short context: latency of a single call
        dict(name="decode_one", kind="attention", rows=1, tokens=1, packed=False, heads=2, group=8, dim=128, page=64,
             mode="e4m3", context=701, spread=0, window=0),
        # a serving batch at ordinary, uneven context lengths
        dict(name="decode_batch", kind="attention", rows=64, tokens=1, packed=False, heads=8, group=4, dim=128, page=64,
             mode="e4m3", context=8192, spread=6000, window=0),
        # two users with long documents
        dict(name="decode_long", kind="attention", rows=2, tokens=1, packed=False, heads=4, group=4, dim=128, page=128,
             mode="int8", context=131071, spread=30000, window=0),
        # several drafted tokens checked at once, sliding window, small pages and heads
        dict(name="decode_drafts", kind="attention", rows=24, tokens=5, packed=False, heads=2, group=3, dim=64, page=16,
             mode="int8", context=3001, spread=2900, window=1024),
        # a chunk of three uneven prompts against what is cached of them
        dict(name="prefill_chunk", kind="attention", rows=3, tokens=2048, packed=True, heads=4, group=4, dim=128, page=64,
             mode="e4m3", context=8200, spread=5000, window=0),
        # whole prompts, one K/V head per query head
        dict(name="prefill_prompts", kind="attention", rows=4, tokens=4096, packed=False, heads=16, group=1, dim=128,
             page=64, mode="int8", context=4096, spread=0, window=0),
        # one token of each sequence of a batch goes to the cache
        dict(name="append_token", kind="append", rows=64, tokens=1, packed=False, heads=8, dim=128, page=64, mode="e4m3",
             context=1000, spread=900),
        # uneven prompts go to the cache
        dict(name="append_prompts", kind="append", rows=8, tokens=4096, packed=True, heads=8, dim=128, page=32,
             mode="int8", context=300, spread=299),
        # beams are chosen anew: full pages shared, the last page of a sequence copied for its further beams
        dict(name="fork_batch", kind="fork", rows=128, beams=8, layers=4, heads=4, dim=128, page=64, context=2900,
             spread=2000, pages=8000),
        # the live pages of a fragmented pool move to its start
        dict(name="compact_small", kind="compact", rows=8, beams=1, layers=2, heads=2, dim=64, page=32, context=600,
             spread=400, pages=500),
        # one beam step: selection over beams and vocabulary, the recurrent states follow; one user, and a batch
        dict(name="beam_one", kind="beam", batch=1, beams=4, vocab=32000, dtype="bf16", layers=1, heads=16, dim=128),
        dict(name="beam_batch", kind="beam", batch=16, beams=8, vocab=128000, dtype="bf16", layers=2, heads=16, dim=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "append", "fork", "compact", "beam", "beam"])
    page, dim, mode = rng.choice([16, 32, 64, 128]), rng.choice([64, 128]), rng.choice(["e4m3", "int8"])
    if kind in ("decode", "prefill"):
        heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 8, 16])
        group = min(group, 32 // heads if heads < 16 else 2)
        if kind == "decode":
            rows, tokens = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 5, 8])
            top = min(131072, 60_000_000 // (rows * heads * dim * max(1, group // 4)) * 8 // tokens)
            context = _log(rng, max(tokens, 1), max(tokens + 1, top))
            packed = False
        else:
            rows, tokens = _log(rng, 1, 8), _log(rng, 17, 4096)
            context = tokens + rng.choice([0, _log(rng, 1, 8192)])
            while rows * tokens * context * heads * group > 1_200_000_000:
                rows, tokens = max(1, rows // 2), max(17, tokens * 2 // 3)
                context = max(tokens, context * 3 // 4)
            packed = rng.random() < 0.6
        spread = rng.choice([0, rng.randint(0, context)])
        return dict(kind="attention", rows=rows, tokens=tokens, packed=packed, heads=heads, group=group, dim=dim, page=page,
                    mode=mode, context=context, spread=spread, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
    if kind == "append":
        rows, tokens, context = _log(rng, 1, 128), rng.choice([1, 1, _log(rng, 2, 4096)]), _log(rng, 1, 4000)
        while rows * tokens > 32768:
            rows = max(1, rows // 2)
        return dict(kind="append", rows=rows, tokens=tokens, packed=rng.random() < 0.5, heads=rng.choice([1, 2, 5, 8]), dim=dim,
                    page=page, mode=mode, context=context, spread=rng.randint(0, context))
    if kind in ("fork", "compact"):
        beams = rng.choice([2, 3, 4, 8]) if kind == "fork" else 1
        rows = beams * _log(rng, 1, 128 // beams)
        layers, heads, context = rng.choice([1, 2, 3, 4]), rng.choice([1, 2, 4]), _log(rng, 1, 2500)
        need = rows * -(-(context + 1) // page) + rows
        return dict(kind=kind, rows=rows, beams=beams, layers=layers, heads=heads, dim=dim, page=page, context=context,
                    spread=rng.randint(0, context), pages=need + rng.randint(0, need))
    beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
    batch = _log(rng, 1, max(1, 128 // beams))
    return dict(kind="beam", batch=batch, beams=beams, vocab=_log(rng, 100, 128000), dtype=rng.choice(["bf16", "f32"]),
                layers=rng.choice([1, 2]), heads=rng.choice([2, 4, 16]), dim=dim)


def _lens(case):
    """(length, new tokens) of each row: uneven, fixed by the case.  An attention row's new tokens are the last of its length."""
    got = []
    for r in range(case["rows"]):
        less = (r * 7919 + 13) % (case["spread"] + 1)
        n = case.get("tokens", 0)
        if case.get("packed"):
            n = max(1, n - (r * 613) % n)
        # a row may hold nothing, an attention row fewer tokens than the call has queries
        length = max(0, case["context"] - less)
        got.append((length, n))
    return got


def _pairs(case):
    """(visible query-key pairs, keys that are seen at all) over all rows."""
    pairs = keys = 0
    w = case["window"]
    for length, n in _lens(case):
        first = length - n  # position of the first query
        lo = max(first, 0)
        if length <= lo:
            continue
        # sum over p in [lo, length) of min(p + 1, window)
        if w:
            a, b = lo, min(length, max(lo, w))
            pairs += (a + 1 + b) * (b - a) // 2 + w * (length - b)
            keys += length - max(0, lo - w + 1)
        else:
            pairs += (lo + 1 + length) * (length - lo) // 2
            keys += length
    return pairs, keys


def work(case):
    k = case["kind"]
    if k == "attention":
        pairs, keys = _pairs(case)
        hq = case["heads"] * case["group"]
        n = sum(n for _, n in _lens(case))
        blocks = keys / case["page"] + case["rows"]
        return {"bytes": 2 * keys * case["heads"] * case["dim"] + blocks * (8 * case["heads"] + 4) + n * hq * (4 * case["dim"] + 4),
                "flops": 4 * case["dim"] * hq * pairs}
    if k == "append":
        n = sum(n for _, n in _lens(case)) * case["heads"] * case["dim"]
        return {"bytes": 6 * n, "flops": 4 * n}
    page_bytes = case["layers"] * 2 * case["heads"] * (case["page"] * case["dim"] + 4) if k != "beam" else 0
    if k == "fork":
        lens = [a for a, _ in _lens(case)]
        par = _parents(case)
        kept, moved = set(), 0
        for p in par:
            if p >= 0 and lens[p] % case["page"]:
                moved += p in kept
                kept.add(p)
        cols = case["context"] // case["page"] + 2
        return {"bytes": 2 * moved * page_bytes + 8 * case["rows"] * cols + 8 * case["pages"] + 12 * case["rows"], "flops": 0}
    if k == "compact":
        used = _pages_used(case)
        live = sum(used)
        moved = sum(1 for p in _places(case, live) if p >= live)
        cols = case["context"] // case["page"] + 2
        return {"bytes": 2 * moved * page_bytes + 8 * case["rows"] * cols + 8 * case["pages"], "flops": 0}
    rows = case["batch"] * case["beams"]
    logits = rows * case["vocab"]
    states = case["layers"] * rows * case["heads"] * case["dim"] ** 2
    return {"bytes": logits * (2 if case["dtype"] == "bf16" else 4) + 8 * states, "flops": 3 * logits}


def _pages_used(case):
    return [-(-a // case["page"]) for a, _ in _lens(case)]


def _places(case, n):
    """n different pages of the pool in a scattered order, fixed by the case."""
    return random.Random(case["pages"] * 31 + n).sample(range(case["pages"]), n)


def _parents(case):
    """Which old row each new row takes: within its group of beams; now and then a group ends (-1)."""
    r, got = random.Random(case["rows"] * 101 + case["context"]), []
    for b in range(0, case["rows"], case["beams"]):
        ended = r.random() < 0.08
        got += [-1 if ended else b + r.randrange(case["beams"]) for _ in range(case["beams"])]
    return got


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _quantise(x, mode):
    """Codes and scales of x [..., page, dim] fp32, one scale for the last two axes."""
    s = x.abs().amax((-2, -1)) / torch.tensor(CODE_MAX[mode], device=x.device)
    r = 1.0 / s
    r = torch.where(torch.isinf(r), torch.zeros_like(r), r)
    return _encode(x * r[..., None, None], mode), torch.where(r == 0, torch.zeros_like(s), s)


def _encode(u, mode):
    if mode == "e4m3":
        return u.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return u.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _decode(codes, mode):
    return codes.view(torch.float8_e4m3fn if mode == "e4m3" else torch.int8).float()


def _pool(gen, planes, pages, case, mode):
    """Pages of K and V as they come from a model: unit variance, some channels larger, heads of unlike size."""
    h, page, d = case["heads"], case["page"], case["dim"]
    codes = torch.empty(planes, pages, h, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(planes, pages, h, device="cuda")
    some = max(1, (1 << 27) // (h * page * d))
    for i in range(planes):
        chan = torch.exp(0.4 * torch.randn(h, 1, d, generator=gen, device="cuda"))
        for a in range(0, pages, some):
            b = min(pages, a + some)
            x = torch.randn(b - a, h, page, d, generator=gen, device="cuda") * chan
            codes[i, a:b], scales[i, a:b] = _quantise(x, mode)
    return codes, scales


def _table(used, places, cols):
    table = torch.full((len(used), cols), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(used):
        table[r, :n] = torch.tensor(places[at:at + n], dtype=torch.int32)
        at += n
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "kind": case["kind"], "mode": case.get("mode", "e4m3")}
    if case["kind"] == "beam":
        rows, v = case["batch"] * case["beams"], case["vocab"]
        # a peaked next-token distribution; running scores of a few tokens in; now and then a finished beam
        x = 2.5 * torch.randn(case["batch"], case["beams"], v, generator=gen, device="cuda")
        s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["scores"] = -20.0 - 3.0 * torch.rand(case["batch"], case["beams"], generator=gen, device="cuda")
        s["finished"] = torch.rand(case["batch"], case["beams"], generator=gen, device="cuda") < 0.06
        shape = (rows, case["heads"], case["dim"], case["dim"])
        s["states"] = [0.3 * torch.randn(shape, generator=gen, device="cuda") for _ in range(case["layers"])]
        s["spare"] = [torch.empty(shape, device="cuda") for _ in range(case["layers"])]  # the other of two buffers
        return s
    lens = _lens(case)
    s["lengths"] = torch.tensor([a for a, _ in lens], dtype=torch.int32, device="cuda")
    page = case["page"]
    if case["kind"] in ("attention", "append"):
        h, g, d, n = case["heads"], case.get("group", 1), case["dim"], sum(n for _, n in lens)
        after = [a + (n if case["kind"] == "append" else 0) for a, n in lens]
        used = [-(-a // page) for a in after]
        pages = sum(used) + 3
        places = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        s["codes"], s["scales"] = _pool(gen, 2, pages, case, s["mode"])
        s["table"] = _table(used, places, max(used + [1])).cuda()
        # q, k, v lie side by side, as one projection writes them
        qkv = torch.randn(n, (g + 2) * h, d, generator=gen, device="cuda").to(torch.bfloat16)
        q, k, v = 2 * qkv[:, :g * h], qkv[:, g * h:(g + 1) * h], qkv[:, (g + 1) * h:]
        s["q"], s["k"], s["v"] = q, k, v
        s["cu"], s["most"] = None, case["tokens"]
        if case["packed"]:
            ends = [0]
            for _, m in lens:
                ends.append(ends[-1] + m)
            s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
            s["most"] = max(m for _, m in lens)
        else:
            s["q"], s["k"], s["v"] = (x.unflatten(0, (case["rows"], case["tokens"])) for x in (q, k, v))
        s["scale"] = d ** -0.5
        return s
    used = _pages_used(case)
    live = sum(used)
    s["table"] = _table(used, _places(case, live), case["context"] // page + 2).cuda()
    refs = torch.zeros(case["pages"], dtype=torch.int32)
    refs[s["table"][s["table"] >= 0].cpu().long()] = 1
    s["refs"] = refs.cuda()
    s["parents"] = torch.tensor(_parents(case), dtype=torch.int32, device="cuda") if case["kind"] == "fork" else None
    shape = (case["layers"], 2, case["pages"], case["heads"])
    # codes of finite values: pages move as they are
    codes = torch.randint(0, 120, shape + (page, case["dim"]), generator=gen, device="cuda", dtype=torch.uint8)
    s["codes"], s["scales"] = codes, torch.rand(shape, generator=gen, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return {"attention": _attention, "append": _append, "fork": _fork, "compact": _compact, "beam": _beam}[s["kind"]](s)


def _held(codes, mode):
    """Codes as the numbers they stand for, in units of their scale."""
    return codes.view(torch.float8_e4m3fn if mode == "e4m3" else torch.int8)


def _rows_of(cu, total):
    """Row and place within the row of each packed token."""
    t = torch.arange(total, device=cu.device)
    row = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return row, t - cu[row]


def _attention(s):
    q, codes, scales, table, lengths, mode = (s[k] for k in ("q", "codes", "scales", "table", "lengths", "mode"))
    window = s["case"]["window"]
    if own:
        from gated_delta_rule_54_gb300 import kv8_attention
        o, lse = kv8_attention(q, codes, scales, table, lengths, cu_seqlens=s["cu"], max_seqlen=s["most"], mode=mode,
                               scale=s["scale"], causal=True, window=window, need_lse=True)
        return {"o": o, "lse": lse}
    rows, cols = table.shape
    h, page, d = codes.shape[2:]
    g = q.shape[-2] // h
    # the cache in 32 bits: [rows, heads, keys, dim]
    at = table.clamp(min=0).long()
    k, v = ((_decode(codes[i][at], mode) * scales[i][at][..., None, None]).transpose(1, 2).reshape(rows, h, cols * page, d)
            for i in (0, 1))
    x, n = q.float(), torch.full((rows,), q.shape[1] if s["cu"] is None else 0, device=q.device)
    if s["cu"] is not None:
        row, place = _rows_of(s["cu"], q.shape[0])
        n = s["cu"][1:] - s["cu"][:-1]
        x = torch.zeros(rows, s["most"], h * g, d, device=q.device)
        x[row, place] = q.float()
    t = x.shape[1]
    x = x.view(rows, t, h, g, d).permute(0, 2, 1, 3, 4).reshape(rows, h, t * g, d)
    p = (x @ k.transpose(2, 3)).view(rows, h, t, g, cols * page) * s["scale"]
    j = torch.arange(cols * page, device=q.device)
    pos = (lengths - n)[:, None] + torch.arange(t, device=q.device)  # [rows, t]
    seen = (j <= pos[..., None]) & (j < lengths[:, None, None])
    if window:
        seen &= j > pos[..., None] - window
    p = p.masked_fill(~seen[:, None, :, None], float("-inf"))
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(p - m)
    z = p.sum(-1, keepdim=True)
    lse = (torch.log(z) + m)[..., 0]  # [rows, h, t, g]
    o = (p.view(rows, h, t * g, -1) @ v).view(rows, h, t, g, d) / torch.where(z == 0, torch.ones_like(z), z)
    o = o.permute(0, 2, 1, 3, 4).reshape(rows, t, h * g, d)
    lse = lse.permute(0, 2, 1, 3).reshape(rows, t, h * g)
    if s["cu"] is not None:
        o, lse = o[row, place], lse[row, place]
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _append(s):
    k, v, codes, scales, table, start, mode = (s[n] for n in ("k", "v", "codes", "scales", "table", "lengths", "mode"))
    if own:
        from gated_delta_rule_54_gb300 import kv8_append
        kv8_append(k, v, codes, scales, table, start, cu_seqlens=s["cu"], max_seqlen=s["most"], mode=mode)
        return {"codes": _held(codes, mode), "scales": scales}
    rows, cols = table.shape
    h, page, d = codes.shape[2:]
    if s["cu"] is None:
        t = k.shape[1]
        row = torch.arange(rows, device=k.device).repeat_interleave(t)
        place = torch.arange(t, device=k.device).repeat(rows)
        n = torch.full((rows,), t, device=k.device, dtype=torch.int32)
        k, v = k.flatten(0, 1), v.flatten(0, 1)
    else:
        row, place = _rows_of(s["cu"], k.shape[0])
        n = s["cu"][1:] - s["cu"][:-1]
    pos = start[row] + place
    to, slot = table[row, pos // page].long(), pos % page
    # pages that get tokens, and how many old ones each keeps
    base = torch.arange(cols, device=k.device) * page
    hit = (base + page > start[:, None]) & (base < (start + n)[:, None])
    old = (start[:, None] - base).clamp(min=0)
    pages, old = table[hit].long(), old[hit]
    top = torch.tensor(CODE_MAX[mode], device=k.device)
    for i, x in enumerate((k, v)):
        x = x.float()
        most = torch.zeros(codes.shape[1], h, device=x.device).index_reduce_(0, to, x.abs().amax(-1), "amax")[pages] / top
        was = torch.where(old[:, None] > 0, scales[i][pages], torch.zeros_like(most))
        now = torch.maximum(was, most)
        r = 1.0 / now
        r = torch.where(torch.isinf(r), torch.zeros_like(r), r)
        now = torch.where(r == 0, torch.zeros_like(now), now)
        c = codes[i][pages]
        again = _encode(_decode(c, mode) * was[..., None, None] * r[..., None, None], mode)
        grown = (torch.arange(page, device=x.device) < old[:, None])[:, None, :, None] & (now > was)[..., None, None]
        codes[i][pages] = torch.where(grown, again, c)
        scales[i][pages] = now
        all_r = torch.zeros(codes.shape[1], h, device=x.device)
        all_r[pages] = r
        codes[i][to[:, None], torch.arange(h, device=x.device), slot[:, None]] = _encode(x * all_r[to][..., None], mode)
    return {"codes": _held(codes, mode), "scales": scales}


def _fork(s):
    codes, scales, table, lengths, parents, refs = (s[n] for n in ("codes", "scales", "table", "lengths", "parents", "refs"))
    if own:
        from gated_delta_rule_54_gb300 import kv8_fork
        table, lengths, refs, missing = kv8_fork(codes, scales, table, lengths, parents, refs)
        return {"codes": _held(codes, "e4m3"), "scales": scales, "table": table, "lengths": lengths, "refs": refs, "missing": missing}
    rows, cols = table.shape
    page = codes.shape[4]
    used, whole = (lengths + page - 1) // page, lengths // page
    some = parents >= 0
    par = parents.clamp(min=0).long()
    r = torch.arange(rows, device=table.device)
    col = torch.arange(cols, device=table.device)
    children = torch.zeros(rows, device=table.device, dtype=torch.int32).index_add_(0, par, some.int())
    first = torch.full((rows,), rows, device=table.device).index_reduce_(0, par, torch.where(some, r, rows), "amin")
    copied = some & (lengths % page > 0)[par] & (first[par] != r)
    # shared pages are held once per child, a partly filled one once
    own_page = col < used[:, None]
    more = torch.where(col < whole[:, None], children[:, None] - 1, children[:, None].clamp(max=1) - 1)
    refs = refs.index_add(0, torch.where(own_page, table, 0).long().flatten(), torch.where(own_page, more, 0).int().flatten())
    rank = torch.cumsum(copied.int(), 0)
    fresh = torch.searchsorted(torch.cumsum((refs == 0).int(), 0), rank)
    got = copied & (fresh < refs.numel())
    lens = torch.where(some, lengths[par], 0)
    out = torch.where((col < ((lens + page - 1) // page)[:, None]), table[par], -1)
    last = (lens // page).long().clamp(max=cols - 1)
    out[r, last] = torch.where(copied, torch.where(got, fresh, -1).int(), out[r, last])
    src, dst = table[par, last][got].long(), fresh[got]
    codes[:, :, dst] = codes[:, :, src]
    scales[:, :, dst] = scales[:, :, src]
    refs[dst] = 1
    missing = (copied & ~got).sum().int().reshape(1)
    return {"codes": _held(codes, "e4m3"), "scales": scales, "table": out, "lengths": lens, "refs": refs, "missing": missing}


def _compact(s):
    codes, scales, table, lengths, refs = (s[n] for n in ("codes", "scales", "table", "lengths", "refs"))
    if own:
        from gated_delta_rule_54_gb300 import kv8_compact
        table, refs, live = kv8_compact(codes, scales, table, lengths, refs)
        return {"codes": _held(codes, "e4m3"), "scales": scales, "table": table, "refs": refs, "live": live}
    page, at = codes.shape[4], torch.arange(refs.numel(), device=refs.device)
    alive = refs > 0
    live = alive.sum()
    src, dst = at[alive & (at >= live)], at[~alive & (at < live)]
    codes[:, :, dst] = codes[:, :, src]
    scales[:, :, dst] = scales[:, :, src]
    to = at.clone()
    to[src] = dst
    owns = torch.arange(table.shape[1], device=table.device) < ((lengths + page - 1) // page)[:, None]
    table = torch.where(owns, to[table.clamp(min=0).long()].int(), -1)
    refs = refs.clone()
    refs[dst] = refs[src]
    refs[src] = 0
    return {"codes": _held(codes, "e4m3"), "scales": scales, "table": table, "refs": refs, "live": live.int().reshape(1)}


EOS = 2


def _beam(s):
    logits, scores, finished, states, spare = (s[n] for n in ("logits", "scores", "finished", "states", "spare"))
    batch, w, v = logits.shape
    if own:
        from gated_delta_rule_54_gb300 import beam_reorder, beam_select
        scores, parents, tokens, finished = beam_select(logits, scores, finished, eos=EOS)
        states = beam_reorder(states, parents, w, out=spare)
        return {"scores": scores, "parents": parents, "tokens": tokens, "finished": finished, "states": states}
    x = logits.float()
    m = x.amax(-1, keepdim=True)
    offset = scores - torch.log(torch.exp(x - m).sum(-1))
    # the best of each beam in order of logit, then token; a finished beam goes on with one candidate
    best, token = torch.sort(x, dim=-1, descending=True, stable=True)
    best, token = best[..., :w], token[..., :w]
    cand = (best - m) + offset[..., None]
    if cand.shape[-1] < w:
        cand = torch.nn.functional.pad(cand, (0, w - cand.shape[-1]), value=float("-inf"))
        token = torch.nn.functional.pad(token, (0, w - token.shape[-1]))
    only = torch.full_like(cand, float("-inf"))
    only[..., 0] = scores
    cand = torch.where(finished[..., None], only, cand)
    token = torch.where(finished[..., None], torch.full_like(token, EOS), token)
    score, at = torch.sort(cand.flatten(1), dim=-1, descending=True, stable=True)
    score, at = score[:, :w], at[:, :w]
    token = token.flatten(1).gather(1, at).int()
    beam = at // w
    done = finished.gather(1, beam) | (token == EOS)
    parents = (beam + torch.arange(batch, device=beam.device)[:, None] * w).int()
    out = [a[parents.flatten().long()] for a in states]
    return {"scores": score, "parents": parents, "tokens": token, "finished": done, "states": out}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, row by row
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "fork": _exact_pages, "compact": _exact_pages,
            "beam": _exact_beam}[case["kind"]](case, s)


def _grid(codes, mode):
    """Values of code bytes from the format's definition."""
    b = torch.arange(256, dtype=torch.float64)
    if mode == "int8":
        lut = torch.where(b < 128, b, b - 256)
    else:
        sign, e, f = torch.where(b >= 128, -1.0, 1.0), (b % 128) // 8, b % 8
        lut = sign * torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7))
    return lut.to(codes.device)[codes.int()]


def _exact_attention(case, s):
    if _pairs(case)[0] * case["heads"] * case["group"] * case["dim"] > 4e11:
        return None
    q, h, g, page = s["q"], case["heads"], case["group"], case["page"]
    o, lse = [], []
    at = 0
    for r, (length, n) in enumerate(_lens(case)):
        qr = (q[at:at + n] if case["packed"] else q[r]).double()
        at += n
        keys = -(-length // page) * page
        ids = s["table"][r, :keys // page].long()
        first = length - n
        orow = torch.zeros(n, h * g, case["dim"], dtype=torch.float64, device=q.device)
        lrow = torch.full((n, h * g), float("-inf"), dtype=torch.float64, device=q.device)
        for head in range(h if length else 0):
            kk, vv = ((_grid(s["codes"][i][ids, head], s["mode"]) * s["scales"][i][ids, head].double()[:, None, None])
                      .reshape(keys, -1)[:length] for i in (0, 1))
            for part in range(0, n, 1024):
                i = torch.arange(part, min(n, part + 1024), device=q.device) + first
                j = torch.arange(length, device=q.device)
                ok = j[None] <= i[:, None]
                if case["window"]:
                    ok &= i[:, None] - j[None] < case["window"]
                for x in range(g):
                    hq = head * g + x
                    t = (qr[part:part + 1024, hq] @ kk.T) / math.sqrt(case["dim"])
                    t = torch.where(ok, t, float("-inf"))
                    lse_t = torch.logsumexp(t, -1)
                    some = torch.isfinite(lse_t)
                    orow[part:part + 1024, hq] = torch.where(some[:, None], torch.softmax(t, -1).nan_to_num() @ vv, 0.0)
                    lrow[part:part + 1024, hq] = lse_t
        o.append(orow)
        lse.append(lrow)
    join = torch.cat if case["packed"] else torch.stack
    return {"o": join(o), "lse": join(lse)}


def _round_to(u, mode):
    if mode == "int8":
        return torch.round(u).clamp(-127, 127)
    a = u.abs().clamp(max=448.0)
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(u) * torch.minimum(torch.round(a / step) * step, torch.tensor(448.0, dtype=a.dtype, device=a.device))


def _exact_append(case, s):
    page, mode, top = case["page"], s["mode"], CODE_MAX[s["mode"]]
    values, scales = _grid(s["codes"], mode), s["scales"].double()
    table, at = s["table"].tolist(), 0
    if case["rows"] * (case["tokens"] // page + 2) > 6000:
        return None
    for r, (start, n) in enumerate(_lens(case)):
        for i, x in enumerate((s["k"], s["v"])):
            x = (x[at:at + n] if case["packed"] else x[r]).double()
            for b in range(start // page, (start + n - 1) // page + 1):
                p, lo, hi = table[r][b], max(start, b * page), min(start + n, (b + 1) * page)
                new, old = x[lo - start:hi - start].transpose(0, 1), lo - b * page
                was = scales[i, p] if old else torch.zeros_like(scales[i, p])
                now = torch.maximum(was, new.abs().amax((1, 2)) / top)
                grown = now > was
                again = _round_to(values[i, p, :, :old] * (was / now)[:, None, None], mode)
                values[i, p, :, :old] = torch.where(grown[:, None, None], again, values[i, p, :, :old])
                values[i, p, :, old:old + hi - lo] = _round_to(new / now[:, None, None], mode)
                scales[i, p] = now
        at += n
    return {"codes": values if mode == "e4m3" else None, "scales": scales}


def _exact_pages(case, s):
    """Pages one at a time; tables are whole numbers and have no value in 64 bits."""
    page, refs = case["page"], s["refs"].tolist()
    lens, table = [a for a, _ in _lens(case)], s["table"].tolist()
    codes, scales = s["codes"].clone(), s["scales"].double()
    moves = []
    if case["kind"] == "compact":
        live = sum(x > 0 for x in refs)
        moves = list(zip([p for p in range(live, len(refs)) if refs[p]], [p for p in range(live) if not refs[p]]))
    else:
        kept, parents = set(), s["parents"].tolist()
        for r, a in enumerate(lens):
            for c in range(-(-a // page)):
                refs[table[r][c]] -= 1
        for r, p in enumerate(parents):
            for c in range(lens[p] // page if p >= 0 else 0):
                refs[table[p][c]] += 1
            if p >= 0 and lens[p] % page and p not in kept:
                refs[table[p][lens[p] // page]] += 1
                kept.add(p)
        kept.clear()
        free = iter([p for p, x in enumerate(refs) if not x])
        for p in parents:
            if p >= 0 and lens[p] % page:
                if p in kept:
                    moves.append((table[p][lens[p] // page], next(free)))
                kept.add(p)
    for a, b in moves:
        codes[:, :, b] = codes[:, :, a]
        scales[:, :, b] = scales[:, :, a]
    got = {"codes": codes.view(torch.float8_e4m3fn), "scales": scales, "table": None, "refs": None}
    got.update({"live": None} if case["kind"] == "compact" else {"lengths": None, "missing": None})
    return got


def _exact_beam(case, s):
    w, out, picks = case["beams"], [], []
    for b in range(case["batch"]):
        cand = []
        for i in range(w):
            if bool(s["finished"][b, i]):
                cand.append((-float(s["scores"][b, i]), i, 0))
                continue
            lp = torch.log_softmax(s["logits"][b, i].double(), -1)
            val, tok = torch.sort(lp, descending=True, stable=True)
            cand += [(-(float(x) + float(s["scores"][b, i])), i, j) for j, x in enumerate(val[:w].tolist())]
        cand.sort()
        out.append([-c[0] for c in cand[:w]])
        picks += [b * w + c[1] for c in cand[:w]]
    at = torch.tensor(picks, device="cuda")
    return {"scores": torch.tensor(out, dtype=torch.float64, device="cuda"), "parents": None, "tokens": None, "finished": None,
            "states": [x[at].double() for x in s["states"]]}

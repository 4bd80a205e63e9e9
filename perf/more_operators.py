"""Cases of a beam step's further operators, beside the 8-bit paged cache and the beam selection.

A hybrid stack answers with an 8-bit cache of K and V per attention layer

  codes   uint8 [2, pages, heads, page, dim]   (0: K, 1: V)
  scales  f32   [2, pages, heads]              value = code * scale
  table   int32 [rows, columns]                page of each block of a row's tokens, -1 where there is none
  lengths int32 [rows]                         tokens of a row (append: position of its first new token)

and per step and layer it

  rotary  rotates new queries and keys by their positions and appends keys and values to the cache
  shared  attends, where the rows of a group have their first tokens in common: those are read once for all
  logits  applies penalties for repeated tokens, a bias and a grammar's mask before the beams are selected

``run`` computes a case in its plain form, or, with ``own``, by the package's entry points.
"""
import math

import torch

own = False

CODE_MAX = {"e4m3": 448.0, "int8": 127.0}
INF = float("inf")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user, one token: latency of a single call
        dict(name="rotary_one", kind="rotary", rows=1, tokens=1, packed=False, heads=2, group=8, dim=128, rotary=128,
             interleaved=False, page=64, mode="e4m3", context=701, spread=0),
        # one token of each sequence of a serving batch
        dict(name="rotary_batch", kind="rotary", rows=64, tokens=1, packed=False, heads=8, group=4, dim=128, rotary=128,
             interleaved=False, page=64, mode="e4m3", context=1000, spread=900),
        # a chunk of a long document for three users: small pages, half of each head rotated, neighbouring pairs
        dict(name="rotary_chunk", kind="rotary", rows=3, tokens=701, packed=True, heads=4, group=3, dim=64, rotary=32,
             interleaved=True, page=16, mode="int8", context=60001, spread=40000),
        # uneven prompts
        dict(name="rotary_prompts", kind="rotary", rows=8, tokens=4096, packed=True, heads=8, group=4, dim=128, rotary=128,
             interleaved=False, page=64, mode="e4m3", context=0, spread=0),
        # the beams of one user after an ordinary prompt
        dict(name="shared_one", kind="shared", batch=1, beams=4, tokens=1, heads=4, group=4, dim=128, page=64, mode="e4m3",
             prefix=1472, prefix_spread=0, tail=100, tail_spread=0),
        # beam search for a batch of users: uneven prompts, answers of some length
        dict(name="shared_beams", kind="shared", batch=16, beams=8, tokens=1, heads=8, group=4, dim=128, page=64, mode="e4m3",
             prefix=4096, prefix_spread=3000, tail=150, tail_spread=60),
        # a serving batch behind one long system prompt, each row with a dialogue of its own
        dict(name="shared_prompt", kind="shared", batch=1, beams=64, tokens=1, heads=8, group=4, dim=128, page=64, mode="e4m3",
             prefix=16384, prefix_spread=0, tail=1024, tail_spread=1000),
        # beams over a long document
        dict(name="shared_long", kind="shared", batch=1, beams=8, tokens=1, heads=4, group=4, dim=128, page=128, mode="int8",
             prefix=131072, prefix_spread=0, tail=77, tail_spread=0),
        # several drafted tokens of every beam are checked at once, small heads and pages, odd sizes
        dict(name="shared_drafts", kind="shared", batch=5, beams=3, tokens=5, heads=2, group=3, dim=64, page=16, mode="int8",
             prefix=3001, prefix_spread=2100, tail=333, tail_spread=320),
        # one user: penalties over what the beams have said
        dict(name="logits_one", kind="logits", batch=1, beams=4, vocab=32000, dtype="bf16", history=500, spread=200,
             penalties=True, bias=False, allowed=1.0),
        # an answer in a grammar: few tokens may follow
        dict(name="logits_grammar", kind="logits", batch=8, beams=3, vocab=32003, dtype="f32", history=0, spread=0,
             penalties=False, bias=False, allowed=0.02),
        # a batch with everything
        dict(name="logits_batch", kind="logits", batch=16, beams=8, vocab=128000, dtype="bf16", history=4000, spread=3900,
             penalties=True, bias=True, allowed=0.9),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rotary", "rotary", "shared", "shared", "shared", "logits", "logits"])
    page, dim, mode = rng.choice([16, 32, 64, 128]), rng.choice([64, 128]), rng.choice(["e4m3", "int8"])
    heads, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8])
    if kind == "rotary":
        rows, tokens, context = _log(rng, 1, 128), rng.choice([1, 1, _log(rng, 2, 4096)]), _log(rng, 1, 60000)
        while rows * tokens * heads * (group + 2) * dim > 8 * 2500 * 8 * 6 * 128 or rows * (context + tokens) * heads * dim > 1 << 29:
            rows, context = max(1, rows // 2), context * 2 // 3
        return dict(kind=kind, rows=rows, tokens=tokens, packed=rng.random() < 0.5, heads=heads, group=group, dim=dim,
                    rotary=16 * rng.randint(1, dim // 16), interleaved=rng.random() < 0.4, page=page, mode=mode, context=context,
                    spread=rng.randint(0, context))
    if kind == "shared":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 33, 64])
        batch, tokens = _log(rng, 1, max(1, 128 // beams)), rng.choice([1, 1, 1, 2, 3, 5])
        # bytes of the cache as in the larger listed cases, and not more scores than there
        top = min(131072, (1 << 26) // (batch * heads * dim), 3_000_000_000 // (batch * beams * tokens * heads * group * dim))
        prefix = _log(rng, 1, max(2, top))
        tail = _log(rng, tokens, max(tokens + 1, min(2048, (1 << 25) // (batch * beams * heads * dim))))
        return dict(kind=kind, batch=batch, beams=beams, tokens=tokens, heads=heads, group=group, dim=dim, page=page, mode=mode,
                    prefix=prefix, prefix_spread=rng.choice([0, rng.randint(0, prefix)]), tail=tail,
                    tail_spread=rng.choice([0, rng.randint(0, tail)]))
    beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
    history = rng.choice([0, _log(rng, 1, 4000)])
    allowed = rng.choice([1.0, 0.9, 0.3, 0.02] if history else [0.9, 0.3, 0.02])
    return dict(kind=kind, batch=_log(rng, 1, max(1, 128 // beams)), beams=beams, vocab=_log(rng, 100, 128000),
                dtype=rng.choice(["bf16", "f32"]) if beams < 5 else "bf16", history=history, spread=rng.randint(0, history),
                penalties=history > 0, bias=rng.random() < 0.5, allowed=allowed)


def _lens(case):
    """(first position, new tokens) of each row of an append: uneven, fixed by the case."""
    got = []
    for r in range(case["rows"]):
        n = case["tokens"]
        if case["packed"]:
            n = max(1, n - (r * 613) % n)
        got.append((case["context"] - (r * 7919 + 13) % (case["spread"] + 1), n))
    return got


def _prefixes(case):
    return [case["prefix"] - (g * 4547 + 11) % (case["prefix_spread"] + 1) for g in range(case["batch"])]


def _tails(case):
    """Tokens of each row after its group's first ones; its queries are the last of them."""
    return [case["tail"] - (r * 7919 + 13) % (case["tail_spread"] + 1) for r in range(case["batch"] * case["beams"])]


def _histories(case):
    return [case["history"] - (r * 7919 + 13) % (case["spread"] + 1) for r in range(case["batch"] * case["beams"])]


def work(case):
    k = case["kind"]
    if k == "rotary":
        lens = _lens(case)
        n, d = sum(n for _, n in lens), case["dim"]
        places = len(set().union(*(range(a, a + m) for a, m in lens)))
        return {"bytes": n * case["heads"] * d * (6 + 4 * case["group"]) + places * case["rotary"] * 4,
                "flops": n * case["heads"] * (4 * d + 3 * case["rotary"] * (1 + case["group"]))}
    if k == "shared":
        h, d, t = case["heads"], case["dim"], case["tokens"]
        pre, tails = _prefixes(case), _tails(case)
        keys = sum(pre) + sum(tails)
        pairs = sum(case["beams"] * t * p for p in pre)
        pairs += sum(max(0, n - i) for n in tails for i in range(t))
        queries = len(tails) * t * h * case["group"]
        return {"bytes": 2 * keys * h * d + (keys / case["page"] + len(tails)) * (8 * h + 4) + queries * (4 * d + 4),
                "flops": 4 * d * h * case["group"] * pairs}
    rows, size = case["batch"] * case["beams"], 2 if case["dtype"] == "bf16" else 4
    # what the mask forbids need not be read
    n = rows * case["vocab"] * size * (1 + case["allowed"]) + 4 * sum(_histories(case))
    n += 4 * case["vocab"] if case["bias"] else 0
    n += rows * case["vocab"] / 8 if case["allowed"] < 1 else 0
    return {"bytes": n, "flops": 3 * rows * case["vocab"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _encode(u, mode):
    if mode == "e4m3":
        return u.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return u.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _decode(codes, mode):
    return codes.view(torch.float8_e4m3fn if mode == "e4m3" else torch.int8).float()


def _pool(gen, pages, case):
    """Pages of K and V as they come from a model: unit variance, some channels larger, heads of unlike size."""
    h, page, d, mode = case["heads"], case["page"], case["dim"], case["mode"]
    codes = torch.empty(2, pages, h, page, d, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, pages, h, device="cuda")
    some = max(1, (1 << 27) // (h * page * d))
    for i in range(2):
        chan = torch.exp(0.4 * torch.randn(h, 1, d, generator=gen, device="cuda"))
        for a in range(0, pages, some):
            b = min(pages, a + some)
            x = torch.randn(b - a, h, page, d, generator=gen, device="cuda") * chan
            s = x.abs().amax((-2, -1)) / CODE_MAX[mode]
            codes[i, a:b], scales[i, a:b] = _encode(x / s[..., None, None], mode), s
    return codes, scales


def _angles(positions, rotary):
    """cos and sin of position * 10000^(-2 j / rotary), which a program makes once."""
    f = 10000.0 ** (-2.0 * torch.arange(rotary // 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rotary": _prepare_rotary, "shared": _prepare_shared, "logits": _prepare_logits}[case["kind"]](case, seed, gen)


def _prepare_rotary(case, seed, gen):
    lens, page, h, g, d = _lens(case), case["page"], case["heads"], case["group"], case["dim"]
    used, n = [-(-(a + m) // page) for a, m in lens], sum(m for _, m in lens)
    # the pages that get tokens lie scattered in a pool; rows' older pages are not looked at
    hit = [range(a // page, u) for (a, _), u in zip(lens, used)]
    pages = sum(len(x) for x in hit) + 3
    places = iter(torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist())
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32)
    for r, cols in enumerate(hit):
        for c in cols:
            table[r, c] = next(places)
    s = {"case": case, "kind": "rotary", "mode": case["mode"], "interleaved": case["interleaved"], "table": table.cuda()}
    s["codes"], s["scales"] = _pool(gen, pages, case)
    s["start"] = torch.tensor([a for a, _ in lens], dtype=torch.int32, device="cuda")
    s["cos"], s["sin"] = _angles(max(a + m for a, m in lens), case["rotary"])
    # q, k, v lie side by side, as one projection writes them
    qkv = torch.randn(n, (g + 2) * h, d, generator=gen, device="cuda").to(torch.bfloat16)
    x = qkv[:, :g * h], qkv[:, g * h:(g + 1) * h], qkv[:, (g + 1) * h:]
    s["cu"], s["most"] = None, case["tokens"]
    if case["packed"]:
        ends = [0]
        for _, m in lens:
            ends.append(ends[-1] + m)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["most"] = max(m for _, m in lens)
    else:
        x = [t.unflatten(0, (case["rows"], case["tokens"])) for t in x]
    s["q"], s["k"], s["v"] = x
    return s


def _prepare_shared(case, seed, gen):
    page, h, g, d, beams = case["page"], case["heads"], case["group"], case["dim"], case["beams"]
    pre, tails = _prefixes(case), _tails(case)
    lens = [pre[r // beams] + n for r, n in enumerate(tails)]
    used = [-(-n // page) for n in lens]
    # whole pages of a group's first tokens are its rows' in common; what follows is a row's own
    pages = sum(p // page for p in pre) + sum(u - pre[r // beams] // page for r, u in enumerate(used))
    places = iter(torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist())
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32)
    for a in range(case["batch"]):
        common = pre[a] // page
        table[a * beams:(a + 1) * beams, :common] = torch.tensor([next(places) for _ in range(common)], dtype=torch.int32)
    for r, u in enumerate(used):
        for c in range(pre[r // beams] // page, u):
            table[r, c] = next(places)
    s = {"case": case, "kind": "shared", "mode": case["mode"], "beams": beams, "table": table.cuda(), "scale": d ** -0.5,
         "most": (max(pre), max(tails))}
    s["codes"], s["scales"] = _pool(gen, pages, case)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["shared"] = torch.tensor(pre, dtype=torch.int32, device="cuda")
    qkv = torch.randn(len(lens), case["tokens"], (g + 2) * h, d, generator=gen, device="cuda").to(torch.bfloat16)
    s["q"] = 2 * qkv[:, :, :g * h]
    return s


def _prepare_logits(case, seed, gen):
    b, w, v = case["batch"], case["beams"], case["vocab"]
    s = {"case": case, "kind": "logits"}
    # a peaked next-token distribution
    x = 2.5 * torch.randn(b, w, v, generator=gen, device="cuda")
    s["logits"] = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
    s.update(tokens=None, lengths=None, repetition=None, frequency=None, presence=None, bias=None, mask=None)
    if case["penalties"]:
        # few tokens are used often; histories end at different places, and what lies behind them is old
        u = torch.rand(b, w, case["history"] + -case["history"] % 4, generator=gen, device="cuda")
        s["tokens"] = (v ** u).int().clamp(max=v - 1)
        s["lengths"] = torch.tensor(_histories(case), dtype=torch.int32, device="cuda").view(b, w)
        s["repetition"] = 1.0 + 0.3 * torch.rand(b, w, generator=gen, device="cuda")
        s["frequency"] = 0.2 * torch.rand(b, w, generator=gen, device="cuda")
        s["presence"] = 0.5 * torch.rand(b, w, generator=gen, device="cuda")
    if case["bias"]:
        some = torch.rand(v, generator=gen, device="cuda") < 0.01
        s["bias"] = torch.where(some, 4.0 * torch.randn(v, generator=gen, device="cuda"), 0.0)
    if case["allowed"] < 1:
        # a grammar allows runs of tokens; 32 to a word, the lowest bit first
        words = (v + 31) // 32
        at = torch.rand(b, w, words, 4, 1, generator=gen, device="cuda") < case["allowed"]
        bits = (at.expand(-1, -1, -1, -1, 8).reshape(b, w, words, 32).long() << torch.arange(32, device="cuda")).sum(-1)
        s["mask"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return {"rotary": _rotary, "shared": _shared, "logits": _logits}[s["kind"]](s)


def _held(codes, mode):
    """Codes as the numbers they stand for, in units of their scale."""
    return codes.view(torch.float8_e4m3fn if mode == "e4m3" else torch.int8)


def _turn(x, cos, sin, interleaved):
    """x [tokens, heads, dim], cos and sin [tokens, 1, pairs]: the first 2 * pairs dims rotated pair by pair."""
    n = 2 * cos.shape[-1]
    a, b = (x[..., 0:n:2], x[..., 1:n:2]) if interleaved else (x[..., :n // 2], x[..., n // 2:n])
    a, b = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., n:]), -1)


def _rotary(s):
    q, k, v, codes, scales, table, start, mode = (s[n] for n in ("q", "k", "v", "codes", "scales", "table", "start", "mode"))
    if own:
        from gated_delta_rule_54_gb300 import kv8_append_rotary
        q = kv8_append_rotary(q, k, v, codes, scales, table, start, s["cos"], s["sin"], interleaved=s["interleaved"],
                              cu_seqlens=s["cu"], max_seqlen=s["most"], mode=mode)
        return {"q": q, "codes": _held(codes, mode), "scales": scales}
    rows, cols = table.shape
    h, page = codes.shape[2:4]
    shape = q.shape
    if s["cu"] is None:
        t = q.shape[1]
        row = torch.arange(rows, device=k.device).repeat_interleave(t)
        place = torch.arange(t, device=k.device).repeat(rows)
        n = torch.full((rows,), t, device=k.device, dtype=torch.int32)
        q, k, v = q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1)
    else:
        at = torch.arange(q.shape[0], device=q.device)
        row = torch.searchsorted(s["cu"][1:].contiguous(), at, right=True)
        place = at - s["cu"][row]
        n = s["cu"][1:] - s["cu"][:-1]
    pos = start[row] + place
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    turned = _turn(q.float(), cos, sin, s["interleaved"]).to(torch.bfloat16).view(shape)
    k, v = _turn(k.float(), cos, sin, s["interleaved"]), v.float()
    to, slot = table[row, pos // page].long(), pos % page
    # pages that get tokens, and how many old ones each keeps
    base = torch.arange(cols, device=k.device) * page
    hit = (base + page > start[:, None]) & (base < (start + n)[:, None])
    old = (start[:, None] - base).clamp(min=0)
    pages, old = table[hit].long(), old[hit]
    top = torch.tensor(CODE_MAX[mode], device=k.device)
    for i, x in enumerate((k, v)):
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
    return {"q": turned, "codes": _held(codes, mode), "scales": scales}


def _shared(s):
    q, codes, scales, table, lengths, shared, beams, mode = (
        s[n] for n in ("q", "codes", "scales", "table", "lengths", "shared", "beams", "mode"))
    if own:
        from gated_delta_rule_54_gb300 import kv8_attention_shared
        o, lse = kv8_attention_shared(q, codes, scales, table, lengths, shared, beams, mode=mode, scale=s["scale"], need_lse=True)
        return {"o": o, "lse": lse}
    rows, t = q.shape[:2]
    h, page, d = codes.shape[2:]
    g, groups = q.shape[2] // h, rows // beams
    x = q.float().view(rows, t, h, g, d).permute(0, 2, 1, 3, 4)  # [rows, h, t, g, d]

    def keys(rows_of, at):
        """K and V [n, h, keys, d] of the table rows ``rows_of`` [n] at positions ``at`` [n, keys]."""
        ids, slot = rows_of[torch.arange(at.shape[0], device=at.device)[:, None], at // page].long().clamp(min=0), at % page
        return ((_decode(codes[i], mode)[ids, :, slot] * scales[i][ids][..., None]).transpose(1, 2) for i in (0, 1))

    last = table.shape[1] * page - 1
    pos = (lengths - t)[:, None] + torch.arange(t, device=q.device)  # [rows, t]
    # the group's first tokens: all its rows' queries against one copy
    at = torch.arange(s["most"][0], device=q.device).clamp(max=last).expand(groups, -1)
    k, v0 = keys(table[::beams], at)
    xg = x.reshape(groups, beams, h, t * g, d).transpose(1, 2).reshape(groups, h, beams * t * g, d)
    p0 = (xg @ k.transpose(2, 3)).view(groups, h, beams, t, g, -1).transpose(1, 2).reshape(rows, h, t, g, -1) * s["scale"]
    first = shared.repeat_interleave(beams)
    seen = (torch.arange(at.shape[1], device=q.device) < torch.minimum(pos + 1, first[:, None])[..., None])[:, None, :, None]
    p0 = p0.masked_fill(~seen, -INF)
    # a row's own tokens
    at = first[:, None] + torch.arange(s["most"][1], device=q.device)
    k, v1 = keys(table, at.clamp(max=last))
    p1 = (x.reshape(rows, h, t * g, d) @ k.transpose(2, 3)).view(rows, h, t, g, -1) * s["scale"]
    p1 = p1.masked_fill(~(at[:, None] <= pos[..., None])[:, None, :, None], -INF)
    m = torch.maximum(p0.amax(-1, keepdim=True), p1.amax(-1, keepdim=True))
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    p0, p1 = torch.exp(p0 - m), torch.exp(p1 - m)
    z = p0.sum(-1, keepdim=True) + p1.sum(-1, keepdim=True)
    o = (p0.view(groups, beams, h, t * g, -1).transpose(1, 2).reshape(groups, h, beams * t * g, -1) @ v0)
    o = o.view(groups, h, beams, t, g, d).transpose(1, 2).reshape(rows, h, t, g, d)
    o = o + (p1.view(rows, h, t * g, -1) @ v1).view(rows, h, t, g, d)
    o = (o / torch.where(z == 0, torch.ones_like(z), z)).permute(0, 2, 1, 3, 4).reshape(q.shape)
    lse = (torch.log(z) + m)[..., 0].permute(0, 2, 1, 3).reshape(rows, t, h * g)
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _logits(s):
    if own:
        from gated_delta_rule_54_gb300 import beam_logits
        return beam_logits(s["logits"], s["tokens"], s["lengths"], s["repetition"], s["frequency"], s["presence"], s["bias"],
                           s["mask"])
    x = s["logits"].float()
    v = x.shape[-1]
    if s["tokens"] is not None:
        there = torch.arange(s["tokens"].shape[-1], device=x.device) < s["lengths"][..., None]
        n = torch.zeros_like(x).scatter_add_(-1, s["tokens"].long(), there.float())
        r = s["repetition"][..., None]
        y = torch.where(x > 0, x / r, x * r) - s["frequency"][..., None] * n - s["presence"][..., None]
        x = torch.where(n > 0, y, x)
    if s["bias"] is not None:
        x = x + s["bias"]
    if s["mask"] is not None:
        ok = (s["mask"][..., None] >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1
        x = x.masked_fill(ok.flatten(-2)[..., :v] == 0, -INF)
    return x.to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, row by row
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "shared": _exact_shared, "logits": _exact_logits}[case["kind"]](case, s)


def _grid(codes, mode):
    """Values of code bytes from the format's definition."""
    b = torch.arange(256, dtype=torch.float64)
    if mode == "int8":
        lut = torch.where(b < 128, b, b - 256)
    else:
        sign, e, f = torch.where(b >= 128, -1.0, 1.0), (b % 128) // 8, b % 8
        lut = sign * torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7))
    return lut.to(codes.device)[codes.int()]


def _round_to(u, mode):
    if mode == "int8":
        return torch.round(u).clamp(-127, 127)
    a = u.abs().clamp(max=448.0)
    step = 2.0 ** (torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(u) * torch.minimum(torch.round(a / step) * step, torch.tensor(448.0, dtype=a.dtype, device=a.device))


def _exact_rotary(case, s):
    page, mode, top, half = case["page"], s["mode"], CODE_MAX[s["mode"]], case["rotary"] // 2
    if case["rows"] * (case["tokens"] // page + 2) > 6000:
        return None
    # dims of the two parts of a pair
    j = torch.arange(half, device="cuda")
    one, two = (2 * j, 2 * j + 1) if case["interleaved"] else (j, half + j)
    values, scales = _grid(s["codes"], mode), s["scales"].double()
    table, at, turned = s["table"].tolist(), 0, []
    for r, (start, n) in enumerate(_lens(case)):
        q, k, v = ((s[x][at:at + n] if case["packed"] else s[x][r]).double() for x in ("q", "k", "v"))
        at += n
        cos, sin = (s[x][start:start + n].double()[:, None] for x in ("cos", "sin"))
        for x in (q, k):
            a, b = x[..., one], x[..., two]
            x[..., one], x[..., two] = a * cos - b * sin, a * sin + b * cos
        turned.append(q)
        for i, x in enumerate((k, v)):
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
    join = torch.cat if case["packed"] else torch.stack
    return {"q": join(turned), "codes": values if mode == "e4m3" else None, "scales": scales}


def _exact_shared(case, s):
    h, g, page, beams, t = case["heads"], case["group"], case["page"], case["beams"], case["tokens"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(o.shape[:-1], -INF, dtype=torch.float64, device="cuda")
    pre, tails = _prefixes(case), _tails(case)
    if len(tails) * h * max(t * g, 8) * max(pre) * case["dim"] > 4e11 or len(tails) * h > 20000:
        return None

    def of(row, a, b, head):
        at = torch.arange(a, b, device="cuda")
        ids = s["table"][row][at // page].long()
        return (_grid(s["codes"][i][ids, head, at % page], s["mode"]) * s["scales"][i][ids, head].double()[:, None] for i in (0, 1))

    for a in range(case["batch"]):
        for head in range(h):
            k0, v0 = of(a * beams, 0, pre[a], head)
            for r in range(a * beams, (a + 1) * beams):
                n = pre[a] + tails[r]
                k1, v1 = of(r, pre[a], n, head)
                x = s["q"][r, :, head * g:(head + 1) * g].double()
                w = torch.cat((x @ k0.T, x @ k1.T), -1) / math.sqrt(case["dim"])
                pos = torch.arange(n - t, n, device="cuda")
                w = torch.where(torch.arange(n, device="cuda") <= pos[:, None, None], w, -INF)
                z = torch.logsumexp(w, -1)
                w = torch.where(torch.isfinite(z)[..., None], torch.softmax(w, -1).nan_to_num(), 0.0)
                o[r, :, head * g:(head + 1) * g] = w[..., :pre[a]] @ v0 + w[..., pre[a]:] @ v1
                lse[r, :, head * g:(head + 1) * g] = z
    return {"o": o, "lse": lse}


def _exact_logits(case, s):
    got = s["logits"].double()
    for r in range(case["batch"] * case["beams"]):
        i = r // case["beams"], r % case["beams"]
        x = got[i]
        if s["tokens"] is not None:
            seen, n = torch.unique(s["tokens"][i][:int(s["lengths"][i])], return_counts=True)
            seen, rep = seen.long(), s["repetition"][i].double()
            y = x[seen]
            y = torch.where(y > 0, y / rep, y * rep) - s["frequency"][i].double() * n - s["presence"][i].double()
            x[seen] = y
        if s["bias"] is not None:
            x += s["bias"].double()
        if s["mask"] is not None:
            v = torch.arange(case["vocab"], device=x.device)
            word = s["mask"][i].long()[v // 32]
            x[(word // 2 ** (v % 32)) % 2 == 0] = -INF
    return got

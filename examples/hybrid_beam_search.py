"""Beam search with a hybrid stack: gated-delta-rule layers and attention over an 8-bit paged cache.

The model is small and its weights are random; what it shows is how the pieces meet:

  prompt   gdn_chunk_fwd_qdq gives each GDN layer's state, kv8_append and kv8_attention take the
           prompt through the attention layers
  step     kv8_reserve makes room for one token per row, gdn_decode_qdq steps the states in
           place, kv8_append and kv8_attention the caches
  beams    beam_select picks the continuations; beam_reorder moves the states with them and
           kv8_fork the pages (shared where they are full, copied where they are not)
  end      kv8_compact packs what is live

Nothing in a step waits for the host.  Run: python examples/hybrid_beam_search.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass, field

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_54_gb300 as gdn  # noqa: E402


@dataclass
class Config:
    vocab: int = 1000
    width: int = 256
    layers: str = "ggag"        # g: gated delta rule, a: attention
    heads: int = 2              # key heads of a GDN layer, K/V heads of an attention layer
    group: int = 2              # value / query heads per key head
    dim: int = 64
    page: int = 16
    mode: str = "e4m3"          # of the recurrent states and of the cache
    seed: int = 0


class HybridModel:
    """Weights, and one function per layer kind; every projection is one matrix product."""

    def __init__(self, cfg: Config):
        self.cfg = cfg
        gen = torch.Generator("cuda").manual_seed(cfg.seed)
        h, g, d, w = cfg.heads, cfg.group, cfg.dim, cfg.width
        wide = {"g": (2 + g) * h * d + 2 * g * h, "a": (2 + g) * h * d}

        def weight(n, m):
            return (torch.randn(n, m, generator=gen, device="cuda") * n ** -0.5).to(torch.bfloat16)

        self.embed = weight(cfg.vocab, w) * 8
        self.inp = [weight(w, wide[kind]) for kind in cfg.layers]
        self.out = [weight(h * g * d, w) for _ in cfg.layers]
        self.head = weight(w, cfg.vocab) * 4

    def project(self, layer, x):
        """x [rows, tokens, width] -> (q, k, v) as views of one tensor, and a GDN layer's beta, g."""
        c = self.cfg
        h, g, d = c.heads, c.group, c.dim
        y = F.rms_norm(x, (c.width,)) @ self.inp[layer]
        sizes = ((h, h, g * h) if c.layers[layer] == "g" else (g * h, h, h))
        heads = y[..., :(2 + g) * h * d].unflatten(-1, (sum(sizes), d))
        q, k, v = heads.split(sizes, dim=2)
        if c.layers[layer] == "a":
            return q, k, v, None, None
        rest = y[..., (2 + g) * h * d:].float()
        beta, decay = rest[..., :g * h].sigmoid(), -F.softplus(rest[..., g * h:])
        q, k = (F.normalize(t.float(), dim=-1).to(torch.bfloat16) for t in (q, k))
        return q, k, v.contiguous(), beta.contiguous(), decay.contiguous()

    def logits(self, x):
        return F.rms_norm(x, (self.cfg.width,)) @ self.head


@dataclass
class Session:
    """What a running search holds: states, the cache's pool, and who owns which page."""
    states: list
    codes: torch.Tensor
    scales: torch.Tensor
    table: torch.Tensor
    lengths: torch.Tensor
    refs: torch.Tensor
    missing: torch.Tensor = field(default=None)


def start(model: HybridModel, rows: int, pages: int, columns: int) -> Session:
    c = model.cfg
    codes, scales = gdn.kv8_pool(c.layers.count("a"), pages, c.heads, c.dim, page=c.page)
    i32 = dict(dtype=torch.int32, device="cuda")
    states = [torch.zeros(rows, c.heads * c.group, c.dim, c.dim, device="cuda") for k in c.layers if k == "g"]
    return Session(states, codes, scales, torch.full((rows, columns), -1, **i32), torch.zeros(rows, **i32),
                   torch.zeros(pages, **i32), torch.zeros(1, **i32))


def advance(model: HybridModel, s: Session, tokens: torch.Tensor) -> torch.Tensor:
    """tokens [rows, n] go through the stack; the logits after each row's last one, [rows, vocab].
    A prompt (the first call, n > 1) takes the chunked form of the GDN layers."""
    c, (rows, n) = model.cfg, tokens.shape
    first = s.lengths
    s.table, s.lengths, s.refs, missing = gdn.kv8_reserve(s.codes, s.scales, s.table, first,
                                                          torch.full_like(first, n), s.refs)
    s.missing = s.missing + missing
    x, state, cache = model.embed[tokens], 0, 0
    for layer, kind in enumerate(c.layers):
        q, k, v, beta, decay = model.project(layer, x)
        if kind == "g":
            q, k = q.contiguous(), k.contiguous()
            if n > 1:
                o, final, _ = gdn.gdn_chunk_fwd_qdq(q, k, v, beta, decay, s.states[state], state_mode=c.mode, w_mode=c.mode)
                s.states[state].copy_(final)
            else:
                o, _ = gdn.gdn_decode_qdq(q, k, v, beta, decay, s.states[state], state_mode=c.mode, state_out=s.states[state])
            o = o.to(torch.bfloat16)
            state += 1
        else:
            gdn.kv8_append(k, v, s.codes[cache], s.scales[cache], s.table, first, mode=c.mode)
            o = gdn.kv8_attention(q, s.codes[cache], s.scales[cache], s.table, s.lengths, mode=c.mode)
            cache += 1
        x = x + o.flatten(2) @ model.out[layer]
    return model.logits(x[:, -1])


def search(model: HybridModel, prompts: torch.Tensor, beams: int, steps: int, eos: int = 1, pages: int = None):
    """prompts [batch, n] -> (tokens [batch, beams, steps], scores [batch, beams], the session)."""
    batch, n = prompts.shape
    page, rows = model.cfg.page, batch * beams
    columns = -(-(n + steps) // page)
    s = start(model, rows, rows * columns + rows if pages is None else pages, columns)
    logits = advance(model, s, prompts.repeat_interleave(beams, 0))
    scores = torch.full((batch, beams), float("-inf"), device="cuda")
    scores[:, 0] = 0.0                       # the beams are one and the same so far
    done = torch.zeros(batch, beams, dtype=torch.bool, device="cuda")
    history = torch.zeros(rows, 0, dtype=torch.int32, device="cuda")
    for step in range(steps):
        scores, parents, tokens, done = gdn.beam_select(logits.view(batch, beams, -1), scores, done, eos=eos)
        parents = parents.flatten()
        gdn.beam_reorder(s.states, parents, beams)
        s.table, s.lengths, s.refs, missing = gdn.kv8_fork(s.codes, s.scales, s.table, s.lengths, parents, s.refs)
        s.missing = s.missing + missing
        history = torch.cat([history[parents.long()], tokens.view(rows, 1)], 1)
        if step + 1 < steps:
            logits = advance(model, s, tokens.view(rows, 1).long())
    s.table, s.refs, _ = gdn.kv8_compact(s.codes, s.scales, s.table, s.lengths, s.refs)
    return history.view(batch, beams, steps), scores, s


def main():
    model = HybridModel(Config())
    prompts = torch.randint(2, model.cfg.vocab, (3, 75), generator=torch.Generator().manual_seed(1)).cuda()
    tokens, scores, s = search(model, prompts, beams=4, steps=24)
    live = int((s.refs > 0).sum())
    print("pages: %d live of %d (a copy per row would hold %d), %d missing" % (
        live, s.refs.numel(), int(((s.lengths + model.cfg.page - 1) // model.cfg.page).sum()), int(s.missing)))
    for b in range(tokens.shape[0]):
        for w in range(2):
            print("prompt %d beam %d  score %8.3f  %s ..." % (b, w, float(scores[b, w]), tokens[b, w, :10].tolist()))


if __name__ == "__main__":
    main()

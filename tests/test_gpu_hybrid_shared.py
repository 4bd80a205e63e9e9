"""GPU: the beam search with its prompts read once for all beams, keys turned by position and a cost
for repeated tokens: append, attention, logits, selection and reordering together.

Every final beam is replayed in a session of the same shape and the same groups, in which no row
changes places; rows do not depend on their neighbours, so states and cached codes have to be
the same bit for bit, and the scores agree to the rounding of a log-softmax per step (2^-19 of
numbers below 32, plus the rounding of the running score).  Beside the search with kv8_attention, whose
outputs differ by roundings, the first step's logits agree to those: bf16 outputs (2^-8 of
each number, of both) that go through the rest of the stack."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_beam_search as ex  # noqa: E402

import gated_delta_rule_54_gb300 as gdn  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode,batch,beams,n,steps,cost", [("e4m3", 2, 4, 37, 20, 0.7), ("int8", 1, 3, 64, 35, 0.0), ("e4m3", 3, 1, 5, 4, 1.5)])
def test_search_equals_replay(mode, batch, beams, n, steps, cost):
    model = ex.HybridModel(ex.Config(vocab=200, mode=mode, seed=3))
    prompts = torch.randint(2, 200, (batch, n), generator=torch.Generator().manual_seed(5)).cuda()
    tokens, scores, s = ex.search(model, prompts, beams, steps, eos=-1, shared=True, frequency=cost)
    assert int(s.missing) == 0 and gdn.load().gdn_device_error(0) == 0
    rows, page = batch * beams, model.cfg.page
    r = ex.start(model, rows, s.refs.numel(), s.table.shape[1])
    logits = ex.advance(model, r, prompts.repeat_interleave(beams, 0))
    ex.share(r, batch, beams, n // page * page)
    total = torch.zeros(rows, dtype=torch.float64, device="cuda")
    said = tokens.view(rows, steps).int()
    for step in range(steps):
        t = said[:, step].long()
        x = logits.double().clone()
        if cost:  # the definition, on the logits as they are rounded
            count = torch.zeros_like(x).scatter_add_(1, said[:, :step].long(), torch.ones(rows, step, dtype=torch.float64, device="cuda"))
            x = (logits.float() - torch.tensor(cost, device="cuda") * count.float()).to(logits.dtype).double()
        total += torch.log_softmax(x, -1).gather(1, t[:, None])[:, 0]
        if step + 1 < steps:
            logits = ex.advance(model, r, t[:, None])
    assert torch.all((total - scores.flatten()).abs() <= steps * (2.0 ** -19 * 32 + 2.0 ** -24 * scores.abs().max()))
    assert torch.equal(s.lengths, r.lengths)
    for a, b in zip(s.states, r.states):
        assert torch.equal(a, b)
    for row in range(rows):
        have = int(r.lengths[row])
        for c in range(-(-have // page)):
            x, y, m = int(s.table[row, c]), int(r.table[row, c]), min(page, have - c * page)
            assert torch.equal(s.codes[:, :, x, :, :m], r.codes[:, :, y, :, :m])
            assert torch.equal(s.scales[:, :, x], r.scales[:, :, y])


def test_step_captured_and_replayed():
    """A decode step over a layer's cache (append, attention, logits, selection) in a graph, on contents that change."""
    torch.manual_seed(8)
    rows, beams, heads, group, dim, page, vocab = 6, 3, 2, 2, 64, 16, 300
    i32 = dict(dtype=torch.int32, device="cuda")
    codes, scales = gdn.kv8_pool(1, 40, heads, dim, page=page)
    table = torch.arange(rows * 6, **i32).view(rows, 6)
    table[1:3, :2], table[4:, :2] = table[0, :2].clone(), table[3, :2].clone()
    start, shared = torch.full((rows,), 40, **i32), torch.full((2,), 32, **i32)
    a = torch.arange(96, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    cos, sin = a.cos(), a.sin()
    x = torch.randn(rows, 40, 2 * heads, dim, device="cuda").to(torch.bfloat16)
    gdn.kv8_append(x[:, :, :heads], x[:, :, heads:], codes[0], scales[0], table, torch.zeros_like(start))
    qkv = torch.randn(rows, 1, (group + 2) * heads, dim, device="cuda").to(torch.bfloat16)
    head = torch.randn(group * heads * dim, vocab, device="cuda").to(torch.bfloat16)
    said, cost = torch.randint(0, vocab, (2, beams, 12), **i32), torch.full((2, beams), 0.3, device="cuda")
    scores = torch.zeros(2, beams, device="cuda")

    def step():
        q = gdn.kv8_append_rotary(qkv[:, :, :4], qkv[:, :, 4:6], qkv[:, :, 6:], codes[0], scales[0], table, start, cos, sin)
        o = gdn.kv8_attention_shared(q, codes[0], scales[0], table, start + 1, shared, beams)
        logits = gdn.beam_logits((o.flatten(1) @ head).view(2, beams, vocab), said, None, None, cost)
        return (o, logits) + gdn.beam_select(logits, scores)

    before = codes.clone(), scales.clone()
    want = step()
    after = codes.clone(), scales.clone()
    codes.copy_(before[0]), scales.copy_(before[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        codes.copy_(before[0]), scales.copy_(before[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got + (codes, scales), want + after))
    qkv.neg_(), said.add_(7), start.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    eager = step()
    assert all(torch.equal(p, q) for p, q in zip(got, eager))


def test_shared_and_plain_attention_agree():
    model = ex.HybridModel(ex.Config(vocab=500, seed=6))
    prompts = torch.randint(2, 500, (2, 150), generator=torch.Generator().manual_seed(7)).cuda()
    out = []
    for on in (False, True):
        s = ex.start(model, 6, 200, 12)
        logits = ex.advance(model, s, prompts.repeat_interleave(3, 0))
        if on:
            ex.share(s, 2, 3, 144)
        out.append(ex.advance(model, s, logits.topk(3).indices[::3].reshape(6, 1)))
    a, b = (x.float() for x in out)
    # an attention layer and two layers behind it: a few bf16 roundings of the largest logit
    assert (a - b).abs().max() <= 8 * 2.0 ** -8 * a.abs().max()


def test_two_streams_at_once():
    """A step's three operators on two streams at once, each with rows of its own, as one after the other."""
    rows, beams, heads, group, dim, page, vocab = 8, 4, 2, 4, 128, 64, 40000
    todo = []
    for seed in (3, 4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape, t=torch.bfloat16: torch.randn(*shape, generator=g, device="cuda").to(t)
        kv = gdn.kv8_pool(1, rows * 40, heads, dim, page=page)
        table = torch.arange(rows * 40, device="cuda", dtype=torch.int32).view(rows, 40)
        at, shared = torch.full((rows,), 2300, dtype=torch.int32, device="cuda"), torch.full((rows // beams,), 2176, dtype=torch.int32, device="cuda")
        gdn.kv8_append(rand(rows, 2300, heads, dim), rand(rows, 2300, heads, dim), kv[0][0], kv[1][0], table, torch.zeros_like(at))
        angles = torch.rand(2400, dim // 2, generator=g, device="cuda")
        q, k, v = rand(rows, 1, heads * group, dim), rand(rows, 1, heads, dim), rand(rows, 1, heads, dim)
        logits, cost = rand(2, beams, vocab), torch.rand(2, beams, generator=g, device="cuda")
        said = torch.randint(0, vocab, (2, beams, 900), generator=g, device="cuda", dtype=torch.int32)

        def step(codes=kv[0][0], scales=kv[1][0], table=table, at=at, shared=shared, cos=angles.cos(), sin=angles.sin(),
                 q=q, k=k, v=v, logits=logits, said=said, cost=cost):
            turned = gdn.kv8_append_rotary(q, k, v, codes, scales, table, at, cos, sin)
            o, lse = gdn.kv8_attention_shared(turned, codes, scales, table, at + 1, shared, beams, need_lse=True)
            return turned, o, lse, gdn.beam_logits(logits, said, frequency=cost)
        todo.append((step, step()))
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in todo]
    got = [[] for _ in todo]
    for _ in range(10):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i].append(todo[i][0]())  # (the same tokens at the same places: nothing changes)
    torch.cuda.synchronize()
    for (_, want), many in zip(todo, got):
        for one in many:
            assert all(torch.equal(a, b) for a, b in zip(one, want))
    assert gdn.load().gdn_device_error(0) == 0

"""GPU: beam selection and the reordering of states, against the oracle.

Scores are fp32: the maximum is exact, the sum of exponentials is off by 2^-20 of itself at
most (expf to 2 ulp, partial sums of at most 2^10 terms), and the two additions round to
2^-24 of numbers up to the score's size.  Inputs are drawn so that no two candidates that
are not equal by construction lie nearer than that.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import GdnError, beam_reorder, beam_select
from oracle import serve as ref

pytestmark = pytest.mark.gpu


def _check(logits, scores, finished, k, eos):
    x = logits.float().cpu().numpy()
    fin = np.zeros(scores.shape, bool) if finished is None else finished.cpu().numpy()
    best, parents, tokens, done = ref.beam_select(x, scores.cpu().numpy(), fin, k, eos)
    got = beam_select(logits, scores, finished, k=k, eos=eos)
    g = got[0].cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(g), np.isneginf(best))
    ok = np.isfinite(best)
    assert np.all(np.abs(g[ok] - best[ok]) <= 2.0 ** -20 + 2.0 ** -22 * (np.abs(best[ok]) + 40))
    assert np.array_equal(got[1].cpu().numpy(), parents)
    assert np.array_equal(got[2].cpu().numpy(), tokens)
    assert np.array_equal(got[3].cpu().numpy(), done)
    assert all(torch.equal(a, b) for a, b in zip(got, beam_select(logits, scores, finished, k=k, eos=eos)))


CASES = [
    # batch, beams, vocab, k, dtype
    (1, 1, 1, 1, torch.float32), (1, 1, 3, 5, torch.float32), (2, 4, 7, 4, torch.bfloat16),
    (3, 5, 1001, 5, torch.float32), (1, 4, 32000, 4, torch.bfloat16), (2, 32, 5003, 32, torch.float32),
    (16, 8, 50257, 8, torch.bfloat16), (1, 2, 130001, 8, torch.float32), (4, 3, 4096, 1, torch.bfloat16),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_select(case):
    batch, beams, vocab, k, dtype = CASES[case]
    gen = torch.Generator("cuda").manual_seed(case)
    x = (3 * torch.randn(batch, beams, vocab, generator=gen, device="cuda")).to(dtype)
    scores = -10 * torch.rand(batch, beams, generator=gen, device="cuda")
    _check(x, scores, None, k, -1)
    fin = torch.rand(batch, beams, generator=gen, device="cuda") < 0.4
    eos = int(x[0, 0].float().argmax())
    _check(x, scores, fin, k, eos)
    scores[:, 1:] = float("-inf")                 # the first step: only beam 0 is real
    _check(x, scores, None, k, eos)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_and_masks(dtype):
    """Equal logits, masked tokens, beams with nothing left, and numbers that are none."""
    x = torch.zeros(3, 4, 3000, device="cuda", dtype=dtype)
    x[:, :, ::7] = 2.0
    x[1, 0] = float("-inf")
    x[1, 1, 5:] = float("-inf")
    x[1, 2, :] = float("nan")
    x[2, :, 11] = float("nan")
    x[2, 3, 1:] = float("-inf")
    scores = torch.tensor([[-1.0, -1.0, -1.0, -2.0]] * 3, device="cuda")
    for k in (4, 9):
        _check(x, scores, None, k, 0)
    y = torch.full((1, 2, 100), float("-inf"), device="cuda", dtype=dtype)
    _check(y, scores[:1, :2].contiguous(), None, 2, 3)
    y[0, 1, 50] = float("inf")                    # as the largest finite number: all of the mass
    best, parents, tokens, _ = beam_select(y, scores[:1, :2].contiguous(), k=1)
    assert float(best) == -1.0 and int(parents) == 1 and int(tokens) == 50


def test_strided_and_offset_rows():
    base = torch.randn(2, 3, 1003 + 5, device="cuda")
    scores = -torch.rand(2, 3, device="cuda")
    _check(base[..., 1:1004], scores, None, 3, -1)
    _check(base.to(torch.bfloat16)[..., 3:1006], scores, None, 3, 4)


@pytest.mark.parametrize("beams,rows", [(1, 3), (3, 12), (4, 10), (8, 64), (16, 16), (32, 40)])
def test_reorder(beams, rows):
    gen = torch.Generator().manual_seed(rows)
    shapes = [(rows, 3, 64, 64), (rows, 4), (rows, 1000)]
    types = [torch.float32, torch.float32, torch.int64]
    states = [torch.randn(s, generator=gen).mul(100).to(t).cuda() for s, t in zip(shapes, types)]
    r = torch.arange(rows)
    group = r // beams * beams
    parents = group + torch.randint(0, beams, (rows,), generator=gen)
    parents = torch.minimum(parents, torch.tensor(rows - 1))
    parents[torch.rand(rows, generator=gen) < 0.2] = -1
    parents[torch.rand(rows, generator=gen) < 0.2] = -5 if beams == 4 else -1
    want = [torch.where((parents >= 0).view(-1, *[1] * (s.dim() - 1)).cuda(), s[parents.clamp(min=0).cuda()], torch.zeros_like(s)) for s in states]
    p = parents.int().cuda()
    spare = [torch.empty_like(s) for s in states]
    out = beam_reorder(states, p, beams, out=spare)
    assert all(a is b for a, b in zip(out, spare)) and all(torch.equal(a, b) for a, b in zip(out, want))
    # in place: what is no row of the group, and not -1, leaves the row as it is
    keep = (parents < -1).cuda()
    want = [torch.where(keep.view(-1, *[1] * (s.dim() - 1)), s, w) for s, w in zip(states, want)]
    beam_reorder(states, p, beams)
    assert all(torch.equal(a, b) for a, b in zip(states, want))


def test_reorder_many_states_any_parents():
    states = [torch.randn(6, 40, device="cuda") for _ in range(150)]
    parents = torch.tensor([5, 0, 0, 2, 4, 1], dtype=torch.int32, device="cuda")
    out = beam_reorder(states, parents, 2, out=[torch.empty_like(s) for s in states])
    assert all(torch.equal(o, s[parents.long()]) for o, s in zip(out, states))
    assert beam_reorder([], parents, 2) == []


def test_refusals():
    x, s = torch.zeros(1, 2, 8, device="cuda"), torch.zeros(1, 2, device="cuda")
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    st = torch.zeros(4, 4, device="cuda")
    for bad, kind in [
        (lambda: beam_select(x.half(), s), GdnError), (lambda: beam_select(x, s, k=33), GdnError),
        (lambda: beam_select(x, s, k=0), GdnError), (lambda: beam_select(x, s, eos=8), GdnError),
        (lambda: beam_select(x, s[:, :1]), ValueError), (lambda: beam_select(x, s.double()), ValueError),
        (lambda: beam_select(x, s, s), ValueError), (lambda: beam_select(x[..., ::2], s), ValueError),
        (lambda: beam_select(x.cpu(), s), ValueError),
        (lambda: beam_select(x, s, workspace=torch.empty(8, dtype=torch.uint8, device="cuda")), GdnError),
        (lambda: beam_reorder([st], p[:3], 2), ValueError), (lambda: beam_reorder([st], p, 33), GdnError),
        (lambda: beam_reorder([st[:, :3].contiguous()], p, 2), GdnError),
        (lambda: beam_reorder([st], p, 2, out=[]), ValueError),
        (lambda: beam_reorder([torch.zeros(8, 4, device="cuda")[:4]], p, 2, out=[torch.zeros(4, 5, device="cuda")]), ValueError),
    ]:
        with pytest.raises(kind):
            bad()
    whole = torch.zeros(5, 4, device="cuda")
    with pytest.raises(GdnError):                 # overlapping, but not the same
        beam_reorder([whole[:4]], p, 2, out=[whole[1:]])

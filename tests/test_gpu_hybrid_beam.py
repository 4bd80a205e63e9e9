"""GPU: the hybrid beam search runs its parts together, and what it ends with is what each beam
would have reached by itself.

Every final beam's tokens are replayed in a session of the same shape in which no row ever
changes places: rows are independent of each other in every kernel, so the recurrent states
and the cached codes have to come out the same bit for bit, through all reorderings, shared
pages and copies; the scores agree to the rounding of a log-softmax per step (2^-19 of
numbers below 32, plus the rounding of the running score)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_beam_search as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode,batch,beams,n,steps", [("e4m3", 2, 4, 37, 20), ("int8", 1, 3, 64, 35), ("e4m3", 3, 1, 5, 4)])
def test_search_equals_replay(mode, batch, beams, n, steps):
    model = ex.HybridModel(ex.Config(vocab=200, mode=mode, seed=3))
    prompts = torch.randint(2, 200, (batch, n), generator=torch.Generator().manual_seed(5)).cuda()
    tokens, scores, s = ex.search(model, prompts, beams, steps, eos=-1)
    assert int(s.missing) == 0
    rows = batch * beams
    r = ex.start(model, rows, s.refs.numel(), s.table.shape[1])
    logits = ex.advance(model, r, prompts.repeat_interleave(beams, 0))
    total = torch.zeros(rows, dtype=torch.float64, device="cuda")
    for step in range(steps):
        t = tokens.view(rows, steps)[:, step].long()
        total += torch.log_softmax(logits.double(), -1).gather(1, t[:, None])[:, 0]
        if step + 1 < steps:
            logits = ex.advance(model, r, t[:, None])
    assert torch.all((total - scores.flatten()).abs() <= steps * (2.0 ** -19 * 32 + 2.0 ** -24 * scores.abs().max()))
    assert torch.equal(s.lengths, r.lengths)
    for a, b in zip(s.states, r.states):
        assert torch.equal(a, b)
    page = model.cfg.page
    for row in range(rows):
        have = int(r.lengths[row])
        for c in range(-(-have // page)):
            x, y, m = int(s.table[row, c]), int(r.table[row, c]), min(page, have - c * page)
            assert torch.equal(s.codes[:, :, x, :, :m], r.codes[:, :, y, :, :m])
            assert torch.equal(s.scales[:, :, x], r.scales[:, :, y])
    # every holder is counted, shared pages are full, and the live pages are the first ones
    used = torch.bincount(s.table[s.table >= 0].long(), minlength=s.refs.numel())
    assert torch.equal(used.int(), s.refs) and not s.refs[int((s.refs > 0).sum()):].any()


def test_finished_beams_stay():
    model = ex.HybridModel(ex.Config(vocab=60, seed=4))
    prompts = torch.randint(2, 60, (4, 20), generator=torch.Generator().manual_seed(6)).cuda()
    tokens, scores, s = ex.search(model, prompts, 3, 15, eos=7)
    assert int(s.missing) == 0
    ended = (tokens == 7).int().cumsum(-1) > 0
    assert torch.all(tokens[ended] == 7) and torch.all(torch.diff(scores, dim=1) <= 0)

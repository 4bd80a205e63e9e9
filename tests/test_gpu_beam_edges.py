"""GPU: corners of beam selection and of the reordering of states."""
import pytest
import torch

from gated_delta_rule_54_gb300 import GdnError, beam_reorder, beam_select

pytestmark = pytest.mark.gpu


def test_reorder_buffers_that_meet():
    """Buffers of different states may not meet where one is written; a source may serve twice."""
    a, b, c, d = (torch.randn(6, 40, device="cuda") for _ in range(4))
    before = [x.clone() for x in (a, b)]
    parents = torch.tensor([1, 0, 0, 2, 4, 3], dtype=torch.int32, device="cuda")
    for states, out in (([a, b], [b, a]), ([a, b], [c, c]), ([a, b], [a, a]), ([a, b], [c, a])):
        with pytest.raises(GdnError):
            beam_reorder(states, parents, 2, out=out)
    with pytest.raises(GdnError):
        beam_reorder([a, a], parents, 2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((a, b), before))
    beam_reorder([a, a], parents, 2, out=[c, d])
    want = a[parents.long()]
    assert torch.equal(c, want) and torch.equal(d, want)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_that_are_no_numbers(sign):
    """A beam whose score is NaN, of either sign, comes after all others."""
    x = torch.randn(2, 4, 300, device="cuda")
    nan = torch.tensor(float("nan"), device="cuda").copysign(torch.tensor(sign, device="cuda"))
    scores = torch.tensor([[-1.0, -2.0, -3.0, -4.0]] * 2, device="cuda")
    finished = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    finished[1, 2] = True
    low = scores.clone()
    scores[0, 1] = scores[1, 2] = nan
    low[0, 1] = low[1, 2] = float("-inf")
    for a, b in zip(beam_select(x, scores, finished, k=16, eos=5), beam_select(x, low, finished, k=16, eos=5)):
        assert torch.equal(a, b)

"""GPU: uses that the serving operators' documentation names, against plain restatements with every rounding."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import beam_logits, kv8_append_rotary, kv8_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("v", [999, 4096])
def test_repetition_over_the_prompt_as_well(v):
    """A call for it, then one for the penalties that see the answer only: bit for bit with fp32 logits."""
    rng = np.random.default_rng(v)
    rows, f32 = 4, np.float32
    x = (4 * rng.standard_normal((rows, v))).astype(f32)
    said = rng.integers(0, 300, (rows, 400)).astype(np.int32)          # a prompt of 320 and an answer of 80
    rep, freq, pres = (rng.uniform(0.3, 2, rows).astype(f32) for _ in range(3))
    bias = rng.standard_normal(v).astype(f32)
    want = x.copy()
    for r in range(rows):
        t = np.unique(said[r])
        y = want[r, t]
        want[r, t] = np.where(y > 0, (y / rep[r]).astype(f32), (y * rep[r]).astype(f32))
        t, n = np.unique(said[r, 320:], return_counts=True)
        want[r, t] = ((want[r, t] - (freq[r] * n.astype(f32)).astype(f32)).astype(f32) - pres[r]).astype(f32)
        want[r] = (want[r] + bias).astype(f32)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda().view(2, 2, *a.shape[1:])
    y = cuda(x)
    beam_logits(y, cuda(said), repetition=cuda(rep), out=y)
    y = beam_logits(y, cuda(said[:, 320:]), None, None, cuda(freq), cuda(pres), torch.from_numpy(bias).cuda())
    assert np.array_equal(y.cpu().numpy().reshape(rows, v), want)


@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("interleaved", [False, True])
def test_only_the_dims_that_turn_are_lost_without_angles(tokens, interleaved):
    torch.manual_seed(tokens)
    dim, half, page = 64, 16, 16
    q, k, v = (torch.randn(2, tokens, h, dim, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    cos, sin = torch.ones(40, half, device="cuda"), torch.zeros(40, half, device="cuda")
    codes, scales = kv8_pool(1, 12, 2, dim, page=page)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    start = torch.tensor([0, 50], dtype=torch.int32, device="cuda")     # row 1 is past the angles
    got = kv8_append_rotary(q, k, v, codes[0], scales[0], table, start, cos, sin, interleaved=interleaved)
    assert torch.equal(got[0], q[0])
    assert torch.isnan(got[1, ..., :2 * half]).all() and torch.equal(got[1, ..., 2 * half:], q[1, ..., 2 * half:])
    hit = table[1, 50 // page:(50 + tokens - 1) // page + 1].long()
    assert torch.isnan(scales[0, 0][hit]).all() and torch.isfinite(scales[0, 1]).all()
    assert torch.isfinite(scales[0, 0][table[0].long()]).all()

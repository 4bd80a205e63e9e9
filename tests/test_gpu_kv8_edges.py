"""GPU: corners of the 8-bit cache and of the attention over it, against the oracle.

Tolerances are those that test_gpu_kv8.py derives, with the terms that a test adds."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import kv8_attention, kv8_pool
from oracle import serve as ref
from test_gpu_kv8 import _check, _cuda, _pool, _table

pytestmark = pytest.mark.gpu


def _q(rng, rows, tokens, heads, dim, std=1.5):
    return torch.from_numpy(rng.standard_normal((rows, tokens, heads, dim)) * std).to(torch.bfloat16).cuda()


# ---- V blocks whose scales lie far apart ----------------------------------
@pytest.mark.parametrize("mode,dim,page", [("e4m3", 128, 16), ("int8", 64, 64), ("e4m3", 64, 32), ("int8", 128, 128)])
@pytest.mark.parametrize("tokens,group", [(1, 2), (8, 2), (40, 2), (200, 1)])
def test_v_scales_far_apart(mode, dim, page, tokens, group):
    """Blocks 2^130 apart, in either order, and seen by some rows of a tile only."""
    rng = np.random.default_rng(31)
    lengths, heads = [200, 333, 390], 2
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table = _table(rng, lengths, page, pages)
    for r, n in enumerate(lengths):
        for c in range(-(-n // page)):
            scales[1, table[r, c]] *= np.float32(2.0) ** ((-65, 65, 0)[(c + r) % 3])
    q = _q(rng, 3, tokens, heads * group, dim)
    got = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), mode=mode, need_lse=True)
    _check(got, q.float().cpu().numpy(), codes, scales, table, lengths, mode, dim ** -0.5)


@pytest.mark.parametrize("tokens", [1, 40])
@pytest.mark.parametrize("mode,dim,page", [("e4m3", 128, 64), ("int8", 64, 16)])
def test_codes_under_a_scale_of_zero(mode, dim, page, tokens):
    """value = code * scale: under a scale of 0 any codes are zeros, in K and in V."""
    rng = np.random.default_rng(32)
    lengths = [300, 130]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, 1, page, dim, mode)
    table = _table(rng, lengths, page, pages)
    scales[1, table[0, 1]] = scales[0, table[0, 0]] = 0
    scales[1, table[1, :-(-130 // page)]] = 0              # row 1: all of V
    q = _q(rng, 2, tokens, 2, dim)
    got = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), mode=mode, need_lse=True)
    _check(got, q.float().cpu().numpy(), codes, scales, table, lengths, mode, dim ** -0.5)
    assert torch.all(got[0][1] == 0)


# ---- what follows a call in the stream sees its outputs -------------------
def test_next_kernel_sees_rows_without_keys():
    """No row has a key, so nothing is left to join: a copy right behind the call has the zeros."""
    rows, heads = 3000, 8
    codes, scales = kv8_pool(1, 4, heads, 128, page=16)
    table = torch.full((rows, 64), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(rows, dtype=torch.int32, device="cuda")
    q = torch.randn(rows, 2, heads * 8, 128, device="cuda").to(torch.bfloat16)
    out, seen = torch.empty_like(q), torch.empty_like(q)
    for _ in range(20):
        out.fill_(7.0)
        kv8_attention(q, codes[0], scales[0], table, lengths, out=out)
        seen.copy_(out)
        assert int(torch.count_nonzero(seen)) == 0

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


# ---- q with one channel far above the others ------------------------------
@pytest.mark.parametrize("mode", ["e4m3", "int8"])
@pytest.mark.parametrize("dim,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("tokens,group", [(1, 4), (4, 4), (20, 1), (150, 2)])
def test_q_with_a_large_channel(mode, dim, page, tokens, group):
    """A channel of q 2^10 to 2^14 times the others, where K is nothing or the same for all keys.

    q of an E4M3 cache is the sum of an E4M3 and an E5M2 number (or two E4M3 numbers): with
    the row's largest in [2^7, 2^8) the first is off by 2^-4 of an element's binade, which
    leaves at most three bits, down to elements of 2^-6; below, the first is off by at most
    2^-10 and three bits of that leave 2^-14: 2^-21 of the row's largest for elements below
    2^-13 of it.  INT8 caches take q in fp16, exact here."""
    rng = np.random.default_rng(33)
    lengths = [1, 2, 5, 40, 300]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, 1, page, dim, mode)
    codes[0, ..., 5] = 0
    codes[0, ..., 9] = 0x78 if mode == "e4m3" else 90      # 256 or 90 of the scale
    scales[0] = scales[0, 0]                               # the channel is the same for all keys
    table = _table(rng, lengths, page, pages)
    args = _cuda(codes, scales, table, np.array(lengths, np.int32))
    for channel in (5, 9):
        for e in (10, 12, 14):
            q = _q(rng, len(lengths), tokens, group, dim)
            q[..., channel] *= 2.0 ** e
            o, lse = (x.float().cpu().numpy().astype(np.float64) for x in kv8_attention(q, *args, mode=mode, need_lse=True))
            x = q.float().cpu().numpy().astype(np.float64)
            for r, n in enumerate(lengths):
                ro, rl, absum, top, dots = ref.attention(x[r], codes, scales, table[r], n, mode, dim ** -0.5)
                score = 2.0 ** -20 * (dots + 1)
                if mode == "e4m3":
                    keys = codes[0][table[r, :-(-n // page)], 0].reshape(-1, dim)[:n]
                    k = np.abs(ref.decode_codes(keys, mode)) * float(scales[0, 0, 0])
                    most = np.abs(x[r]).max(-1, keepdims=True)
                    small = np.abs(x[r]) < 2.0 ** -13 * most
                    score = score + dim ** -0.5 * 2.0 ** -21 * most[..., 0] * (small @ k.T).max(-1)
                seen = np.isfinite(rl)
                assert np.all(np.abs(lse[r][seen] - rl[seen]) <= 2.0 ** -16 + score[seen]), (channel, e, r)
                tol = (1.01 * 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -15 + 2 * np.expm1(score)[..., None]) * absum
                       + 2.0 ** -25 * n * top[..., None] + 1e-37)
                assert np.all(np.abs(o[r] - ro) <= tol), (channel, e, r)

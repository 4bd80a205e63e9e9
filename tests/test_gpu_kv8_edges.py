"""GPU: corners of the 8-bit cache and of the attention over it, against the oracle.

Tolerances are those that test_gpu_kv8.py derives, with the terms that a test adds."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import GdnError, kv8_append, kv8_attention, kv8_pool, kv8_reserve, load
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


@pytest.mark.parametrize("tokens,group", [(1, 4), (8, 2), (40, 2)])
@pytest.mark.parametrize("mode,dim,page", [("e4m3", 128, 64), ("int8", 64, 16), ("int8", 128, 128)])
@pytest.mark.parametrize("power", [-127.5, -120, 110])
def test_v_scales_of_any_size(mode, dim, page, tokens, group, power):
    """V near the ends of its range: scales from 2^-128, the smallest that append writes."""
    rng = np.random.default_rng(35)
    lengths = [1, 60, 150]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, 1, page, dim, mode)
    scales[1] = np.float32(2.0 ** power)
    table = _table(rng, lengths, page, pages)
    q = _q(rng, 3, tokens, group, dim)
    got = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), mode=mode, need_lse=True)
    _check(got, q.float().cpu().numpy(), codes, scales, table, lengths, mode, dim ** -0.5)


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


@pytest.mark.parametrize("mode,dim,page", [("e4m3", 128, 64), ("int8", 64, 16), ("e4m3", 64, 32)])
@pytest.mark.parametrize("tokens,group", [(1, 4), (4, 4), (40, 2)])
@pytest.mark.parametrize("up", [122, 118, -104, -112])
def test_q_of_any_size(mode, dim, page, tokens, group, up):
    """Queries near the ends of their type's range against K that brings the scores back."""
    rng = np.random.default_rng(34)
    lengths = [3, 100, 333]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, 1, page, dim, mode)
    scales[0] *= np.float32(2.0) ** -(up - (4 if up > 0 else 0))
    table = _table(rng, lengths, page, pages)
    q = (_q(rng, 3, tokens, group, dim).float() * 2.0 ** up).to(torch.bfloat16)
    got = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), mode=mode, need_lse=True)
    _check(got, q.float().cpu().numpy(), codes, scales, table, lengths, mode, dim ** -0.5)


# ---- numbers that are none ------------------------------------------------
def _positions(length, tokens, window):
    """[tokens, length]: which key each query sees."""
    pos = length - tokens + np.arange(tokens)[:, None]
    j = np.arange(length)[None]
    return (j <= pos) & ((j > pos - window) if window else True)


BAD = [
    # lengths, tokens, heads, group, dim, page, mode, window
    ([100, 64, 130], 1, 2, 2, 128, 64, "e4m3", 0),
    ([100, 64, 130], 1, 2, 2, 64, 16, "int8", 40),
    ([150, 70], 6, 2, 2, 128, 16, "e4m3", 30),
    ([150, 70], 6, 2, 2, 64, 32, "int8", 0),
    ([9000, 6000], 1, 2, 4, 128, 64, "int8", 0),      # a line of tiles: parts are joined
    ([9000, 6000], 1, 2, 16, 64, 128, "e4m3", 3000),
    ([200, 130], 130, 2, 1, 128, 16, "e4m3", 0),
    ([200, 130], 130, 2, 1, 64, 64, "int8", 50),
    ([3000, 2500], 20, 2, 2, 128, 128, "int8", 0),    # few blocks: the keys are split
    ([3000, 2500], 20, 2, 2, 64, 32, "e4m3", 700),
]


@pytest.mark.parametrize("case", range(len(BAD)))
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_blocks_that_are_no_numbers(case, what):
    """A query that sees a key of a block whose K or V scale is not finite gets NaN; nobody else does."""
    lengths, tokens, heads, group, dim, page, mode, window = BAD[case]
    rng = np.random.default_rng(40 + case)
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table = _table(rng, lengths, page, pages)
    poisoned, hit = scales.copy(), []
    for r, n in enumerate(lengths):                    # a block near the end of head r % heads
        c = max(0, -(-n // page) - 2)
        poisoned[(r + case) % 2, table[r, c], r % heads] = what
        hit.append((c * page, (c + 1) * page))
    q = _q(rng, len(lengths), tokens, heads * group, dim)
    args = dict(mode=mode, window=window, need_lse=True)
    o, lse = kv8_attention(q, *_cuda(codes, poisoned, table, np.array(lengths, np.int32)), **args)
    clean = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), **args)
    for r, n in enumerate(lengths):
        sees = torch.from_numpy(_positions(n, tokens, window)[:, hit[r][0]:hit[r][1]].any(1)).cuda()
        of = slice(r % heads * group, (r % heads + 1) * group)
        for x, y in zip((o[r], lse[r]), (clean[0][r], clean[1][r])):
            assert torch.all(torch.isnan(x[sees][:, of]))
            y = y.clone()
            bad = torch.zeros_like(y, dtype=torch.bool)
            bad[:, of] = sees.view(-1, 1, *[1] * (y.dim() - 2))
            assert torch.allclose(x[~bad].float(), y[~bad].float(), rtol=2.0 ** -7, atol=1e-3)
            assert not torch.any(torch.isnan(x[~bad]))
    assert load().gdn_device_error(0) == 0


@pytest.mark.parametrize("case", range(len(BAD)))
def test_queries_that_are_no_numbers(case):
    lengths, tokens, heads, group, dim, page, mode, window = BAD[case]
    rng = np.random.default_rng(60 + case)
    lengths = lengths + [0]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table = _table(rng, lengths, page, pages)
    q = _q(rng, len(lengths), tokens, heads * group, dim)
    args = (*_cuda(codes, scales, table, np.array(lengths, np.int32)),)
    clean = kv8_attention(q, *args, mode=mode, window=window, need_lse=True)
    bad = torch.zeros(q.shape[:-1], dtype=torch.bool, device="cuda")
    for r in range(len(lengths)):
        for i, what in enumerate((float("nan"), float("inf"), float("-inf"))):
            t, h = (7 * r + 3 * i) % tokens, (r + i) % (heads * group)
            q[r, t, h, (11 * r + i) % dim] = what
            bad[r, t, h] = True
    o, lse = kv8_attention(q, *args, mode=mode, window=window, need_lse=True)
    none = torch.isneginf(clean[1])
    assert torch.all(torch.isnan(o[bad & ~none])) and torch.all(torch.isnan(lse[bad & ~none]))
    assert torch.all(o[none] == 0) and torch.all(torch.isneginf(lse[none]))
    assert torch.equal(o[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("mode", ["e4m3", "int8"])
@pytest.mark.parametrize("tokens", [1, 50])
def test_append_of_what_is_no_number(mode, tokens):
    """A NaN among a block's tokens makes its scale NaN, an infinity makes it infinite, for good; other blocks are
    as ever."""
    rng = np.random.default_rng(70)
    heads, dim, page, rows = 3, 64, 16, 2
    codes, scales = np.zeros((2, 16, heads, page, dim), np.uint8), np.zeros((2, 16, heads), np.float32)
    table = np.arange(16, dtype=np.int32).reshape(2, 8)
    c, s, t = _cuda(codes, scales, table)
    bad = np.zeros(scales.shape, bool)
    for step in range(3):
        x = rng.standard_normal((2, rows, tokens, heads, dim)).astype(np.float32)
        x = torch.from_numpy(x).to(torch.bfloat16)
        clean = x.float().numpy()
        if step == 1:                                  # position 3 or so of the first, or a whole block
            x[0, 0, 0, 1, 7], x[1, 1, tokens // 2, 2, 0], x[0, 1, 0, 0, 3] = float("nan"), float("inf"), float("-inf")
        start = np.full(rows, step * tokens, np.int32)
        kv8_append(x[0].cuda(), x[1].cuda(), c, s, t, _cuda(start)[0], mode=mode)
        ref.append(clean[0], clean[1], codes, scales, table, start, [tokens] * rows, mode)
        if step == 0:
            continue
        got = s.cpu().numpy()
        b0, b1 = (tokens * 1) // page, (tokens + tokens // 2) // page
        want = {(0, table[0, b0], 1): np.nan, (1, table[1, b1], 2): np.inf, (0, table[1, b0], 0): np.inf}
        for at, v in want.items():
            assert np.isnan(got[at]) if np.isnan(v) else got[at] == v
            bad[at] = True
        assert np.array_equal(got[~bad], scales[~bad])
        assert np.array_equal(c.cpu().numpy()[~bad], codes[~bad])
    n = np.full(rows, 3 * tokens, np.int32)
    q = _q(rng, rows, 1, heads, dim)
    o, lse = kv8_attention(q, c, s, t, _cuda(n)[0], mode=mode, need_lse=True)
    lost = torch.tensor([[False, True, False], [True, False, True]], device="cuda")
    assert torch.equal(torch.isnan(lse[:, 0]), lost) and torch.equal(torch.isnan(o[:, 0]).all(-1), lost)


# ---- packed calls: tokens of no row, and rows above the bound -------------
@pytest.mark.parametrize("most,group", [(3, 2), (60, 2)])
def test_packed_tokens_of_no_row(most, group):
    rng = np.random.default_rng(80)
    heads, dim, page, mode = 2, 64, 16, "e4m3"
    counts, lengths = [most, 0, 1, most], [90, 20, 0, 75]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table = _table(rng, lengths, page, pages)
    starts = 5 + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total = int(starts[-1]) + 40
    q = torch.from_numpy(rng.standard_normal((total, heads * group, dim))).to(torch.bfloat16).cuda()
    out = torch.full_like(q, 7.0)
    filler = torch.full((total, heads * group), 9.0, device="cuda")
    del filler                                         # (the next tensor of this size finds the 9s)
    o, lse = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), mode=mode, need_lse=True, out=out,
                           cu_seqlens=torch.from_numpy(starts).cuda(), max_seqlen=most)
    _check((o, lse), q.float().cpu().numpy(), codes, scales, table, lengths, mode, dim ** -0.5, starts)
    for part in (slice(0, 5), slice(int(starts[-1]), total)):
        assert torch.all(o[part] == 0) and torch.all(torch.isneginf(lse[part]))


@pytest.mark.parametrize("most,group", [(3, 2), (60, 2)])
def test_packed_rows_above_the_bound(most, group):
    """max_seqlen is a promise; a row that breaks it gets NaN, not an uninitialised rest."""
    rng = np.random.default_rng(81)
    heads, dim, page, mode = 2, 64, 16, "int8"
    counts, lengths = [most, most + 2, 1], [90, 100, 30]
    pages = sum(-(-n // page) for n in lengths)
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table = _table(rng, lengths, page, pages)
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(starts[-1]), heads * group, dim))).to(torch.bfloat16).cuda()
    out = torch.full_like(q, 7.0)
    o, lse = kv8_attention(q, *_cuda(codes, scales, table, np.array(lengths, np.int32)), mode=mode, need_lse=True, out=out,
                           cu_seqlens=torch.from_numpy(starts).cuda(), max_seqlen=most)
    over = slice(int(starts[1]), int(starts[2]))
    assert torch.all(torch.isnan(o[over])) and torch.all(torch.isnan(lse[over]))
    for r in (0, 2):
        sl = slice(int(starts[r]), int(starts[r + 1]))
        _check((o[sl], lse[sl]), q[sl].float().cpu().numpy(), codes, scales, table[r:r + 1], [lengths[r]], mode, dim ** -0.5,
               np.array([0, counts[r]]))


@pytest.mark.parametrize("most,length", [(0, 40), (0, 40000), (-1, 40)])
def test_packed_bounds_without_a_token(most, length):
    """A bound of 0 leaves rows with tokens above it; below 0 it is none."""
    codes, scales = kv8_pool(1, 4, 1, 64, page=16)
    table = torch.zeros(2, -(-length // 16), dtype=torch.int32, device="cuda")
    lengths = torch.full((2,), length, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 3], dtype=torch.int32, device="cuda")
    q = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda: kv8_attention(q, codes[0], scales[0], table, lengths, cu_seqlens=cu, max_seqlen=most, need_lse=True)
    if most < 0:
        with pytest.raises(GdnError):
            call()
        return
    o, lse = call()
    assert torch.all(torch.isnan(o[:3])) and torch.all(torch.isnan(lse[:3]))
    assert torch.all(o[3:] == 0) and torch.all(torch.isneginf(lse[3:]))


# ---- pages ----------------------------------------------------------------
def test_reserve_counts_all_that_is_missing():
    """Rows that want more pages than any pool has are counted in full."""
    codes, scales = kv8_pool(1, 6, 1, 64, page=16)
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    lengths, refs = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    extra = torch.tensor([1 << 30, 16, 1 << 30], dtype=torch.int32, device="cuda")
    t, n, r, missing = kv8_reserve(codes, scales, table, lengths, extra, refs)
    assert t.tolist() == [[0, 1, 2, 3], [4, -1, -1, -1], [5, -1, -1, -1]] and n.tolist() == [64, 16, 64]
    assert int(missing) == 2 * (1 << 26) + 1 - 6

"""GPU: the 8-bit paged cache and the attention over it, against the oracle.

Tolerances.  Codes, scales and tables are bit-exact.  An output of the attention may be off
by the rounding to bf16 (8 significant bits: 2^-8 of itself), by the fp16 rounding of the probabilities (2^-11 of
the sum of p |v|; below fp16's normal range 2^-25 of the largest p * V scale per key), by the
fp32 sums of the products (2^-15 of the sum of p |v| for up to 4096 keys in steps of 16), and
by the scores' own error, 2^-20 of the largest sum of |q k| (eight fp32 steps) plus 2^-20 for
the exponential, which moves every weight by that much relative to the others (twice).  The
log-sum-exp is off by the scores' error plus 2^-16 for its sum.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import kv8_append, kv8_attention, kv8_pool, load
from oracle import serve as ref

pytestmark = pytest.mark.gpu


def _pool(rng, pages, heads, page, dim, mode):
    """A layer's cache of random tokens, blocks of unlike size."""
    x = rng.standard_normal((2, pages, heads, page, dim)) * np.exp(0.5 * rng.standard_normal((2, pages, heads, 1, 1)))
    s = (np.abs(x).max((3, 4)) / ref.CODE_MAX[mode]).astype(np.float32)
    return ref.encode((x / s[..., None, None]).astype(np.float32), mode), s


def _table(rng, lengths, page, pages, cols=None):
    used = [-(-n // page) for n in lengths]
    cols = max(used + [1]) if cols is None else cols
    ids, t = rng.permutation(pages), np.full((len(lengths), cols), -1, np.int32)
    at = 0
    for r, n in enumerate(used):
        t[r, :n] = ids[at:at + n]
        at += n
    return t


def _cuda(*xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _check(got, q, codes, scales, table, lengths, mode, scale, starts=None, **kw):
    """got = (o, lse), rows of queries split by ``starts`` (packed) or along dim 0."""
    o, lse = (x.float().cpu().numpy().astype(np.float64) for x in got)
    for r, n in enumerate(lengths):
        sl = slice(starts[r], starts[r + 1]) if starts is not None else r
        ro, rl, absum, top, dots = ref.attention(q[sl].astype(np.float64), codes, scales, table[r], int(n), mode, scale, **kw)
        seen = np.isfinite(rl)
        assert np.array_equal(np.isneginf(lse[sl]), ~seen)
        assert np.all(o[sl][~seen] == 0)
        score = 2.0 ** -20 * (dots + 1)
        tol = (1.01 * 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -15 + 2 * score[..., None]) * absum
               + 2.0 ** -25 * max(int(n), 1) * top[..., None] + 1e-37)
        err = np.abs(o[sl] - ro)
        assert np.all(err <= tol), "row %d: %.3g over %.3g" % (r, err.max(), (tol[err > tol]).min())
        d = np.abs(lse[sl][seen] - rl[seen])
        assert np.all(d <= 2.0 ** -16 + score[seen]), "row %d: lse off by %.3g" % (r, d.max())


def _run(rng, lengths, tokens, heads, group, dim, page, mode, packed=False, holes=(), causal=True,
         window=0, scale=None, qstd=1.5, spoil=None, cols=None):
    lens = np.array(lengths, np.int32)
    pages = int(sum(-(-n // page) for n in lengths)) + 3
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table = _table(rng, lengths, page, pages, cols)
    if spoil:
        spoil(codes, scales, table)
    for r, n in enumerate(lengths):  # slots past a row's end hold bytes that are no numbers
        if n % page and table.shape[1] > n // page:
            codes[:, table[r, n // page], :, n % page:] = 0x7f if mode == "e4m3" else 0x80
    for r, c in holes:
        table[r, c] = (-1, pages, -7, 1 << 30)[c % 4]
    counts = tokens if packed else [tokens] * len(lengths)
    total, hq = int(sum(counts)), heads * group
    # q is part of a wider tensor, as a projection writes it
    wide = torch.from_numpy(rng.standard_normal((total, hq + 2, dim)) * qstd).to(torch.bfloat16).cuda()
    q = wide[:, 1:1 + hq]
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    args = dict(mode=mode, causal=causal, window=window, need_lse=True, scale=scale)
    if packed:
        args.update(cu_seqlens=torch.from_numpy(starts).cuda(), max_seqlen=max(counts))
    else:
        q = q.unflatten(0, (len(lengths), tokens))
    c, s, t, n = _cuda(codes, scales, table, lens)
    got = kv8_attention(q, c, s, t, n, **args)
    again = kv8_attention(q, c, s, t, n, **args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert load().gdn_device_error(0) == 0
    _check(got, q.float().cpu().numpy(), codes, scales, table, lengths, mode, dim ** -0.5 if scale is None else scale,
           starts if packed else None, causal=causal, window=window)
    return got


DECODE = [
    # lengths, tokens, heads, group, dim, page, mode, window
    ([1], 1, 1, 1, 128, 64, "e4m3", 0),
    ([0, 1, 2, 0], 1, 2, 4, 64, 16, "int8", 0),
    ([700], 1, 2, 8, 128, 64, "e4m3", 0),
    ([31, 32, 33, 63, 64, 65, 127, 128, 129], 1, 2, 2, 128, 32, "e4m3", 0),
    ([31, 32, 33, 63, 64, 65, 127, 128, 129], 1, 2, 3, 64, 16, "int8", 0),
    ([3000, 17, 0, 5001], 1, 3, 5, 128, 128, "int8", 0),
    ([2500, 4097], 1, 1, 16, 64, 64, "e4m3", 0),
    ([9000, 1, 2047, 640, 0, 3, 77], 1, 8, 1, 128, 64, "e4m3", 0),
    ([5000, 3, 900], 5, 2, 3, 64, 16, "int8", 100),
    ([2900, 16, 8], 8, 2, 2, 128, 16, "e4m3", 33),
    ([4, 2, 0, 9], 4, 2, 4, 128, 32, "e4m3", 0),        # fewer tokens than queries
]


@pytest.mark.parametrize("case", range(len(DECODE)))
def test_few_rows(case):
    lengths, tokens, heads, group, dim, page, mode, window = DECODE[case]
    _run(np.random.default_rng(case), lengths, tokens, heads, group, dim, page, mode, window=window)


@pytest.mark.parametrize("rows,heads,most,page,dim,mode", [
    (16, 8, 2000, 64, 128, "e4m3"),    # a CTA per (row, head), long
    (45, 5, 1200, 32, 64, "int8"),     # two waves of them
    (45, 5, 1300, 32, 64, "int8"),     # one column more
    (48, 8, 90, 16, 128, "e4m3"),      # many short ones: a warp's share has several
    (200, 16, 40, 16, 64, "int8"),
    (330, 1, 1, 16, 128, "int8"),
])
def test_many_short_rows(rows, heads, most, page, dim, mode):
    rng = np.random.default_rng(rows + most)
    lengths = rng.integers(0, most + 1, rows)
    lengths[rng.integers(rows)] = most
    for group, tokens in ((2, 1), (3, 4)):
        _run(rng, [int(n) for n in lengths], tokens, heads, group, dim, page, mode)


@pytest.mark.parametrize("rows", [3, 200, 400])
@pytest.mark.parametrize("cols", [0, 2])
def test_rows_without_keys(rows, cols):
    """Nothing in the cache for any row, and tables without columns."""
    codes, scales = kv8_pool(1, 4, 1, 64, page=16)
    table = torch.full((rows, cols), -1, dtype=torch.int32, device="cuda")
    q = torch.randn(rows, 2, 2, 64, device="cuda").to(torch.bfloat16)
    for n in (0, 5):
        lengths = torch.full((rows,), n, dtype=torch.int32, device="cuda")
        o, lse = kv8_attention(q, codes[0], scales[0], table, lengths, need_lse=True)
        assert torch.all(o == 0)
        assert torch.all(torch.isneginf(lse))
    assert load().gdn_device_error(0) == 0


MANY = [
    # lengths, tokens, heads, group, dim, page, mode, window, packed
    ([17], 17, 1, 1, 128, 64, "e4m3", 0, False),
    ([300, 40], 40, 2, 4, 128, 64, "e4m3", 0, False),
    ([257], 257, 1, 1, 64, 16, "int8", 0, False),
    ([700, 130, 0, 33], [300, 130, 5, 40], 2, 2, 128, 32, "int8", 0, True),
    ([500, 90, 1000], [129, 1, 200], 1, 3, 64, 64, "e4m3", 70, True),
    ([1500, 1200], 20, 2, 5, 128, 16, "e4m3", 0, False),     # few blocks: the keys are split
    ([3000], 8, 1, 16, 64, 128, "int8", 500, False),
    ([60, 3], 64, 2, 1, 128, 128, "e4m3", 0, False),         # fewer tokens than queries
    ([640], 128, 1, 2, 128, 64, "int8", 1, False),           # each query sees itself only
]


@pytest.mark.parametrize("case", range(len(MANY)))
def test_many_rows(case):
    lengths, tokens, heads, group, dim, page, mode, window, packed = MANY[case]
    _run(np.random.default_rng(100 + case), lengths, tokens, heads, group, dim, page, mode, packed=packed, window=window)


@pytest.mark.parametrize("tokens,group", [(1, 4), (40, 2)])
def test_not_causal_and_holes_and_scales_of_zero(tokens, group):
    def spoil(codes, scales, table):
        # a block of zeros in V, one in K, and V blocks 2^30 apart in scale
        scales[1, table[0, 1]], codes[1, table[0, 1]] = 0, 0
        scales[0, table[0, 2]], codes[0, table[0, 2]] = 0, 0
        scales[1, table[1, 0]] *= 2.0 ** 20
        scales[1, table[1, 2]] *= 2.0 ** -10
    rng = np.random.default_rng(7)
    _run(rng, [400, 333, 250], tokens, 2, group, 128, 64, "e4m3", causal=False, holes=[(0, 3), (2, 0), (2, 2)], spoil=spoil)
    _run(rng, [400, 333, 250], tokens, 2, group, 64, 32, "int8", holes=[(0, 0), (1, 4), (2, 1)], spoil=spoil)


@pytest.mark.parametrize("tokens", [1, 33])
def test_every_page_missing_and_negative_scale(tokens):
    rng = np.random.default_rng(8)
    o, lse = _run(rng, [100, 64], tokens, 1, 2, 64, 64, "e4m3", holes=[(0, 0), (0, 1)])
    assert torch.all(o[0] == 0) and torch.all(torch.isneginf(lse[0]))
    _run(rng, [200, 90], tokens, 1, 2, 128, 32, "int8", scale=-0.05)
    _run(rng, [200, 90], tokens, 1, 2, 128, 32, "e4m3", scale=2.0)      # sharp: one key takes all


@pytest.mark.parametrize("tokens", [1, 70])
def test_table_narrower_than_the_row(tokens):
    """Keys past the table's columns do not exist; the positions still count them."""
    _run(np.random.default_rng(9), [500, 100], tokens, 2, 2, 128, 64, "e4m3", cols=8)
    rng = np.random.default_rng(10)
    codes, scales = _pool(rng, 6, 1, 16, 64, "int8")
    table = np.array([[3, 1]], np.int32)
    q = torch.randn(1, tokens, 1, 64, device="cuda").to(torch.bfloat16)
    got = kv8_attention(q, *_cuda(codes, scales, table, np.array([100], np.int32)), mode="int8", need_lse=True)
    _check(got, q.float().cpu().numpy(), codes, scales, table, [100], "int8", 64 ** -0.5)


def test_cache_past_32_bits():
    """Pages whose bytes lie past 2^32 in the cache, read and written."""
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 40
    codes = torch.empty(2, pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    scales = torch.empty(2, pages, heads, device="cuda")
    rng = np.random.default_rng(11)
    ids = [pages - 1, 5, pages - 17]
    small_codes, small_scales = _pool(rng, 3, heads, page, dim, "e4m3")
    small_table = np.array([[0, 1, 2]], np.int32)
    for i, p in enumerate(ids):
        codes[:, p], scales[:, p] = _cuda(small_codes[:, i], small_scales[:, i])
    table, start = _cuda(np.array([ids], np.int32), np.array([300], np.int32))
    k, v = (torch.randn(1, 30, heads, dim, device="cuda").to(torch.bfloat16) for _ in range(2))
    kv8_append(k, v, codes, scales, table, start)
    ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), small_codes, small_scales, small_table, [300], [30], "e4m3")
    for i, p in enumerate(ids):
        assert np.array_equal(codes[:, p].cpu().numpy(), small_codes[:, i])
        assert np.array_equal(scales[:, p].cpu().numpy(), small_scales[:, i])
    for t in (1, 30):
        q = torch.randn(1, t, heads * 2, dim, device="cuda").to(torch.bfloat16)
        got = kv8_attention(q, codes, scales, table, start + 30, need_lse=True)
        _check(got, q.float().cpu().numpy(), small_codes, small_scales, small_table, [330], "e4m3", dim ** -0.5)


APPEND = [
    # starts, counts (a list: packed), heads, dim, page, mode
    ([0, 5, 16, 31, 0], 1, 2, 128, 16, "e4m3"),
    ([63, 64, 65, 0], 1, 1, 64, 64, "int8"),
    ([0, 100, 7], [300, 1, 64], 2, 128, 32, "int8"),
    ([3, 0, 0, 250], [0, 129, 1, 270], 3, 64, 128, "e4m3"),
    ([10, 0], 7, 2, 128, 128, "e4m3"),
    ([1, 33], 40, 1, 128, 16, "int8"),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
def test_append_bit_exact(case):
    starts, counts, heads, dim, page, mode = APPEND[case]
    rng = np.random.default_rng(200 + case)
    packed = isinstance(counts, list)
    n = counts if packed else [counts] * len(starts)
    lengths = [a + b for a, b in zip(starts, n)]
    pages = sum(-(-x // page) for x in lengths) + 2
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    scales *= rng.choice([0.3, 1.0, 3.0], scales.shape).astype(np.float32)  # some blocks have to grow
    table = _table(rng, lengths, page, pages)
    wide = torch.from_numpy(rng.standard_normal((sum(n), 3 * heads, dim))).to(torch.bfloat16).cuda()
    wide[:, :, 0] *= 20
    wide[0] = 0                                                      # a token of zeros
    k, v = wide[:, heads:2 * heads], wide[:, 2 * heads:]
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    rows = [x.float().cpu().numpy() for x in (k, v)]
    rows = [[x[cu[r]:cu[r + 1]] for r in range(len(n))] for x in rows]
    if not packed:
        k, v = (x.unflatten(0, (len(starts), counts)) for x in (k, v))
    c, s, t, st = _cuda(codes, scales, table, np.array(starts, np.int32))
    for _ in range(2):  # the same call again changes nothing more
        kv8_append(k, v, c, s, t, st, cu_seqlens=_cuda(cu)[0] if packed else None, max_seqlen=max(n) if packed else None, mode=mode)
        if _ == 0:
            ref.append(*rows, codes, scales, table, starts, n, mode)
        assert np.array_equal(s.cpu().numpy().view(np.uint32), scales.view(np.uint32))
        assert np.array_equal(c.cpu().numpy(), codes)


@pytest.mark.parametrize("mode", ["e4m3", "int8"])
def test_append_token_by_token_skips_what_is_no_page(mode):
    rng = np.random.default_rng(5)
    heads, dim, page = 2, 64, 16
    codes, scales = np.zeros((2, 6, heads, page, dim), np.uint8), np.zeros((2, 6, heads), np.float32)
    table = np.array([[4, 0, 2], [1, -1, 5], [9, 3, 6]], np.int32)
    c, s, t = _cuda(codes, scales, table)
    for i in range(50):                      # past the table's last column too
        x = (rng.standard_normal((2, 3, 1, heads, dim)) * (0.0 if i == 0 else 2.0 ** (i % 7))).astype(np.float32)
        k, v = (torch.from_numpy(a).to(torch.bfloat16).cuda() for a in x)
        kv8_append(k, v, c, s, t, _cuda(np.full(3, i, np.int32))[0], mode=mode)
        ref.append(k.float().cpu().numpy(), v.float().cpu().numpy(), codes, scales, table, [i] * 3, [1] * 3, mode)
        assert np.array_equal(c.cpu().numpy(), codes) and np.array_equal(s.cpu().numpy(), scales), i


def test_other_stream_and_graph():
    """Work goes to the current stream, and a captured call replays on new contents."""
    rng = np.random.default_rng(3)
    codes, scales = _pool(rng, 8, 2, 64, 128, "e4m3")
    table = np.array([[3, 1, 0], [5, 7, 2]], np.int32)
    c, s, t, n = _cuda(codes, scales, table, np.array([180, 70], np.int32))
    side = torch.cuda.Stream()
    for tokens in (1, 20):
        q = torch.randn(2, tokens, 4, 128, device="cuda").to(torch.bfloat16)
        want = kv8_attention(q, c, s, t, n)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = kv8_attention(q, c, s, t, n)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        q2 = q.clone()
        with torch.cuda.graph(graph):
            out = kv8_attention(q2, c, s, t, n)
        q2.copy_(-q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kv8_attention(-q, c, s, t, n))


def test_empty_calls():
    codes, scales = kv8_pool(1, 4, 2, 64, page=16)
    t, n = torch.full((0, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert kv8_attention(q, codes[0], scales[0], t, n).shape == q.shape
    kv8_append(q, q, codes[0], scales[0], t, n)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    for cols in (0, 3):
        t = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
        for tokens in (1, 20):
            q = torch.randn(2, tokens, 2, 64, device="cuda").to(torch.bfloat16)
            for lengths in (none, none + 40):
                o, lse = kv8_attention(q, codes[0], scales[0], t, lengths, need_lse=True)
                assert torch.all(o == 0) and torch.all(torch.isneginf(lse))
            kv8_append(q, q, codes[0], scales[0], t, none)
    assert not codes.any() and not scales.any()


def test_refusals():
    codes, scales = kv8_pool(1, 4, 2, 64, page=16)
    codes, scales = codes[0], scales[0]
    t, n = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    from gated_delta_rule_54_gb300 import GdnError
    for bad, kind in [
        (lambda: kv8_attention(q.float(), codes, scales, t, n), GdnError),
        (lambda: kv8_attention(q[..., :32], codes, scales, t, n), ValueError),
        (lambda: kv8_attention(q[:, :, :3], codes, scales, t, n), ValueError),
        (lambda: kv8_attention(q.cpu(), codes, scales, t, n), ValueError),
        (lambda: kv8_attention(q, codes.float(), scales, t, n), ValueError),
        (lambda: kv8_attention(q, codes, scales[:, :2], t, n), ValueError),
        (lambda: kv8_attention(q, codes, scales, t.long(), n), ValueError),
        (lambda: kv8_attention(q, codes, scales, t, n.repeat(2)), ValueError),
        (lambda: kv8_attention(q, codes, scales, t, n, mode="none"), ValueError),
        (lambda: kv8_attention(q, codes, scales, t, n, scale=float("nan")), GdnError),
        (lambda: kv8_attention(q, codes, scales, t, n, window=-1), GdnError),
        (lambda: kv8_attention(q, codes[:, :, :, :8].contiguous(), scales, t, n), GdnError),
        (lambda: kv8_attention(q.transpose(2, 3).contiguous().transpose(2, 3), codes, scales, t, n), ValueError),
        (lambda: kv8_attention(q, codes, scales, t, n, out=torch.empty_like(q[:, :, :2])), ValueError),
        (lambda: kv8_append(q, q, codes, scales, t, n), ValueError),
        (lambda: kv8_append(q[:, :, :2], q[:, :, :2].half(), codes, scales, t, n), ValueError),
        (lambda: kv8_append(q[0, :, :2], q[0, :, :2], codes, scales, t, n, cu_seqlens=n), ValueError),
    ]:
        with pytest.raises(kind):
            bad()
    long = torch.zeros(1, 300, dtype=torch.int32, device="cuda")
    with pytest.raises(GdnError):       # a workspace that is too small is an error, not a fallback
        kv8_attention(q, codes, scales, long, n, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()

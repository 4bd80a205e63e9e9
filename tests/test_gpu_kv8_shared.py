"""GPU: attention of rows that have their first tokens in common, against the oracle.

Tolerances as for the attention over the cache (test_gpu_kv8.py): bf16 rounding of the output
(2^-8 of itself), fp16 rounding of the probabilities (2^-11 of the sum of p |v|, and 2^-25
of the largest p * V scale per key below fp16's normal range), 2^-15 of that sum for the fp32
sums and the join of the parts, and 2^-20 of the largest sum of |q k| (and of 1) for the
scores and the exponential, twice."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import GdnError, kv8_attention, kv8_attention_shared, kv8_pool, kv8_shared_workspace_bytes, load
from oracle import serve as ref

pytestmark = pytest.mark.gpu


def _pool(rng, pages, heads, page, dim, mode):
    x = rng.standard_normal((2, pages, heads, page, dim)) * np.exp(0.5 * rng.standard_normal((2, pages, heads, 1, 1)))
    s = (np.abs(x).max((3, 4)) / ref.CODE_MAX[mode]).astype(np.float32)
    return ref.encode((x / s[..., None, None]).astype(np.float32), mode), s


def _cuda(*xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _inputs(rng, shared, tails, tokens, heads, group, dim, page, mode, qstd=1.5, cols=None, together=True):
    """A pool, a table and queries: groups of len(tails) // len(shared) rows."""
    beams = len(tails) // len(shared)
    lens = [max(shared[r // beams], 0) + n for r, n in enumerate(tails)]
    used = [-(-n // page) for n in lens]
    cols = max(used + [1]) if cols is None else cols
    pages = sum(used) + 3
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    ids, table, at = rng.permutation(pages), np.full((len(tails), max(cols, max(used + [1]))), -1, np.int32), 0
    for r, u in enumerate(used):
        table[r, :u] = ids[at:at + u]
        at += u
        whole = max(shared[r // beams], 0) // page
        if together and r % beams:
            table[r, :whole] = table[r // beams * beams, :whole]
    for r, n in enumerate(lens):  # slots past a row's end hold bytes that are no numbers
        if n % page and (r % beams == 0 or n // page >= max(shared[r // beams], 0) // page):
            codes[:, table[r, n // page], :, n % page:] = 0x7f if mode == "e4m3" else 0x80
    wide = torch.from_numpy(rng.standard_normal((len(tails), tokens, heads * group + 2, dim)) * qstd).to(torch.bfloat16).cuda()
    return codes, scales, table[:, :cols], np.array(lens, np.int32), np.array(shared, np.int32), beams, wide[:, :, 1:-1]


def _check(got, q, codes, scales, table, lens, shared, beams, mode, scale, causal=True):
    o, lse = (x.float().cpu().numpy().astype(np.float64) for x in got)
    q = q.float().cpu().numpy().astype(np.float64)
    for r, n in enumerate(lens):
        first = r // beams * beams
        ro, rl, absum, top, dots = ref.attention_shared(q[r], codes, scales, table[first], table[r], min(int(shared[r // beams]), int(lens[first])),
                                                        int(n), mode, scale, causal)
        seen = np.isfinite(rl)
        assert np.array_equal(np.isneginf(lse[r]), ~seen)
        assert np.all(o[r][~seen] == 0)
        score = 2.0 ** -20 * (dots + 1)
        tol = (1.01 * 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -15 + 2 * score[..., None]) * absum
               + 2.0 ** -25 * max(int(n), 1) * top[..., None] + 1e-37)
        err = np.abs(o[r] - ro)
        assert np.all(err <= tol), "row %d: %.3g over %.3g" % (r, err.max(), (tol[err > tol]).min())
        d = np.abs(lse[r][seen] - rl[seen])
        assert np.all(d <= 2.0 ** -16 + score[seen]), "row %d: lse off by %.3g" % (r, d.max())


def _run(rng, shared, tails, tokens, heads, group, dim, page, mode, scale=None, causal=True, spoil=None, **kw):
    codes, scales, table, lens, common, beams, q = _inputs(rng, shared, tails, tokens, heads, group, dim, page, mode, **kw)
    if spoil:
        spoil(codes, scales, table, lens, common)
    c, s, t, n, p = _cuda(codes, scales, table, lens, common)
    args = dict(mode=mode, scale=scale, causal=causal, need_lse=True)
    got = kv8_attention_shared(q, c, s, t, n, p, beams, **args)
    again = kv8_attention_shared(q, c, s, t, n, p, beams, **args)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert load().gdn_device_error(0) == 0
    _check(got, q, codes, scales, table, lens, common, beams, mode, dim ** -0.5 if scale is None else scale, causal)
    return got


CASES = [
    # tokens in common, tails, tokens, heads, group, dim, page, mode
    ([64], [1], 1, 1, 1, 128, 64, "e4m3"),
    ([0], [1, 0, 5], 1, 2, 2, 64, 16, "int8"),
    ([1], [1, 2, 40], 1, 1, 4, 128, 16, "int8"),
    ([700], [30, 31, 1, 77], 1, 2, 4, 128, 64, "e4m3"),
    ([127, 128, 129], [33] * 12, 1, 1, 4, 128, 128, "e4m3"),
    ([640, 17, 0, 333], [3, 60, 9, 0, 1, 2, 128, 65], 1, 2, 3, 64, 32, "int8"),
    ([3001, 900], [300, 5, 64, 12, 7, 300], 5, 2, 3, 64, 16, "int8"),
    ([2000], [64] * 33, 1, 1, 8, 128, 32, "e4m3"),            # 264 query rows of a K/V head
    ([1000, 1500], [9, 40, 300, 2] * 2, 2, 3, 5, 128, 16, "int8"),
    ([130], [4] * 70, 3, 1, 2, 64, 64, "e4m3"),               # 420
    ([9000], [70, 3], 1, 2, 16, 64, 64, "e4m3"),
    ([512], [512] * 5, 1, 8, 1, 128, 128, "int8"),
    ([400], [1, 2, 3, 4], 8, 1, 2, 64, 16, "e4m3"),           # queries that stand before the tokens' end
    ([2, 3], [1, 0, 2, 1], 6, 1, 2, 128, 16, "int8"),         # and before the row's begin
    ([5000], [100], 1, 1, 4, 128, 64, "e4m3"),                # one row
    ([250] * 40, [30] * 80, 1, 2, 2, 64, 32, "e4m3"),         # many groups
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_oracle(case):
    _run(np.random.default_rng(case), *CASES[case])


@pytest.mark.parametrize("dim,mode,page", [(128, "e4m3", 64), (64, "int8", 16), (128, "int8", 128), (64, "e4m3", 32)])
def test_every_prefix_around_a_tile(dim, mode, page):
    rng = np.random.default_rng(dim + page)
    shared = [0, 1, 15, 16, 31, 32, 33, 63, 65, 127, 128, 129, 255, 256, 257]
    _run(rng, shared, [int(x) for x in rng.integers(0, 40, 2 * len(shared))], 2, 1, 3, dim, page, mode)


def test_not_causal_and_a_negative_scale():
    rng = np.random.default_rng(20)
    _run(rng, [300, 40], [20, 1, 3, 64], 4, 2, 2, 128, 64, "e4m3", causal=False)
    _run(rng, [300, 40], [20, 1, 3, 64], 3, 2, 2, 64, 16, "int8", scale=-0.07)
    _run(rng, [300, 40], [20, 1, 3, 64], 1, 2, 2, 64, 16, "int8", scale=2.0)


def test_shared_counts_that_do_not_fit():
    """Below 0, past the rows' lengths, past the table: cut, and each query sees its own keys only."""
    rng = np.random.default_rng(21)

    def longer(codes, scales, table, lens, common):
        common[:] = [-5, 290, 1 << 30, (1 << 31) - 1]
    _run(rng, [100, 100, 100, 100], [200, 20, 30, 100, 7, 7, 64, 5], 2, 1, 2, 128, 32, "e4m3", spoil=longer, together=False)
    rng = np.random.default_rng(22)

    def shorter(codes, scales, table, lens, common):
        lens[:] = [90, 200, 0, -3, 150, 1 << 30]
    _run(rng, [100, 100, 100], [50] * 6, 2, 1, 2, 64, 16, "int8", spoil=shorter)
    _run(np.random.default_rng(23), [500], [40, 90], 1, 2, 4, 128, 64, "e4m3", cols=7)      # a table narrower than the rows


def test_holes_and_scales():
    def spoil(codes, scales, table, lens, common):
        table[0, 1], table[1, 12], table[3, 11] = -1, 99999, -7
        scales[1, table[0, 2]], codes[1, table[0, 2]] = 0, 0
        scales[0, table[0, 3]], codes[0, table[0, 3]] = 0, 0
        scales[1, table[0, 4]] *= 2.0 ** 20
        scales[1, table[0, 6]] *= 2.0 ** -10
        scales[1, table[1, 13]] *= 2.0 ** 15
    for dim, mode, page in ((128, "e4m3", 16), (64, "int8", 16)):
        _run(np.random.default_rng(24), [200], [40, 50, 33, 7], 1, 2, 4, dim, page, mode, spoil=spoil)
    def nothing(codes, scales, table, lens, common):
        table[:] = -1
    o, lse = _run(np.random.default_rng(25), [200, 10], [40, 50, 33, 7], 2, 1, 2, 64, 32, "e4m3", spoil=nothing)
    assert not o.any() and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("tiny", [2.0 ** -135, 2.0 ** -110, 2.0 ** 100])
def test_v_scales_of_all_sizes(tiny):
    """Blocks whose V scales lie far apart: a query that looks at the small ones only keeps them."""
    rng = np.random.default_rng(26)
    for pages_small in (range(0, 4), range(4, 8), range(1, 8, 2)):
        def spoil(codes, scales, table, lens, common):
            for c in pages_small:
                scales[1, table[0, c]] *= np.float32(tiny)
        codes, scales, table, lens, common, beams, q = _inputs(rng, [256], [40, 3], 1, 1, 2, 128, 32, "e4m3")
        spoil(codes, scales, table, lens, common)
        c, s, t, n, p = _cuda(codes, scales, table, lens, common)
        got = kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)
        _check(got, q, codes, scales, table, lens, common, beams, "e4m3", 128 ** -0.5)
        same = kv8_attention(q, c, s, *_cuda(np.concatenate([np.repeat(table[:1, :8], 2, 0), table[:, 8:]], 1)), n, need_lse=True)
        _check(same, q, codes, scales, table, lens, common, beams, "e4m3", 128 ** -0.5)


def test_what_is_no_number():
    """A query that is not finite is NaN, and one that sees a key of a block whose scale is not; others are not touched."""
    rng = np.random.default_rng(27)
    codes, scales, table, lens, common, beams, q = _inputs(rng, [256, 64], [40, 3, 20, 9, 50, 11], 2, 2, 3, 64, 16, "e4m3")
    q = q.clone()
    c, s, t, n, p = _cuda(codes, scales, table, lens, common)
    clean = kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)
    q[0, 1, 2, 7], q[2, 0, 5, 0] = float("inf"), float("nan")
    s[0, table[1, 16], 1] = float("nan")            # a K block of row 1's own tokens
    s[1, table[3, 2], 0] = float("inf")             # a V block of the second group's first tokens
    o, lse = kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)
    want = torch.zeros_like(lse, dtype=torch.bool)
    want[0, 1, 2] = want[2, 0, 5] = True
    want[1, :, 3:] = True
    want[3:, :, :3] = True
    assert torch.equal(torch.isnan(lse), want)
    assert torch.equal(torch.isnan(o), want[..., None].expand_as(o))
    assert torch.equal(o[~want], clean[0][~want]) and torch.equal(lse[~want], clean[1][~want])


def test_a_rows_result_does_not_depend_on_its_neighbours():
    """Rows in another order, and a row whose scores are far larger beside them."""
    rng = np.random.default_rng(28)
    for tokens, group, count in ((1, 4, 8), (2, 3, 40)):
        codes, scales, table, lens, common, beams, q = _inputs(rng, [1472], [40] * count, tokens, 2, group, 128, 64, "e4m3")
        c, s, t, n, p = _cuda(codes, scales, table, lens, common)
        q = q.clone()
        o, lse = kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)
        order = torch.from_numpy(rng.permutation(count)).cuda()
        o2, lse2 = kv8_attention_shared(q[order], c, s, t[order].contiguous(), n, p, beams, need_lse=True)
        assert torch.equal(o2, o[order]) and torch.equal(lse2, lse[order])
        q[1::2] *= 30
        o3, lse3 = kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)
        assert torch.equal(o3[::2], o[::2]) and torch.equal(lse3[::2], lse[::2])


@pytest.mark.parametrize("beams,tokens,group", [(12, 1, 4), (16, 2, 2), (7, 3, 3)])
def test_a_place_in_the_group_does_not_count_where_ctas_have_uneven_shares(beams, tokens, group):
    """Up to 64 query rows of a K/V head, more tiles than CTAs: 2 groups x 4 heads x 40 tiles and more."""
    rng = np.random.default_rng(31)
    codes, scales, table, lens, common, beams, q = _inputs(rng, [5056, 6016], [40] * (2 * beams), tokens, 4, group, 128, 64, "e4m3")
    c, s, t, n, p = _cuda(codes, scales, table, lens, common)
    o, lse = kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)
    order = torch.from_numpy(np.concatenate([rng.permutation(beams), beams + rng.permutation(beams)])).cuda()
    o2, lse2 = kv8_attention_shared(q[order], c, s, t[order].contiguous(), n[order], p, beams, need_lse=True)
    assert torch.equal(o2, o[order]) and torch.equal(lse2, lse[order])


@pytest.mark.parametrize("mode,beams,group", [("e4m3", 4, 4), ("int8", 8, 4), ("e4m3", 16, 4), ("int8", 40, 4)])
def test_neighbours_do_not_count_whatever_the_scales_of_v(mode, beams, group):
    """Scores of a row may outgrow its earlier ones where V's scale is small; rows beside it that are
    spoilt, or have far larger scores, or none, change no bit of it."""
    rng = np.random.default_rng(33)
    codes, scales, table, lens, common, n, q = _inputs(rng, [6016], [40] * beams, 1, 2, group, 128, 64, mode, qstd=4.0)
    scales[1] *= np.exp2(rng.integers(-30, 5, scales[1].shape)).astype(np.float32)
    c, s, t, l, p = _cuda(codes, scales, table, lens, common)
    q = q.clone()
    o, lse = kv8_attention_shared(q, c, s, t, l, p, n, mode=mode, need_lse=True)
    for change in (30.0, 0.0, float("nan")):
        q2 = q.clone()
        q2[1::2] *= change
        o2, lse2 = kv8_attention_shared(q2, c, s, t, l, p, n, mode=mode, need_lse=True)
        assert torch.equal(o2[::2], o[::2]) and torch.equal(lse2[::2], lse[::2]), change


@pytest.mark.parametrize("mode,beams", [("e4m3", 4), ("int8", 8), ("e4m3", 16), ("int8", 12)])
def test_a_columns_references_move_for_itself(mode, beams):
    """In one tile, pages 22 and 23, scores are three times as large and V's scale 2^-25: they outgrow the
    earlier ones by more than 2^8 but their products with V's scale do not, unless a row's q is eight
    times as large.  That tile has nearly all of a row's weight, and so its part the row's log-sum-exp."""
    rng = np.random.default_rng(35)
    # (8 x 47 tiles, two or three to a CTA: some begin with tiles 9 and 10)
    codes, scales, table, lens, common, n, q = _inputs(rng, [6016], [40] * beams, 1, 8, 4, 64, 64, mode)
    late = np.unique(table[:, 22:24])
    scales[0][late] *= 3
    scales[1][late] *= np.float32(2.0 ** -25)
    c, s, t, l, p = _cuda(codes, scales, table, lens, common)
    q = q.clone()
    want = kv8_attention_shared(q, c, s, t, l, p, n, mode=mode, need_lse=True)
    _check(want, q, codes, scales, table, lens, common, n, mode, 64 ** -0.5)
    q[1::2] *= 8
    got = kv8_attention_shared(q, c, s, t, l, p, n, mode=mode, need_lse=True)
    assert torch.equal(got[0][::2], want[0][::2]) and torch.equal(got[1][::2], want[1][::2])
    assert load().gdn_device_error(0) == 0


def test_stream_graph_workspace_and_far_pages():
    rng = np.random.default_rng(29)
    heads, page, dim = 8, 128, 128
    codes, scales, table, lens, common, beams, q = _inputs(rng, [1100], [40, 150, 9], 1, heads, 2, dim, page, "e4m3")
    c, s, t, n, p = _cuda(codes, scales, table, lens, common)
    want = kv8_attention_shared(q, c, s, t, n, p, beams)
    torch.cuda.synchronize()
    far = (1 << 32) // (heads * page * dim) + 5
    big = torch.zeros(2, far + len(codes[0]), heads, page, dim, dtype=torch.uint8, device="cuda")
    bs = torch.zeros(2, far + len(codes[0]), heads, device="cuda")
    big[:, far:], bs[:, far:] = c, s
    t2 = torch.where(t >= 0, t + far, t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = kv8_attention_shared(q, big, bs, t2, n, p, beams)
    side.synchronize()
    assert torch.equal(got, want)
    need = kv8_shared_workspace_bytes(q, c, s, t, n, beams)
    room = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    graphs = []
    q2 = q.clone()
    for _ in range(2):     # two graphs that use one workspace, one after the other
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, kv8_attention_shared(q2, c, s, t, n, p, beams, workspace=room)))
    for graph, out in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert torch.equal(out, want)
    p.fill_(500)
    n.sub_(8)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    _check((graphs[0][1], kv8_attention_shared(q, c, s, t, n, p, beams, need_lse=True)[1]), q, codes, scales, table, lens - 8,
           [500], beams, "e4m3", dim ** -0.5)
    if need:
        with pytest.raises(GdnError):
            kv8_attention_shared(q, c, s, t, n, p, beams, workspace=room[:need - 1])
    out = torch.empty_like(want)
    assert kv8_attention_shared(q, c, s, t, n, p, beams, out=out) is out


def test_empty_and_refused():
    codes, scales = kv8_pool(1, 4, 2, 64, page=16)
    codes, scales = codes[0], scales[0]
    t, n = torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.ones(4, dtype=torch.int32, device="cuda")
    p = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(4, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert kv8_attention_shared(q[:0], codes, scales, t[:0], n[:0], p[:0], 2).shape == (0, 1, 4, 64)
    assert kv8_attention_shared(q[:, :0], codes, scales, t, n, p, 2).shape == (4, 0, 4, 64)
    o, lse = kv8_attention_shared(q, codes, scales, t[:, :0], n, p, 2, need_lse=True)
    assert not o.any() and torch.all(torch.isneginf(lse))
    o, lse = kv8_attention_shared(q, codes[:, :0].contiguous(), scales[:, :0].contiguous(), t, n, p, 2, need_lse=True)
    assert not o.any() and torch.all(torch.isneginf(lse))
    f = kv8_attention_shared
    for bad, kind in [
        (lambda: f(q, codes, scales, t, n, p, 3), ValueError), (lambda: f(q, codes, scales, t, n, p, 0), ValueError),
        (lambda: f(q, codes, scales, t, n, p, -2), ValueError), (lambda: f(q, codes, scales, t, n, p, 4), ValueError),
        (lambda: f(q, codes, scales, t, n, p.long(), 2), ValueError), (lambda: f(q, codes, scales, t, n, p.cpu(), 2), ValueError),
        (lambda: f(q, codes, scales, t, n, p[:, None], 2), ValueError), (lambda: f(q[:, 0], codes, scales, t, n, p, 2), ValueError),
        (lambda: f(q.float(), codes, scales, t, n, p, 2), GdnError), (lambda: f(q, codes, scales, t, n, p, 2, scale=float("inf")), GdnError),
        (lambda: f(q, codes, scales, t, n, p, 2, mode="none"), ValueError), (lambda: f(q, codes, scales, t, n, p, 2, out=q[:2]), ValueError),
        (lambda: f(q, codes, scales, t, n, p, 2, workspace=torch.empty(64)), ValueError),
    ]:
        with pytest.raises(kind):
            bad()
    torch.cuda.synchronize()

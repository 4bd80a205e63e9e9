"""GPU: append with the rotation on the way, bit for bit against the oracle.

The definition fixes every rounding (each product and each sum to fp32, queries once to
bf16), so codes, scales and queries have to be equal."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import GdnError, kv8_append, kv8_append_rotary, kv8_pool
from oracle import serve as ref

pytestmark = pytest.mark.gpu


def _angles(positions, half):
    a = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _pool(rng, pages, heads, page, dim, mode):
    x = rng.standard_normal((2, pages, heads, page, dim))
    s = (np.abs(x).max((3, 4)) / ref.CODE_MAX[mode]).astype(np.float32)
    return ref.encode((x / s[..., None, None]).astype(np.float32), mode), s * rng.choice([0.3, 1.0, 3.0], s.shape).astype(np.float32)


def _cuda(*xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _bits(x):
    return np.ascontiguousarray(x).view(np.uint32)


CASES = [
    # starts, counts (a list: packed), heads, group, dim, rotary, interleaved, page, mode
    ([701], 1, 2, 8, 128, 128, False, 64, "e4m3"),
    ([0, 5, 16, 31, 0, 47], 1, 3, 2, 128, 64, True, 16, "e4m3"),
    ([63, 64, 65, 0, 127], 1, 1, 5, 64, 64, False, 64, "int8"),
    ([9, 8, 7], [1, 0, 1], 2, 1, 64, 16, True, 16, "int8"),
    ([0, 100, 7], [300, 1, 64], 2, 3, 128, 96, False, 32, "int8"),
    ([3, 0, 0, 250], [0, 129, 1, 270], 3, 1, 64, 48, True, 128, "e4m3"),
    ([10, 0], 7, 2, 4, 128, 128, True, 128, "e4m3"),
    ([1, 33], 140, 1, 2, 128, 112, False, 128, "int8"),
    ([5, 60], 2, 8, 8, 128, 16, False, 64, "e4m3"),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_bit_exact(case):
    starts, counts, heads, group, dim, rotary, inter, page, mode = CASES[case]
    rng = np.random.default_rng(300 + case)
    packed = isinstance(counts, list)
    n = counts if packed else [counts] * len(starts)
    lengths = [a + b for a, b in zip(starts, n)]
    used = [-(-x // page) for x in lengths]
    pages = sum(used) + 2
    codes, scales = _pool(rng, pages, heads, page, dim, mode)
    table, ids, at = np.full((len(n), max(used)), -1, np.int32), rng.permutation(pages), 0
    for r, u in enumerate(used):
        table[r, :u] = ids[at:at + u]
        at += u
    cos, sin = _angles(max(lengths) + 1, rotary // 2)
    # tokens before the first row and behind the last one belong to none
    lead, total = (2, sum(n) + 5) if packed else (0, sum(n))
    wide = torch.from_numpy(rng.standard_normal((total, (group + 2) * heads + 1, dim))).to(torch.bfloat16).cuda()
    wide[:, :, 0] *= 20
    wide[lead] = 0
    q, k, v = wide[:, :group * heads], wide[:, group * heads:(group + 1) * heads], wide[:, (group + 1) * heads:-1]
    cu = lead + np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    host = [x.float().cpu().numpy() for x in (q, k, v)]
    rows = [[x[cu[r]:cu[r + 1]] for r in range(len(n))] for x in host]
    if not packed:
        q, k, v = (x.unflatten(0, (len(starts), counts)) for x in (q, k, v))
    c, s, t, st, dc, ds = _cuda(codes, scales, table, np.array(starts, np.int32), cos, sin)
    turned = [[ref.turn(x, range(a, a + len(x)), cos, sin, inter) for x, a in zip(part, starts)] for part in rows[:2]]
    ref.append(turned[1], rows[2], codes, scales, table, starts, n, mode)
    want = np.zeros(host[0].shape, np.float32)
    for r in range(len(n)):
        want[cu[r]:cu[r + 1]] = turned[0][r]
    want = torch.from_numpy(want).to(torch.bfloat16)
    for _ in range(2):  # the same call again changes nothing more
        got = kv8_append_rotary(q, k, v, c, s, t, st, dc, ds, interleaved=inter, cu_seqlens=_cuda(cu)[0] if packed else None,
                                max_seqlen=max(n) if packed else None, mode=mode)
        assert got.is_contiguous() and got.shape == q.shape
        assert torch.equal(got.cpu().view(torch.int16).flatten(), want.view(torch.int16).flatten())
        assert np.array_equal(_bits(s.cpu().numpy()), _bits(scales))
        assert np.array_equal(c.cpu().numpy(), codes)


def test_angles_of_zero_are_the_plain_append():
    torch.manual_seed(1)
    for tokens in (1, 20):
        k, v, q = (torch.randn(2, tokens, h, 64, device="cuda").to(torch.bfloat16) for h in (2, 2, 4))
        table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
        start = torch.tensor([3, 9], dtype=torch.int32, device="cuda")
        cos, sin = torch.ones(40, 32, device="cuda"), torch.zeros(40, 32, device="cuda")
        a, b = kv8_pool(1, 4, 2, 64, page=16), kv8_pool(1, 4, 2, 64, page=16)
        kv8_append(k, v, a[0][0], a[1][0], table, start)
        got = kv8_append_rotary(q, k, v, b[0][0], b[1][0], table, start, cos, sin)
        assert torch.equal(got, q)
        assert torch.equal(a[1], b[1])
        assert torch.equal(a[0] & 0x7f, b[0] & 0x7f)      # zeros may differ in sign


@pytest.mark.parametrize("tokens", [1, 9])
def test_positions_without_angles_pages_or_sense(tokens):
    """Positions past cos, before 0, past the table's columns, and pages that are none."""
    rng = np.random.default_rng(4)
    heads, dim, page, mode = 2, 64, 16, "e4m3"
    starts = [30, 60, -4, 10, 40, (1 << 31) - 12]
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7], [8, 9, 10, 11], [12, -1, 99, 13], [14, 15, 16, 17], [18, 19, 20, 21]], np.int32)
    codes, scales = _pool(rng, 22, heads, page, dim, mode)
    cos, sin = _angles(44, 32)
    x = rng.standard_normal((6, tokens, 6, dim)).astype(np.float32)
    dev = torch.from_numpy(x).to(torch.bfloat16).cuda()
    x = dev.float().cpu().numpy()
    c, s, t, st, dc, ds = _cuda(codes, scales, table, np.array(starts, np.int64).astype(np.int32), cos, sin)
    got = kv8_append_rotary(dev[:, :, :2], dev[:, :, 2:4], dev[:, :, 4:], c, s, t, st, dc, ds).float().cpu().numpy()
    for r, a in enumerate(starts):
        want = torch.from_numpy(ref.turn(x[r, :, :2], range(a, a + tokens), cos, sin, False)).to(torch.bfloat16).float().numpy()
        assert np.array_equal(got[r], want, equal_nan=True)
    at = [a if 0 <= a < 64 else 64 for a in starts]
    k = [ref.turn(x[r, :, 2:4], range(a, a + tokens), cos, sin, False) for r, a in enumerate(at)]
    spoilt = np.zeros(scales.shape, bool)                    # K blocks with a position that cos does not have
    for r, a in enumerate(at):
        for i in range(tokens):
            if 44 <= a + i < 64 and 0 <= table[r, (a + i) // page] < 22:
                spoilt[0, table[r, (a + i) // page]] = True
    with np.errstate(invalid="ignore"):
        ref.append([np.nan_to_num(y) for y in k], list(x[:, :, 4:]), codes, scales, table, at, [tokens] * 6, mode)
    assert np.array_equal(np.isnan(s.cpu().numpy()), spoilt)
    same = ~spoilt
    assert np.array_equal(s.cpu().numpy()[same], scales[same])
    assert np.array_equal(c.cpu().numpy()[same], codes[same])


def test_packed_rows_that_break_the_bound():
    """A row with more than max_seqlen tokens: its first keys are taken, its queries are NaN."""
    torch.manual_seed(2)
    x = torch.randn(12, 6, 64, device="cuda").to(torch.bfloat16)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    cos, sin = _cuda(*_angles(32, 16))
    for most, cu in ((4, [0, 7, 10]), (1, [1, 2, 12])):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        codes, scales = kv8_pool(1, 4, 2, 64, page=16)
        got = kv8_append_rotary(x[:, :2], x[:, 2:4], x[:, 4:], codes[0], scales[0], table, start, cos, sin, cu_seqlens=cu, max_seqlen=most)
        for r in range(2):
            a, b = int(cu[r]), int(cu[r + 1])
            assert bool(torch.isnan(got[a:b]).all()) == (b - a > most)
            assert int((codes[0, 1, table[r]] != 0).any(1).any(-1).sum()) == min(b - a, most)
        assert not got[:int(cu[0])].any() and not got[int(cu[2]):].any()


def test_not_numbers():
    torch.manual_seed(3)
    for tokens in (1, 12):
        x = torch.randn(2, tokens, 6, 128, device="cuda").to(torch.bfloat16)
        x[0, 0, 2, 5], x[1, -1, 5, 0] = float("inf"), float("nan")
        table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
        start = torch.zeros(2, dtype=torch.int32, device="cuda")
        codes, scales = kv8_pool(1, 4, 2, 128, page=16)
        cos, sin = _cuda(*_angles(32, 64))
        kv8_append_rotary(x[:, :, :2], x[:, :, 2:4], x[:, :, 4:], codes[0], scales[0], table, start, cos, sin)
        bad = ~torch.isfinite(scales[0])
        assert bad.sum() == 2 and bad[0, 0, 0] and bad[1, 2, 1]


def test_stream_graph_and_far_pages():
    heads, page, dim = 8, 128, 128
    pages = (1 << 32) // (heads * page * dim) + 9
    codes = torch.zeros(2, pages, heads, page, dim, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, pages, heads, device="cuda")
    table = torch.tensor([[pages - 1, 3]], dtype=torch.int32, device="cuda")
    small = kv8_pool(1, 2, heads, dim, page=page)
    near = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    cos, sin = _cuda(*_angles(300, 64))
    side = torch.cuda.Stream()
    torch.manual_seed(5)
    at = 0
    for tokens in (100, 1, 30):
        start = torch.full((1,), at, dtype=torch.int32, device="cuda")
        q, k, v = (torch.randn(1, tokens, h, dim, device="cuda").to(torch.bfloat16) for h in (2 * heads, heads, heads))
        want = kv8_append_rotary(q, k, v, small[0][0], small[1][0], near, start, cos, sin)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = kv8_append_rotary(q, k, v, codes, scales, table, start, cos, sin)
        side.synchronize()
        assert torch.equal(got, want)
        graph = torch.cuda.CUDAGraph()
        q2 = q.clone()
        with torch.cuda.graph(graph):
            out = kv8_append_rotary(q2, k, v, codes, scales, table, start, cos, sin)
        q2.copy_(-q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, -want)
        at += tokens
    assert torch.equal(codes[:, table[0].long()], small[0][0][:, near[0].long()])
    assert torch.equal(scales[:, table[0].long()], small[1][0][:, near[0].long()])


def test_empty_and_refused():
    codes, scales = kv8_pool(1, 4, 2, 64, page=16)
    codes, scales = codes[0], scales[0]
    t, n = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = q[:, :, :2]
    a = torch.ones(50, 32, device="cuda")
    assert kv8_append_rotary(q[:0], k[:0], k[:0], codes, scales, t[:0], n[:0], a, a).shape == (0, 1, 4, 64)
    assert kv8_append_rotary(q[:, :0], k[:, :0], k[:, :0], codes, scales, t, n, a, a).shape == (1, 0, 4, 64)
    assert torch.isnan(kv8_append_rotary(q + 1, k, k, codes, scales, t[:, :0], n, a[:0], a[:0])).all()
    call = lambda **w: kv8_append_rotary(*[{**dict(q=q, k=k, v=k, codes=codes, scales=scales, table=t, start=n, cos=a, sin=a), **w}[x]
                                           for x in ("q", "k", "v", "codes", "scales", "table", "start", "cos", "sin")],
                                         **{x: y for x, y in w.items() if x in ("mode", "cu_seqlens")})
    for bad, kind in [
        (dict(q=q.half()), ValueError), (dict(q=q.cpu()), ValueError), (dict(q=q[:, :, :3]), ValueError), (dict(q=q[..., :32]), ValueError),
        (dict(q=q[0]), ValueError), (dict(q=q.repeat(2, 1, 1, 1)), ValueError), (dict(q=q[:, :, :0]), ValueError),
        (dict(k=q, v=q, q=q), ValueError), (dict(v=q), ValueError), (dict(k=k.squeeze()[0], q=q.squeeze()[0]), ValueError),
        (dict(cos=a.double()), ValueError), (dict(cos=a.cpu()), ValueError), (dict(sin=a[:40]), ValueError), (dict(cos=a[0], sin=a[0]), ValueError),
        (dict(cos=a.t(), sin=a.t()), ValueError), (dict(cos=a[:, :4].contiguous(), sin=a[:, :4].contiguous()), GdnError),
        (dict(cos=torch.ones(50, 40, device="cuda"), sin=torch.ones(50, 40, device="cuda")), GdnError),
        (dict(cos=a.new_ones(50, 0), sin=a.new_ones(50, 0)), GdnError),
        (dict(q=q.float(), k=k.float(), v=k.float()), GdnError), (dict(mode="none"), ValueError), (dict(table=t.long()), ValueError),
        (dict(cu_seqlens=n), ValueError), (dict(q=torch.zeros(1, 1, 4, 68, dtype=torch.bfloat16, device="cuda")[..., :64]), GdnError),
    ]:
        with pytest.raises(kind):
            call(**bad)
    torch.cuda.synchronize()

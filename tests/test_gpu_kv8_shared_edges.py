"""GPU: corners of the attention over shared tokens, on lines of several tiles for each CTA.

Tolerances are those that test_gpu_kv8_shared.py derives.  A line has more tiles than any GPU of this kind has
SMs, so that every CTA goes through some tiles one after the other and carries what it has from one to the
next: two tiles at least, and with up to 16 query rows, where tiles go in turn to two sets, four."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import kv8_append, kv8_attention_shared, load
from oracle import serve as ref
from test_gpu_kv8_shared import _check, _cuda

pytestmark = pytest.mark.gpu

SMS = 152
# query rows of a K/V head as rows x query heads, which decide between 16, 32 and 64 of a block; 64-wide blocks also two
FORMS = [("e4m3", 128, 64, 4, 4), ("int8", 64, 16, 4, 3), ("int8", 128, 128, 2, 8), ("e4m3", 64, 32, 3, 5),
         ("e4m3", 128, 16, 8, 4), ("int8", 64, 64, 10, 3), ("int8", 128, 32, 8, 4), ("e4m3", 64, 128, 30, 1),
         ("e4m3", 128, 128, 16, 4), ("int8", 64, 32, 9, 5), ("int8", 128, 16, 11, 4), ("e4m3", 64, 64, 16, 4),
         ("e4m3", 128, 32, 18, 4), ("int8", 64, 128, 13, 8)]


class Line:
    """One group whose first tokens are tiles of 128 keys, the same for all rows, with a few tokens of each row's own."""

    def __init__(self, seed, mode, dim, page, beams, group, tokens=1, ragged=0):
        self.mode, self.dim, self.page, self.beams, self.group, self.heads = mode, dim, page, beams, group, 8
        rows = beams * group * tokens
        self.tiles = 80 if rows <= 16 else 48
        assert self.heads * self.tiles > (4 if rows <= 16 else 2) * SMS
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.common = self.tiles * 128 - ragged
        self.lens = self.common + 20 + 7 * np.arange(beams) % 50 + tokens
        first, own = self.tiles * 128 // page, -(-int(self.lens.max()) // page) - self.common // page + 1
        pages = first + beams * own
        ids = self.rng.permutation(pages).astype(np.int32)
        self.table = np.full((beams, first + own), -1, np.int32)
        self.table[:, :first] = ids[:first]
        whole = self.common // page
        for r in range(beams):
            use = slice(first + r * own, first + (r + 1) * own)
            self.table[r, whole:whole + own] = ids[use]
            if r == 0:                                       # (the last page in common, where it is not whole)
                self.table[0, whole:first], self.table[0, first:] = ids[whole:first], ids[use][:self.table.shape[1] - first]
        # scores of a few units; dim 0 is for what a test adds to them
        self.q = torch.randn(beams, tokens, self.heads * group, dim, generator=self.gen, device="cuda")
        self.q *= 0.5
        self.q[..., 0] = 8.0
        self.q = self.q.to(torch.bfloat16)
        self.x = torch.randn(2, pages, self.heads, page, dim, generator=self.gen, device="cuda")
        self.x[0, ..., 0] = 0
        self.factor = torch.ones(pages, self.heads, device="cuda")  # of V's scales

    def of(self, per_tile):
        """[tiles, heads] as [pages of these, heads], in the table's order."""
        return np.repeat(per_tile, 128 // self.page, 0), torch.from_numpy(self.table[0, :self.tiles * 128 // self.page].astype(np.int64)).cuda()

    def levels(self, log2):
        """Adds to the scores of tile t for head h, in powers of two."""
        x, ids = self.of(log2)
        c = self.dim ** -0.5 * 1.4426950408889634 * 8.0
        self.x[0, ids, ..., 0] = torch.from_numpy((x / c).astype(np.float32)).cuda()[..., None]

    def v_scales(self, by):
        x, ids = self.of(by)
        self.factor[ids] = torch.from_numpy(x.astype(np.float32)).cuda()

    def cache(self):
        s = self.x.abs().amax((-2, -1)) / ref.CODE_MAX[self.mode]
        u = self.x / s.clamp(min=1e-37)[..., None, None]
        if self.mode == "e4m3":
            codes = u.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            codes = u.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
        s[1] *= self.factor
        return codes.contiguous(), s.contiguous()

    def run(self, codes, scales, q=None, table=None, lens=None):
        t, n, p = _cuda(self.table if table is None else table, (self.lens if lens is None else lens).astype(np.int32),
                        np.array([self.common], np.int32))
        got = kv8_attention_shared(self.q if q is None else q, codes, scales, t, n, p, self.beams, mode=self.mode, need_lse=True)
        assert load().gdn_device_error(0) == 0
        return got

    def check(self, got, codes, scales, table=None, lens=None):
        """Some rows, the first among them."""
        rows = sorted({0, self.beams // 2, self.beams - 1})
        table, lens = (self.table if table is None else table)[rows], (self.lens if lens is None else lens)[rows]
        _check([x[rows] for x in got], self.q[rows], codes.cpu().numpy(), scales.cpu().numpy(), table, lens, [self.common], len(rows),
               self.mode, self.dim ** -0.5)

    def alone(self, got, codes, scales):
        """Bits of every other row are the same beside rows of any other kind."""
        for change in (float("nan"), -30.0):
            q = self.q.clone()
            q[1::2] *= change
            o, lse = self.run(codes, scales, q)
            assert torch.equal(o[::2], got[0][::2]) and torch.equal(lse[::2], got[1][::2]), change


# ---- V scales of 0 -----------------------------------------------------
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS)
def test_tiles_whose_v_is_zero(mode, dim, page, beams, group):
    """V of whole tiles is 0, with the scale 0 that append gives it: two of four, so that a CTA's share, and each set of
    tiles in turn, begins with such a tile and goes on with others."""
    for phase in range(4):
        a = Line(40 + phase, mode, dim, page, beams, group)
        t = (np.arange(a.tiles)[:, None] + np.arange(a.heads)) % 4
        a.v_scales(np.where((t == phase) | (t == (phase + 1) % 4), 0.0, 1.0))
        codes, scales = a.cache()
        codes[1][(scales[1] == 0)] = 0
        got = a.run(codes, scales)
        a.check(got, codes, scales)
        if phase == 0:
            a.alone(got, codes, scales)


# ---- V codes that are no number ----------------------------------------
def _random_cache(gen, pages, heads, page, dim, mode):
    x = torch.randn(2, pages, heads, page, dim, generator=gen, device="cuda")
    s = x.abs().amax((-2, -1)) / ref.CODE_MAX[mode]
    u = x / s[..., None, None]
    if mode == "e4m3":
        return u.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s
    return u.round().clamp(-127, 127).to(torch.int8).view(torch.uint8), s


@pytest.mark.parametrize("spoilt", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("mode,dim,page,group", [("e4m3", 128, 64, 1), ("e4m3", 128, 16, 4), ("e4m3", 64, 32, 2), ("e4m3", 64, 16, 3),
                                                 ("int8", 128, 32, 2), ("int8", 64, 16, 4)])
def test_a_draft_whose_v_is_no_number(mode, dim, page, group, spoilt):
    """It, or it and the one before, opens a new page, whose codes and scale append makes of such a V: the drafts before
    it do not see that page, and are the same to the bit as without it."""
    gen, heads, tokens = torch.Generator(device="cuda").manual_seed(50), 2, 4
    opens = [1, 2, 1]                                  # drafts on the new page, by row
    lens = [6 * page + 1, 5 * page + 2, 9 * page + 1]
    table = torch.full((3, 10), -1, dtype=torch.int32)
    table[:, :2], at = torch.tensor([0, 1]), 2         # two pages in common
    for r, n in enumerate(lens):
        own = -(-n // page) - 2
        table[r, 2:2 + own] = torch.arange(at, at + own)
        at += own
    codes, scales = _random_cache(gen, at, heads, page, dim, mode)
    table, n, p = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.tensor([2 * page], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(3, tokens, heads, dim, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(3, tokens, heads * group, dim, generator=gen, device="cuda").to(torch.bfloat16)
    got = []
    for bad in (False, True):
        if bad:
            v[:, tokens - 1, 1, 5] = spoilt
        c, s = codes.clone(), scales.clone()
        kv8_append(k, v, c, s, table, n - tokens, mode=mode)
        got.append(kv8_attention_shared(q, c, s, table, n, p, 3, mode=mode, need_lse=True))
    (o, lse), (o2, lse2) = got
    lost = torch.zeros(3, tokens, heads * group, dtype=torch.bool, device="cuda")
    for r, x in enumerate(opens):
        lost[r, tokens - x:, group:] = True
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert torch.equal(torch.isnan(o2), lost[..., None].expand_as(o2)) and torch.equal(torch.isnan(lse2), lost)
    assert torch.equal(o2[~lost], o[~lost]) and torch.equal(lse2[~lost], lse[~lost])


@pytest.mark.parametrize("spoilt", [float("nan"), float("inf")])
@pytest.mark.parametrize("mode,dim,page,beams,group", [("e4m3", 128, 64, 4, 4), ("e4m3", 64, 16, 4, 3), ("e4m3", 128, 32, 8, 4),
                                                       ("e4m3", 64, 64, 10, 3), ("e4m3", 128, 16, 16, 4), ("e4m3", 64, 32, 18, 4),
                                                       ("int8", 128, 16, 8, 4), ("int8", 64, 32, 4, 4)])
def test_tokens_in_common_whose_v_is_no_number(mode, dim, page, beams, group, spoilt):
    """Rows that end before such a token's page, though in its tile, are the same to the bit as without it."""
    gen, heads = torch.Generator(device="cuda").manual_seed(51), 2
    common, bad_at = 1400, 128 * 7 + page              # (a page that is not its tile's first one, where it has more)
    cols = -(-common // page) + 2
    table = torch.arange(cols, dtype=torch.int32).repeat(beams, 1)
    table[:, common // page:] = cols + torch.arange(beams * (cols - common // page), dtype=torch.int32).view(beams, -1)
    table[0, common // page:] = torch.arange(common // page, cols)
    codes, scales = _random_cache(gen, int(table.max()) + 1, heads, page, dim, mode)
    short = torch.arange(beams) % 2 == 1
    n = torch.where(short, bad_at - torch.arange(beams) % 3 * 5, common + 9).int().cuda()
    p = torch.tensor([common], dtype=torch.int32, device="cuda")
    table = table.cuda()
    q = torch.randn(beams, 1, heads * group, dim, generator=gen, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(1, page, heads, dim, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    got, first = [], torch.tensor([bad_at], dtype=torch.int32, device="cuda")
    for bad in (False, True):
        if bad:
            v[0, page // 2, 0, 3] = spoilt
        c, s = codes.clone(), scales.clone()
        kv8_append(k, v, c, s, table[:1].contiguous(), first, mode=mode)
        got.append(kv8_attention_shared(q, c, s, table, n, p, beams, mode=mode, need_lse=True))
    (o, lse), (o2, lse2) = got
    lost = torch.zeros(beams, 1, heads * group, dtype=torch.bool, device="cuda")
    lost[~short.cuda(), :, :group] = True
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    assert torch.equal(torch.isnan(o2), lost[..., None].expand_as(o2)) and torch.equal(torch.isnan(lse2), lost)
    assert torch.equal(o2[~lost], o[~lost]) and torch.equal(lse2[~lost], lse[~lost])


# ---- scores that outgrow earlier ones where V's scale is little --------
@pytest.mark.parametrize("by", [0.0, 2.0 ** -120, 2.0 ** -75])
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS[:8:2] + FORMS[9::2])
def test_scores_that_rise_where_v_is_little(mode, dim, page, beams, group, by):
    """One tile of four lies 2^124 above the others, and has a V scale that does not show it; the last tiles' V does."""
    for phase in (0, 2):
        a = Line(60 + phase, mode, dim, page, beams, group)
        t = (np.arange(a.tiles)[:, None] + np.arange(a.heads)) % 4
        late = (np.arange(a.tiles) >= a.tiles - 3)[:, None]
        a.levels(np.where((t == phase) | late, np.where(late, 122.0, 124.0), 0.0))
        a.v_scales(np.where((t == phase) & ~late, by, 1.0))
        a.q[1::4, ..., 0] = 4.0                        # (half of all that, for other rows)
        codes, scales = a.cache()
        got = a.run(codes, scales)
        assert torch.isfinite(got[0]).all() and torch.isfinite(got[1]).all()
        a.check(got, codes, scales)
        if phase == 0:
            a.alone(got, codes, scales)


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS[:13:3] + FORMS[1::6])
def test_scores_and_v_scales_of_all_sizes(mode, dim, page, beams, group, seed):
    """Any of them after any other, by tile and head."""
    a = Line(70 + seed, mode, dim, page, beams, group)
    shape = (a.tiles, a.heads)
    a.levels(a.rng.choice([0.0, 0.0, 40.0, 90.0, 124.0, 127.0], shape) * a.rng.choice([1.0, -1.0, 2.0], (1, a.heads)))
    a.v_scales(a.rng.choice([0.0, 0.0, 2.0 ** -135, 2.0 ** -110, 2.0 ** -60, 1.0, 2.0 ** 60], shape))
    a.q[1::3, ..., 0] = 6.0
    codes, scales = a.cache()
    got = a.run(codes, scales)
    a.check(got, codes, scales)
    a.alone(got, codes, scales)


# ---- scores below what 32 bits hold ------------------------------------
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS[:13:2])
def test_scores_below_fp32s_range(mode, dim, page, beams, group):
    """Such a key has a weight of 0: the result is, to the bit, that of a table without its page, in which a
    CTA's share may begin, or consist, or all that the group has."""
    a = Line(80, mode, dim, page, beams, group)
    a.q[..., 0] = 64.0
    clean = a.cache()
    tile = np.arange(a.tiles)
    for far in ((tile % 4 == 0) | (tile % 4 == 3), tile % 8 < 6, tile >= 0):
        codes, scales = (x.clone() for x in clean)
        x, ids = a.of(far)
        ids = ids[torch.from_numpy(x).cuda()]
        codes[0, ids] = 0
        codes[0, ids, ..., 0] = 0xfe if mode == "e4m3" else 0x81     # -448, -127
        scales[0, ids] = 3e38 / ref.CODE_MAX[mode]
        got = a.run(codes, scales)
        table = a.table.copy()
        table[:, :len(x)][:, x] = -1
        want = a.run(codes, scales, table=table)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        a.check(want, codes, scales, table)


# ---- what the other tests have, on long lines --------------------------
@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS)
def test_long_lines(mode, dim, page, beams, group, tokens):
    """Pages that are missing, an end inside a page with bytes that are no numbers behind it, uneven V scales, rows that
    end before the group's tokens do, several queries to a row."""
    a = Line(90 + tokens, mode, dim, page, beams, group, tokens, ragged=37)
    a.v_scales(np.exp2(a.rng.integers(-12, 3, (a.tiles, a.heads)).astype(float)) * (a.rng.random((a.tiles, a.heads)) > 0.1))
    codes, scales = a.cache()
    table, lens = a.table.copy(), a.lens.copy()
    holes = a.rng.choice(a.common // page, 9, replace=False)
    table[0, holes[:5]], table[0, holes[5:]] = -1, len(scales[0]) + 3
    if beams > 1:
        lens[beams - 1] = a.common - 500
    if beams // 2 > 0 and beams // 2 != beams - 1:
        lens[beams // 2] = tokens - 1                  # a query before the row's begin
    for r, n in enumerate(lens):
        if n % page and n >= a.common:
            codes[:, int(table[r, n // page]), :, n % page:] = 0x7f if mode == "e4m3" else 0x80
    got = a.run(codes, scales, table=table, lens=lens)
    a.check(got, codes, scales, table, lens)
    o, lse = a.run(codes, scales, table=table, lens=lens)
    assert torch.equal(o, got[0]) and torch.equal(lse, got[1])


@pytest.mark.parametrize("power", [-127.5, -120, 110])
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS[::5])
def test_v_scales_near_the_ends_of_their_range(mode, dim, page, beams, group, power):
    a = Line(95, mode, dim, page, beams, group)
    codes, scales = a.cache()
    scales[1] = 2.0 ** power
    a.check(a.run(codes, scales), codes, scales)


@pytest.mark.parametrize("power", [-110, 110])
@pytest.mark.parametrize("mode,dim,page,beams,group", FORMS[2::5])
def test_q_near_the_ends_of_its_range(mode, dim, page, beams, group, power):
    """Scores of ordinary size from a q and a K far from 1."""
    a = Line(96, mode, dim, page, beams, group)
    a.q = (a.q.float() * 2.0 ** power).to(torch.bfloat16)
    codes, scales = a.cache()
    scales[0] *= 2.0 ** -power
    a.check(a.run(codes, scales), codes, scales)

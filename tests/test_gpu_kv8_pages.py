"""GPU: pages of the 8-bit cache — fork, reserve, free, compact, copy — against plain loops."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import (GdnError, kv8_compact, kv8_copy_pages, kv8_fork, kv8_free, kv8_pool,
                                       kv8_reserve)
from oracle import serve as ref

pytestmark = pytest.mark.gpu


def _setup(rng, rows, pages, page, most, layers=2, heads=2, dim=64, shared=True):
    """A pool with random contents, rows of random lengths, some pages shared or held elsewhere."""
    codes, scales = kv8_pool(layers, pages, heads, dim, page=page)
    codes.copy_(torch.from_numpy(rng.integers(0, 256, codes.shape, dtype=np.uint8)))
    scales.copy_(torch.from_numpy(rng.standard_normal(scales.shape).astype(np.float32)))
    lengths = rng.integers(0, most + 1, rows).astype(np.int32)
    lengths[rng.random(rows) < 0.15] = 0
    cols = -(-most // page) + 2
    table, refs = np.full((rows, cols), -1, np.int32), np.zeros(pages, np.int32)
    ids = list(rng.permutation(pages))
    for r in range(rows):
        n = -(-lengths[r] // page)
        for c in range(n):
            if shared and r and c < lengths[r] // page and c < lengths[r - 1] // page and rng.random() < 0.5:
                table[r, c] = table[r - 1, c]     # a common prefix
            else:
                table[r, c] = ids.pop()
            refs[table[r, c]] += 1
    for p in ids[:2]:
        refs[p] += 1                               # held by something that is no row
    return codes, scales, table, lengths, refs


def _cuda(*xs):
    return [torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in xs]


def _moved(codes, scales, moves):
    c, s = codes.clone(), scales.clone()
    for a, b in moves:
        c[:, :, b], s[:, :, b] = codes[:, :, a], scales[:, :, a]
    return c, s


CASES = [(1, 8, 16, 40), (5, 60, 32, 200), (32, 400, 16, 150), (300, 3000, 64, 500), (40, 20000, 128, 1000)]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_fork(case):
    rows, pages, page, most = CASES[case]
    rng = np.random.default_rng(case)
    codes, scales, table, lengths, refs = _setup(rng, rows, pages, page, most)
    for parents in (rng.integers(-1, rows, rows), np.arange(rows), np.full(rows, rows - 1), np.full(rows, -1)):
        parents = parents.astype(np.int32)
        want = ref.fork(table, lengths, refs, parents, page)
        c, s = _moved(codes, scales, want[3])
        got = kv8_fork(codes, scales, *_cuda(table, lengths, parents, refs))
        for x, y in zip(got, want[:3]):
            assert np.array_equal(x.cpu().numpy(), y)
        assert int(got[3]) == want[4]
        assert torch.equal(codes, c) and torch.equal(scales, s)


def test_fork_without_room():
    rng = np.random.default_rng(9)
    codes, scales, table, lengths, refs = _setup(rng, 6, 40, 16, 50, shared=False)
    lengths[:] = 37
    table[:, :3] = np.arange(18).reshape(6, 3)
    table[:, 3:] = -1
    refs[:] = 1                                    # nothing is free but what the fork releases
    parents = np.array([2, 2, 2, 2, 2, 5], np.int32)
    want = ref.fork(table, lengths, refs, parents, 16)
    got = kv8_fork(codes, scales, *_cuda(table, lengths, parents, refs))
    assert want[4] == 0 and int(got[3]) == 0       # four sequences ended: twelve pages came free
    parents = np.array([0, 1, 2, 3, 4, 4], np.int32)
    table2, refs2 = table.copy(), refs.copy()
    refs2[:18] += 1                                # held elsewhere as well
    want = ref.fork(table2, lengths, refs2, parents, 16)
    got = kv8_fork(codes, scales, *_cuda(table2, lengths, parents, refs2))
    assert want[4] == 1 and int(got[3]) == 1 and int(got[0][5, 2]) == -1
    for x, y in zip(got, want[:3]):
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_reserve_free(case):
    rows, pages, page, most = CASES[case]
    rng = np.random.default_rng(50 + case)
    codes, scales, table, lengths, refs = _setup(rng, rows, pages, page, most)
    for extra in (np.ones(rows), rng.integers(-3, 3 * page, rows), np.full(rows, 10 * most)):
        extra = extra.astype(np.int32)
        want = ref.reserve(table, lengths, refs, extra, page)
        got = kv8_reserve(codes, scales, *_cuda(table, lengths, extra, refs))
        for x, y in zip(got, want[:3]):
            assert np.array_equal(x.cpu().numpy(), y)
        assert int(got[3]) == want[3]
    drop = rng.random(rows) < 0.5
    want = ref.fork(table, lengths, refs, np.where(drop, -1, np.arange(rows)), page)
    got = kv8_free(codes, scales, *_cuda(table, lengths, drop, refs))
    for x, y in zip(got, want[:3]):
        assert np.array_equal(x.cpu().numpy(), y)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_compact(case):
    rows, pages, page, most = CASES[case]
    rng = np.random.default_rng(70 + case)
    codes, scales, table, lengths, refs = _setup(rng, rows, pages, page, most)
    want = ref.compact(table, lengths, refs, page)
    c, s = _moved(codes, scales, want[2])
    got = kv8_compact(codes, scales, *_cuda(table, lengths, refs))
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
    assert int(got[2]) == want[3]
    assert torch.equal(codes, c) and torch.equal(scales, s)
    # once more: nothing moves
    again = kv8_compact(codes, scales, got[0], _cuda(lengths)[0], got[1])
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1]) and torch.equal(codes, c)


@pytest.mark.parametrize("full", [True, False])
def test_compact_full_and_empty(full):
    codes, scales = kv8_pool(1, 33, 1, 64, page=16)
    codes.random_(0, 256)
    before = codes.clone()
    refs = torch.full((33,), int(full), dtype=torch.int32, device="cuda")
    table, lengths = torch.full((1, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    t, r, live = kv8_compact(codes, scales, table, lengths, refs)
    assert int(live) == (33 if full else 0) and torch.equal(r, refs) and torch.equal(codes, before)


def test_copy_pages():
    rng = np.random.default_rng(1)
    codes, scales, *_ = _setup(rng, 2, 50, 32, 60, layers=3, heads=3, dim=128)
    perm = rng.permutation(50)
    moves = list(zip(perm[:20], perm[20:40]))
    c, s = _moved(codes, scales, moves)
    src, dst = _cuda(perm[:20].astype(np.int32), perm[20:40].astype(np.int32))
    kv8_copy_pages(codes, scales, src, dst)
    assert torch.equal(codes, c) and torch.equal(scales, s)
    kv8_copy_pages(codes, scales, src[:0], dst[:0])
    bad = torch.tensor([-1, 50, 3], dtype=torch.int32, device="cuda")
    kv8_copy_pages(codes, scales, bad, torch.tensor([4, 5, 99], dtype=torch.int32, device="cuda"))  # no pages: skipped
    assert torch.equal(codes, c)


def test_refusals():
    codes, scales = kv8_pool(1, 8, 1, 64, page=16)
    table, lengths = torch.full((2, 2), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    refs = torch.zeros(8, dtype=torch.int32, device="cuda")
    for bad, kind in [
        (lambda: kv8_fork(codes[0], scales, table, lengths, lengths, refs), ValueError),
        (lambda: kv8_fork(codes, scales, table, lengths, lengths[:1], refs), ValueError),
        (lambda: kv8_fork(codes, scales, table, lengths, lengths, refs[:4]), ValueError),
        (lambda: kv8_fork(codes, scales, table, lengths.long(), lengths, refs), ValueError),
        (lambda: kv8_free(codes, scales, table, lengths, lengths, refs), ValueError),
        (lambda: kv8_compact(codes, scales, table[:, 0], lengths, refs), ValueError),
        (lambda: kv8_compact(codes, scales, table, lengths, refs, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), GdnError),
        (lambda: kv8_copy_pages(codes, scales, lengths, lengths[:1]), ValueError),
    ]:
        with pytest.raises(kind):
            bad()

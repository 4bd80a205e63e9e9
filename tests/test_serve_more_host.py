"""Host side of rotary append, attention over shared tokens and logits: structures, refusals before any CUDA call, oracle pins."""
import ctypes
import os
import re

import numpy as np
import pytest

from gated_delta_rule_54_gb300 import _lib, serve
from gated_delta_rule_54_gb300._lib import GdnKv8Problem, GdnKv8Rotary, GdnLogitsProblem
from oracle import serve as ref

A = 4096  # an address that is never followed: the calls are refused
CSRC = os.path.join(os.path.dirname(os.path.abspath(_lib.__file__)), "csrc")


def test_packed_structures():
    b = serve._ROTARY(1, 2, 3, 4, 5, 6)
    assert len(b) == ctypes.sizeof(GdnKv8Rotary)
    w = GdnKv8Rotary.from_buffer_copy(b)
    assert [getattr(w, n) for n, _ in GdnKv8Rotary._fields_] == [1, 2, 3, 4, 5, 6]
    b = serve._LOGITS(*range(1, 8))
    assert len(b) == ctypes.sizeof(GdnLogitsProblem) and GdnLogitsProblem.from_buffer_copy(b).dtype == 7


def _kv8(**kw):
    return GdnKv8Problem(**{**dict(pages=10, rows=4, total=12, tokens=3, cols=4, heads=2, group=4, dim=128, page=64, mode=1, dtype=0,
                                   causal=1, window=0, scale=0.1, cu_seqlens=None, x_row=4096, x_token=1024, x_head=128), **kw})


def _rotary(**kw):
    return GdnKv8Rotary(**{**dict(positions=100, q_row=1024, q_token=1024, q_head=128, dim=128, interleaved=0), **kw})


def test_rotary_refusals():
    f = _lib.load().gdn_kv8_append_rotary
    good = [A] * 10
    call = lambda p, w, args: f(ctypes.byref(p), None if w is None else ctypes.byref(w), *args, None)
    for p, w, code in [
        (_kv8(dim=96), _rotary(), -3), (_kv8(dtype=2), _rotary(), -2), (_kv8(total=11), _rotary(), -1), (_kv8(), None, -1),
        (_kv8(), _rotary(positions=-1), -1), (_kv8(), _rotary(interleaved=2), -1), (_kv8(), _rotary(dim=0), -3), (_kv8(), _rotary(dim=-16), -3),
        (_kv8(), _rotary(dim=8), -3), (_kv8(), _rotary(dim=144), -3), (_kv8(dim=64), _rotary(dim=80), -3), (_kv8(), _rotary(q_head=4), -7),
        (_kv8(), _rotary(q_token=1), -7), (_kv8(v_token=4), _rotary(), -7),
    ]:
        assert call(p, w, good) == code
    assert f(None, ctypes.byref(_rotary()), *good, None) == -1
    # q, k, v, cos, sin, codes, scales, table, start, q_out
    for i in range(10):
        assert call(_kv8(), _rotary(), good[:i] + [None] + good[i + 1:]) == -1
    for i, by in enumerate((8, 8, 8, 8, 8, 8, 2, 2, 2, 8)):
        assert call(_kv8(), _rotary(), good[:i] + [A + by] + good[i + 1:]) == -7
    assert call(_kv8(total=0, tokens=0), _rotary(), [None] * 10) == 0


def test_shared_refusals():
    lib = _lib.load()
    f, size = lib.gdn_kv8_attention_shared, lib.gdn_kv8_shared_workspace_bytes
    need = size(ctypes.byref(_kv8()), 2)
    assert need > 0
    good = [A] * 8 + [1 << 12]
    call = lambda p, beams, args, room: f(ctypes.byref(p), beams, *args, room, None)
    for p, beams, code in [
        (_kv8(), 0, -1), (_kv8(), -1, -1), (_kv8(), 3, -1), (_kv8(cu_seqlens=A), 2, -1), (_kv8(window=5), 2, -4), (_kv8(dim=32), 2, -3),
        (_kv8(rows=1 << 28, total=3 << 28, heads=1, group=64), 1 << 28, -3), (_kv8(dtype=1), 2, -2),
    ]:
        assert call(p, beams, good[:8] + [A], 1 << 40) == code
        assert size(ctypes.byref(p), beams) == 0
    # q, codes, scales, table, lengths, shared, o (lse may be absent)
    for i in range(7):
        assert call(_kv8(), 2, good[:i] + [None] + good[i + 1:8] + [A], need) == -1
    for i, by in enumerate((8, 8, 2, 2, 2, 2, 8, 2)):
        assert call(_kv8(), 2, good[:i] + [A + by] + good[i + 1:8] + [A], need) == -7
    assert call(_kv8(), 2, good[:8] + [A + 16], need) == -7
    assert call(_kv8(), 2, good[:8] + [A], need - 1) == -5
    assert call(_kv8(), 2, good[:8] + [None], need) == -5
    assert call(_kv8(rows=0, total=0), 2, [None] * 9, 0) == 0


def test_logits_refusals():
    lib = _lib.load()
    base = dict(rows=4, stride=100, bias_row=0, mask_row=0, vocab=100, cols=8, dtype=0)
    prob = lambda **kw: GdnLogitsProblem(**{**base, **kw})
    for kw, code in [({}, 0), (dict(rows=0), 0), (dict(rows=1, stride=0), 0), (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(cols=-1), -1),
                     (dict(stride=99), -1), (dict(dtype=1), -2), (dict(dtype=9), -1), (dict(bias_row=99), -1), (dict(bias_row=-5), -1),
                     (dict(mask_row=3), -1), (dict(mask_row=4, bias_row=100, dtype=2), 0), (dict(rows=1 << 30), -3), (dict(stride=1 << 40), -3)]:
        assert lib.gdn_beam_logits_validate(ctypes.byref(prob(**kw))) == code, kw
    assert lib.gdn_beam_logits_validate(None) == -1
    f = lambda p, *a: lib.gdn_beam_logits(ctypes.byref(p), *a, None)
    B = A + (1 << 20)
    # logits, tokens, lengths, repetition, frequency, presence, bias, mask, out
    assert f(prob(), None, A, A, A, A, A, A, A, B) == -1
    assert f(prob(), A, A, A, A, A, A, A, A, None) == -1
    assert f(prob(), A, None, A, A, None, None, None, None, B) == -1       # penalties without tokens
    assert f(prob(), A + 1, A, A, A, A, A, A, A, B) == -7
    for i in range(1, 8):
        args = [A] * 8
        args[i] = A + 2
        assert f(prob(), *args, B) == -7
    assert f(prob(), A, None, None, None, None, None, None, None, A + 2) == -1   # onto itself, one element on
    assert f(prob(stride=104), A, None, None, None, None, None, None, None, A) == -1
    assert f(prob(rows=0), *[None] * 9) == 0


def test_logits_history_stays_in_32_bits():
    """A thread goes through a history by 32-bit indices, some thousand tokens ahead of it."""
    lib = _lib.load()
    prob = lambda cols: GdnLogitsProblem(rows=1, stride=100, bias_row=0, mask_row=0, vocab=100, cols=cols, dtype=0)
    assert lib.gdn_beam_logits_validate(ctypes.byref(prob(0x7fffffff - 65536))) == 0
    for cols in (0x7fffffff - 65535, 0x7fffffff):
        assert lib.gdn_beam_logits_validate(ctypes.byref(prob(cols))) == -3


def test_dependent_launches_wait_before_any_return():
    """A kernel that may start before its predecessor ends orders the rest of the stream behind it
    only by its own wait, so no thread leaves before that."""
    with open(os.path.join(CSRC, "kv8_shared.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernels = [k for k in re.split(r"__global__", text)[1:] if "grid_dep_wait()" in k]
    assert kernels
    for k in kernels:
        assert not re.search(r"\breturn;", k[k.index("{"):k.index("grid_dep_wait()")])


# ---- the oracle's own pins -------------------------------------------------
def test_oracle_turn():
    x = np.zeros((2, 1, 4), np.float32)
    x[:, 0] = [1, 2, 3, 4]
    cos, sin = np.array([[1, 1], [0, 0.5]], np.float32), np.array([[0, 0], [1, 0.5]], np.float32)
    assert ref.turn(x, [0, 1], cos, sin, False)[:, 0].tolist() == [[1, 2, 3, 4], [-3, -1, 1, 3]]
    assert ref.turn(x, [0, 1], cos, sin, True)[1, 0].tolist() == [-2, 1, -0.5, 3.5]
    assert np.isnan(ref.turn(x, [0, 2], cos, sin, False)[1]).all()
    y = ref.turn(x, [1, 1], cos[:, :1], sin[:, :1], False)
    assert y[0, 0].tolist() == [-2, 1, 3, 4]


@pytest.mark.parametrize("shared", [0, 5, 16, 23, 40])
def test_oracle_shared_attention_is_attention_over_one_copy(shared):
    rng = np.random.default_rng(shared)
    codes = rng.integers(0, 120, (2, 6, 1, 16, 64)).astype(np.uint8)
    scales = rng.random((2, 6, 1)).astype(np.float32)
    first, own, q = np.array([0, 1, 2]), np.array([3, 4, 5]), rng.standard_normal((2, 2, 64))
    joined = codes.copy()
    both = scales.copy()
    whole = shared // 16
    for c in range(whole):
        joined[:, 3 + c], both[:, 3 + c] = codes[:, c], scales[:, c]
    got = ref.attention_shared(q, codes, scales, first, own, shared, 44, "e4m3", 0.1)
    if shared % 16 == 0:
        want = ref.attention(q, joined, both, own, 44, "e4m3", 0.1)
        assert np.allclose(got[0], want[0], rtol=1e-12) and np.allclose(got[1], want[1], rtol=1e-12)
    else:  # a page of which a part is the first row's: its scale counts for that part
        table = np.array([whole, 3 + whole])
        k = np.concatenate([ref.decode_codes(codes[0, c], "e4m3")[0] * scales[0, c, 0] for c in table])
        assert got[0].shape == q.shape and np.isfinite(got[1]).all() and k.shape == (32, 64)


def test_oracle_logits_hand_case():
    x = np.array([[4.0, -4.0, 1.0, 0.0]])
    got = ref.beam_logits(x, [[0, 1, 1, 7, -1, 2]], [5], [2.0], [0.5], [0.25], np.array([[0, 0, 0, 1.0]]), np.array([[True, True, False, True]]))
    assert got.tolist() == [[2 - 0.75, -8 - 1.25, -np.inf, 1.0]]

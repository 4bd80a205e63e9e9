"""Host side of the serving operators: C structures, refusals before any CUDA call, the oracle's pins."""
import ctypes
import struct

import numpy as np
import pytest

from gated_delta_rule_54_gb300 import _lib, serve
from gated_delta_rule_54_gb300._lib import GdnBeamProblem, GdnKv8Pool, GdnKv8Problem
from oracle import serve as ref


def test_packed_problems_match_the_structures():
    b = serve._KV8(1, 2, 3, 4, 5, 6, 7, 64, 16, 1, 0, 1, 9, 0.5, 4096, *range(8, 56, 8))
    assert len(b) == ctypes.sizeof(GdnKv8Problem)
    p = GdnKv8Problem.from_buffer_copy(b)
    assert [getattr(p, n) for n, _ in GdnKv8Problem._fields_] == [1, 2, 3, 4, 5, 6, 7, 64, 16, 1, 0, 1, 9, 0.5, 4096, *range(8, 56, 8)]
    b = serve._POOL(*range(1, 8))
    assert len(b) == ctypes.sizeof(GdnKv8Pool) and GdnKv8Pool.from_buffer_copy(b).dim == 7
    b = serve._BEAM(*range(1, 8))
    assert len(b) == ctypes.sizeof(GdnBeamProblem) and GdnBeamProblem.from_buffer_copy(b).eos == 7
    assert struct.calcsize("P") == 8


def _kv8(**kw):
    p = GdnKv8Problem(pages=10, rows=2, total=6, tokens=3, cols=4, heads=2, group=4, dim=128, page=64, mode=1, dtype=0,
                      causal=1, window=0, scale=0.1, cu_seqlens=None, x_row=4096, x_token=1024, x_head=128)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(total=0, rows=0), 0), (dict(cu_seqlens=4096, total=5), 0), (dict(page=16, dim=64, mode=2), 0),
    (dict(total=5), -1), (dict(rows=-1), -1), (dict(heads=0), -1), (dict(group=0), -1), (dict(window=-1), -1),
    (dict(causal=2), -1), (dict(mode=7), -1), (dict(dtype=9), -1), (dict(scale=float("inf")), -1),
    (dict(scale=float("nan")), -1), (dict(dtype=1), -2), (dict(dtype=2), -2), (dict(dim=96), -3), (dict(page=8), -3),
    (dict(page=256), -3), (dict(pages=1 << 31), -3), (dict(cols=1 << 30), -3), (dict(pages=1 << 30, heads=2), -3),
    (dict(heads=1 << 15), -3), (dict(mode=0), -4), (dict(x_token=1025), -7), (dict(v_head=4), -7),
])
def test_kv8_validate(kw, code):
    assert _lib.load().gdn_kv8_validate(ctypes.byref(_kv8(**kw))) == code
    if code:
        assert _lib.load().gdn_kv8_workspace_bytes(ctypes.byref(_kv8(**kw))) == 0
        assert _lib.load().gdn_kv8_attention(ctypes.byref(_kv8(**kw)), *[None] * 8, 0, None) == code
        assert _lib.load().gdn_kv8_append(ctypes.byref(_kv8(**kw)), *[None] * 7) == code


def test_kv8_null_and_misaligned_pointers():
    lib, p = _lib.load(), ctypes.byref(_kv8(group=1))
    A = 4096                                       # an address that is never followed: the call is refused
    assert lib.gdn_kv8_validate(None) == -1
    assert lib.gdn_kv8_append(p, None, A, A, A, A, A, None) == -1
    assert lib.gdn_kv8_append(p, A + 2, A, A, A, A, A, None) == -7
    assert lib.gdn_kv8_append(p, A, A, A + 8, A, A, A, None) == -7
    assert lib.gdn_kv8_append(p, A, A, A, A + 1, A, A, None) == -7
    assert lib.gdn_kv8_attention(p, None, A, A, A, A, A, None, None, 0, None) == -1
    assert lib.gdn_kv8_attention(p, A, None, A, A, A, A, None, None, 0, None) == -1
    assert lib.gdn_kv8_attention(p, A, A, A, A, A, A + 8, None, None, 0, None) == -7
    big = _kv8(group=1, cols=4000)
    assert lib.gdn_kv8_workspace_bytes(ctypes.byref(big)) > 0
    assert lib.gdn_kv8_attention(ctypes.byref(big), A, A, A, A, A, A, None, None, 0, None) == -5


def test_pool_and_beam_refusals():
    lib, A = _lib.load(), 4096
    pool = dict(pages=10, rows=3, cols=4, page=16, planes=2, heads=1, dim=64)
    ok = GdnKv8Pool(**pool)
    need = lib.gdn_kv8_pool_workspace_bytes(ctypes.byref(ok))
    assert need > 0
    for kw in (dict(rows=0), dict(pages=-1), dict(page=10), dict(dim=32), dict(rows=5000), dict(planes=0), dict(cols=1 << 28)):
        assert lib.gdn_kv8_pool_workspace_bytes(ctypes.byref(GdnKv8Pool(**{**pool, **kw}))) == 0
    r = ctypes.byref(ok)
    assert lib.gdn_kv8_fork(r, A, A, A, A, A, A, A, A, A, A, A, A, need, None) == -1      # parents and drop
    assert lib.gdn_kv8_fork(r, A, A, A, A, A, None, None, A, A, A, A, A, need, None) == -1
    assert lib.gdn_kv8_fork(r, A, A, A, A, A, A, None, A, 2 * A, 2 * A, A, A, need, None) == -1  # table onto itself
    assert lib.gdn_kv8_fork(r, A, A, A, A, A, A, None, 2 * A, 2 * A, 2 * A, A, A, need - 1, None) == -5
    assert lib.gdn_kv8_compact(r, A, A, A, None, A, 2 * A, 2 * A, A, A, need, None) == -1
    assert lib.gdn_kv8_copy_pages(r, A, A, A, A, -1, None) == -1
    assert lib.gdn_kv8_copy_pages(r, A, A, None, None, 0, None) == 0
    beam = dict(batch=2, stride=100, beams=4, vocab=100, k=4, dtype=0, eos=2)
    assert lib.gdn_beam_validate(ctypes.byref(GdnBeamProblem(**beam))) == 0
    for kw, code in ((dict(stride=99), -1), (dict(vocab=0), -1), (dict(beams=33), -3), (dict(k=0), -3), (dict(dtype=1), -2),
                     (dict(dtype=5), -1), (dict(eos=100), -1), (dict(eos=-2), -1), (dict(batch=-1), -1)):
        assert lib.gdn_beam_validate(ctypes.byref(GdnBeamProblem(**{**beam, **kw}))) == code
    p = ctypes.byref(GdnBeamProblem(**beam))
    assert lib.gdn_beam_select(p, None, A, None, A, A, A, A, A, 1 << 20, None) == -1
    assert lib.gdn_beam_select(p, A + 1, A, None, A, A, A, A, A, 1 << 20, None) == -7
    assert lib.gdn_beam_select(p, A, A, None, A, A, A, A, A, 8, None) == -5
    q = lambda *v: struct.pack("%dQ" % len(v), *v)
    assert lib.gdn_beam_reorder(1, q(A), q(A), q(24), A, 4, 2, None) == -3
    assert lib.gdn_beam_reorder(1, q(A), q(A + 32), q(16), A, 4, 2, None) == -1   # overlap
    assert lib.gdn_beam_reorder(1, q(A + 8), q(A + 8), q(16), A, 4, 2, None) == -7
    assert lib.gdn_beam_reorder(1, q(A), q(A), q(16), A, 4, 33, None) == -3
    assert lib.gdn_beam_reorder(0, None, None, None, None, 4, 2, None) == 0


# ---- the oracle's own pins -------------------------------------------------
def test_oracle_codes():
    import oracle
    x = np.concatenate([np.linspace(-1, 1, 4001), [0.0, -0.0]]).astype(np.float32).reshape(1, 1, -1)
    for mode in ("e4m3", "int8"):
        y, s, c = oracle.qdq_groups(x, x.size, mode, with_codes=True)   # the C quantizer of the other operators
        rcp = np.float32(1) / s.ravel()[0]
        assert np.array_equal(ref.encode(x.ravel() * rcp, mode), c.ravel())
        assert np.allclose(ref.decode_codes(c.ravel(), mode) * s.ravel()[0], y.ravel(), rtol=1e-6, atol=0)


def test_oracle_attention_hand_case():
    codes, scales = np.zeros((2, 1, 1, 16, 64), np.uint8), np.ones((2, 1, 1), np.float32)
    codes[0, 0, 0, :3, 0] = [0, 1, 2]              # int8: keys 0, 1, 2 along dim 0
    codes[1, 0, 0, :3, 1] = [10, 20, 40]
    q = np.zeros((2, 1, 64))
    q[:, 0, 0] = np.log(2)                          # weights 1, 2, 4
    o, lse, *_ = ref.attention(q, codes, scales, np.array([0]), 3, "int8", 1.0)
    assert np.allclose(o[:, 0, 1], [(10 + 40) / 3, (10 + 40 + 160) / 7]) and np.allclose(lse[:, 0], np.log([3, 7]))
    o, lse, *_ = ref.attention(q, codes, scales, np.array([0]), 1, "int8", 1.0)
    assert np.all(o[0] == 0) and lse[0, 0] == -np.inf and np.allclose(o[1, 0, 1], 10)
    o, *_ = ref.attention(q, codes, scales, np.array([0]), 3, "int8", 1.0, window=1)
    assert np.allclose(o[:, 0, 1], [20, 40])


def test_oracle_pages_and_beams_hand_cases():
    table = np.array([[2, 5, -1], [7, -1, -1]], np.int32)
    refs = np.array([0, 0, 1, 0, 0, 1, 0, 1], np.int32)
    out, lens, new, moves, missing = ref.fork(table, [20, 16], refs, [0, 0], 16)
    assert out.tolist() == [[2, 5, -1], [2, 0, -1]] and lens.tolist() == [20, 20] and moves == [(5, 0)] and missing == 0
    assert new.tolist() == [1, 0, 2, 0, 0, 1, 0, 0]
    out, new, moves, n = ref.compact(table, [20, 16], refs, 16)
    assert n == 3 and moves == [(5, 0), (7, 1)] and out.tolist() == [[2, 0, -1], [1, -1, -1]]
    assert new.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    out, lens, new, missing = ref.reserve(table, [20, 16], refs, [12, 1], 16)
    assert out.tolist() == [[2, 5, -1], [7, 0, -1]] and lens.tolist() == [32, 17] and missing == 0
    x = np.log(np.array([[[0.5, 0.3, 0.2], [0.9, 0.05, 0.05]]]))
    best, parents, tokens, done = ref.beam_select(x, np.log([[0.6, 0.4]]), np.zeros((1, 2), bool), 2, 1)
    assert tokens.tolist() == [[0, 0]] and parents.tolist() == [[1, 0]] and np.allclose(np.exp(best), [[0.36, 0.3]])
    best, parents, tokens, done = ref.beam_select(x, np.log([[0.6, 0.4]]), np.array([[True, False]]), 2, 1)
    assert tokens.tolist() == [[1, 0]] and parents.tolist() == [[0, 1]] and done.tolist() == [[True, False]]

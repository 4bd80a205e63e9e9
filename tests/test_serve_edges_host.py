"""Host side of the serving operators' corners: what is refused, and what the sources have to keep."""
import ctypes
import os
import re

import pytest

from gated_delta_rule_54_gb300 import _lib

CSRC = os.path.join(os.path.dirname(os.path.abspath(_lib.__file__)), "csrc")


@pytest.mark.parametrize("name", ["kv8_decode.cu", "kv8_pages.cu", "beam.cu"])
def test_dependent_launches_wait_before_any_return(name):
    """A kernel that may start before its predecessor ends orders the rest of the stream behind it
    only by its own wait, so no thread leaves before that."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernels = [k for k in re.split(r"__global__", text)[1:] if "grid_dep_wait()" in k]
    assert kernels
    for k in kernels:
        assert not re.search(r"\breturn\b", k[:k.index("grid_dep_wait()")])


def test_parts_stay_in_the_cta_where_a_wait_gave_up():
    """With a CTA per segment the call has no workspace, and a part that is not whole would be
    stored through a null pointer: the CTA has to leave before it looks for a place for one."""
    with open(os.path.join(CSRC, "kv8_decode.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("kv8_decode_kernel("):text.index("kv8_join_kernel(")]
    gone = body.index("if (__syncthreads_or(bad)) return;")
    assert body.index("s_u0[warp] = part;") < gone < body.index("slot = a.ws")


def test_reorder_refuses_buffers_that_meet():
    """All states move in one launch without order, so what one writes no other may read or write."""
    import struct
    lib, A, row, rows = _lib.load(), 1 << 20, 64, 4
    q = lambda v: struct.pack("%dQ" % len(v), *v)

    def call(src, dst, sizes=None):
        return lib.gdn_beam_reorder(len(src), q(src), q(dst), q(sizes or [row] * len(src)), 4096, rows, 2, None)

    a, b, c, d = (A + i * row * rows for i in range(4))
    bad = -1
    assert call([a, b], [b, a]) == bad                       # swapped
    assert call([a, b], [c, c]) == bad                       # one buffer for two
    assert call([a, a], [a, a]) == bad                       # one state twice, in place
    assert call([a, b], [b, b]) == bad
    assert call([a, b], [a + row, d]) == bad                 # a shifted overlap of its own
    assert call([a, b, d], [c, b + row, d]) == bad           # and of another's
    assert call([a, c], [b, a + 3 * row], [row, row]) == bad
    many = [A + i * row * rows for i in range(200)]
    assert call(many, many[1:] + [many[0]]) == bad
    assert call([a], [4096]) == bad                          # the parents
    # (no device here, or an address that is not one: what is apart comes as far as the launch, and is not tried)
    assert call([a, b], [c, d], [24, 24]) == -3


def _kv8(**kw):
    p = _lib.GdnKv8Problem(pages=10, rows=2, total=2, tokens=1, cols=4, heads=2, group=4, dim=128, page=64, mode=1, dtype=0,
                           causal=1, window=0, scale=0.1, cu_seqlens=None, x_row=1024, x_token=1024, x_head=128)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("tokens", [1, 40])
def test_attention_needs_a_table_of_columns(tokens):
    """A table with columns is read even where the cache has no pages."""
    lib, A = _lib.load(), 4096
    p = ctypes.byref(_kv8(pages=0, tokens=tokens, total=2 * tokens))
    assert lib.gdn_kv8_attention(p, A, None, None, None, A, A, None, A, 1 << 40, None) == -1


@pytest.mark.parametrize("cols,page,code", [((1 << 27) - 1, 16, -3), ((1 << 24) - 1, 128, -3), ((1 << 27) - 4095, 16, -3),
                                            ((1 << 27) - 4096, 16, 0), ((1 << 24) - 512, 128, 0)])
def test_positions_leave_room_to_round_up(cols, page, code):
    """Positions are 32-bit and the kernels round them up to tiles of keys: a table whose last
    positions would pass 2^31 there is refused."""
    assert _lib.load().gdn_kv8_validate(ctypes.byref(_kv8(cols=cols, page=page))) == code


def test_scores_are_read_before_they_are_written_over():
    """Two threads read the halves of a row of S, and both write P over its first half: the
    barrier between these orders TMEM accesses of different threads only with its fences."""
    with open(os.path.join(CSRC, "kv8_prefill.cu")) as f:
        text = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", f.read()))
    read, write = text.index("tmem_ld32(s_col + half * HK, v[0]);"), text.index("tmem_st16(s_col + half * (HK / 2)")
    assert "tc_fence_before(); pair_sync(); tc_fence_after();" in text[read:write]


def test_tmem_loads_are_waited_for_in_one_piece():
    """What a tcgen05.ld gives may be used after its wait only.  A wait in a statement of its own
    does not say so to the compiler, unless the values pass through it."""
    for name in ("tc.cuh", "kv8_prefill.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for piece in re.findall(r"asm volatile\((.*?)\);\n", text, re.S):
            if "tcgen05.wait::ld" in piece:
                assert "tcgen05.ld" in piece or '"+f"' in piece

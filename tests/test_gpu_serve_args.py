"""GPU: what the serving operators' Python entry points take and refuse beside their tensors' types."""
import pytest
import torch

from gated_delta_rule_54_gb300 import (beam_reorder, beam_select, kv8_append, kv8_attention, kv8_compact, kv8_fork,
                                       kv8_free, kv8_pool, kv8_reserve, kv8_workspace_bytes)

pytestmark = pytest.mark.gpu


def _calls():
    codes, scales = kv8_pool(1, 8, 2, 64, page=16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lengths, refs = torch.full((2, 400), -1, **i32), torch.zeros(2, **i32), torch.zeros(8, **i32)
    q = torch.randn(2, 1, 4, 64, device="cuda").to(torch.bfloat16)
    x, s = torch.randn(1, 2, 50, device="cuda"), torch.zeros(1, 2, device="cuda")
    drop = torch.zeros(2, dtype=torch.bool, device="cuda")
    args = (codes, scales, table, lengths)
    return [lambda ws: kv8_attention(q, codes[0], scales[0], table, lengths, workspace=ws),
            lambda ws: kv8_fork(*args, lengths, refs, workspace=ws), lambda ws: kv8_free(*args, drop, refs, workspace=ws),
            lambda ws: kv8_reserve(*args, lengths, refs, workspace=ws), lambda ws: kv8_compact(*args, refs, workspace=ws),
            lambda ws: beam_select(x, s, workspace=ws)], kv8_workspace_bytes(q, codes[0], scales[0], table, lengths)


def test_workspaces():
    """A workspace is on the device and contiguous, and counts by its bytes."""
    calls, need = _calls()
    assert 0 < need < 1 << 24
    room = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for call in calls:
        for bad in (torch.empty(1 << 24, dtype=torch.uint8), room[::2], room[:1].expand(1 << 24), 1 << 24):
            with pytest.raises(ValueError):
                call(bad)
    exact = torch.empty(-(-need // 8), dtype=torch.int64, device="cuda")
    calls[0](exact)
    for call in calls:
        call(room.view(torch.float32))
    torch.cuda.synchronize()


def test_tensors_of_too_few_dims():
    """Tensors with dims missing are refused in words."""
    codes, scales = kv8_pool(1, 8, 2, 64, page=16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, n, cu = torch.full((2, 4), -1, **i32), torch.zeros(2, **i32), torch.zeros(3, **i32)
    for shape in ((), (64,), (4, 64), (2, 4, 64), (1, 2, 1, 4, 64)):
        q = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        for offsets in (None, cu):
            if offsets is not None and len(shape) == 3:
                continue
            with pytest.raises(ValueError):
                kv8_attention(q, codes[0], scales[0], table, n, cu_seqlens=offsets)
            with pytest.raises(ValueError):
                kv8_append(q, q, codes[0], scales[0], table, n, cu_seqlens=offsets)
    parents = torch.zeros(1, **i32)
    with pytest.raises(ValueError):
        beam_reorder([torch.zeros((), device="cuda")], parents, 1)

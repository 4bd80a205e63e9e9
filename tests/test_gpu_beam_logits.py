"""GPU: penalties, biases and masks on logits against the oracle in 64 bits.

Tolerances.  A logit goes through up to five fp32 roundings (the penalty's quotient or
product, frequency * n, two differences, the bias), each off by 2^-24 of a number no larger
than the sum of the parts' magnitudes, and one rounding to bf16 (2^-8 of the result)
where that is the type.  What the mask forbids, and what nothing touches, is exact."""
import numpy as np
import pytest
import torch

from gated_delta_rule_54_gb300 import GdnError, beam_logits, beam_select
from oracle import serve as ref

pytestmark = pytest.mark.gpu

INF = float("inf")


def _words(allowed):
    rows, v = allowed.shape
    bits = np.zeros((rows, -(-v // 32) * 32), np.uint8)
    bits[:, :v] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32).view(np.int32)


CASES = [
    # batch, beams, vocab, dtype, history, penalties, bias (1: one for all, 2: per row), allowed (None: no mask), one mask for all
    (1, 1, 1, "f32", 3, "rfp", 0, None, False),
    (1, 4, 32000, "bf16", 500, "rfp", 0, None, False),
    (2, 3, 50, "bf16", 40, "r", 1, 0.5, False),
    (2, 2, 1003, "f32", 700, "fp", 2, 0.1, True),
    (3, 1, 4099, "bf16", 0, "", 1, 0.02, False),
    (1, 5, 40000, "f32", 5000, "p", 0, 0.9, False),
    (4, 8, 20008, "bf16", 100, "rf", 2, 0.99, False),
    (1, 2, 8, "f32", 0, "", 2, None, False),
    (2, 2, 33, "bf16", 9, "rfp", 0, 0.0, True),         # nothing is allowed
    (40, 4, 9001, "bf16", 33, "rfp", 1, 0.3, False),
    (40, 8, 65536, "bf16", 200, "rfp", 0, 1.0, False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_against_the_oracle(case):
    b, w, v, dtype, history, which, bias, allowed, one_mask = CASES[case]
    rng = np.random.default_rng(400 + case)
    rows = b * w
    x = torch.from_numpy(3 * rng.standard_normal((b, w, v)).astype(np.float32)).cuda()
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    tokens = (rng.random((rows, history)) ** 3 * (v + 3)).astype(np.int32) - 2      # some are no tokens
    lengths = rng.integers(-1, history + 3, rows).astype(np.int32)
    lengths[0] = history
    pen = {n: rng.uniform(0.5, 1.8, rows).astype(np.float32) if n in which else None for n in "rfp"}
    bi = None if not bias else rng.standard_normal((rows if bias == 2 else 1, v)).astype(np.float32)
    ok = None if allowed is None else rng.random((1 if one_mask else rows, v)) < allowed
    shaped = lambda a: None if a is None else torch.from_numpy(a).cuda().view(b, w, *a.shape[1:])
    args = dict(repetition=shaped(pen["r"]), frequency=shaped(pen["f"]), presence=shaped(pen["p"]))
    if history:
        args.update(tokens=shaped(tokens), lengths=shaped(lengths))
    if bi is not None:
        args["bias"] = shaped(bi) if bias == 2 else torch.from_numpy(bi[0]).cuda()
    if ok is not None:
        m = torch.from_numpy(_words(ok)).cuda()
        args["mask"] = m[0] if one_mask else m.view(b, w, -1)
    before = x.clone()
    got = beam_logits(x, **args)
    assert torch.equal(x, before) and got.dtype == x.dtype and got.is_contiguous()
    assert torch.equal(got, beam_logits(x, **args))
    host = x.float().cpu().numpy().reshape(rows, v).astype(np.float64)
    full = lambda a: None if a is None else np.broadcast_to(a, (rows, v))
    want = ref.beam_logits(host, tokens if history and which else None, lengths, pen["r"], pen["f"], pen["p"], full(bi), full(ok))
    g = got.float().cpu().numpy().reshape(rows, v).astype(np.float64)
    gone = np.isneginf(want)
    assert np.array_equal(np.isneginf(g), gone)
    size = np.abs(host) * 2 + (history * 1.8 if "f" in which else 0) + 2 + (np.abs(full(bi)) if bi is not None else 0)
    tol = 5 * 2.0 ** -24 * size + (1.01 * 2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    err = np.abs(g[~gone] - want[~gone])
    assert np.all(err <= tol[~gone]) if dtype == "bf16" or which or bi is not None else np.all(err == 0)
    inplace = x.clone()
    assert beam_logits(inplace, out=inplace, **args) is inplace
    assert torch.equal(inplace, got)


def test_definition_bit_for_bit():
    """fp32 logits and a plain restatement with every rounding."""
    rng = np.random.default_rng(3)
    rows, v, n = 4, 999, 60
    x, f32 = (4 * rng.standard_normal((rows, v))).astype(np.float32), np.float32
    tokens = rng.integers(0, 80, (rows, n)).astype(np.int32)
    r, f, p = (rng.uniform(0.1, 2, rows).astype(f32) for _ in range(3))
    want = x.copy()
    for i in range(rows):
        t, c = np.unique(tokens[i], return_counts=True)
        y = want[i, t]
        y = np.where(y > 0, (y / r[i]).astype(f32), (y * r[i]).astype(f32))
        want[i, t] = ((y - (f[i] * c.astype(f32)).astype(f32)).astype(f32) - p[i]).astype(f32)
    cuda = lambda a: torch.from_numpy(a).cuda().view(2, 2, *a.shape[1:])
    got = beam_logits(cuda(x), cuda(tokens), None, cuda(r), cuda(f), cuda(p))
    assert np.array_equal(got.cpu().numpy().reshape(rows, v), want)


def test_what_is_no_number():
    x = torch.tensor([[[INF, -INF, float("nan"), 1.0, INF, float("nan"), -2.0, 0.0, -0.0]]], device="cuda")
    tokens = torch.tensor([[[0, 1, 2, 3, 6, 6, 7, 8, -1, 9, 1 << 30, -(1 << 31)]]], dtype=torch.int32, device="cuda")
    one = torch.ones(1, 1, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = beam_logits(x.to(dtype), tokens, None, 2 * one, 0 * one, one)
        want = torch.tensor([[[INF, -INF, float("nan"), -0.5, INF, float("nan"), -5.0, -1.0, -1.0]]], device="cuda")
        assert torch.equal(torch.nan_to_num(y.float(), nan=7.0), torch.nan_to_num(want, nan=7.0))
        mask = torch.tensor([0b010001000], dtype=torch.int32, device="cuda")
        y = beam_logits(x.to(dtype), tokens, None, 2 * one, mask=mask)
        assert torch.all(torch.isneginf(y[0, 0, [0, 1, 2, 4, 5, 6, 8]])) and y[0, 0, 3] == 0.5 and y[0, 0, 7] == 0
        low = torch.full((1, 1, 9), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        assert torch.all(torch.isneginf(beam_logits(low, tokens, None, 8 * one)[0, 0, :4]))   # goes past the type


def test_strides_and_orders():
    torch.manual_seed(4)
    wide = torch.randn(3, 4, 70, device="cuda")
    for x in (wide[:, :, 3:67], wide[:, :, :64], wide[1:2, ::2, 1:66], wide[:, 1:2, :64]):
        b, w, v = x.shape
        tokens = torch.randint(0, v, (b, w, 7), dtype=torch.int32, device="cuda")
        pres = torch.rand(b, w, device="cuda")
        bias = torch.randn(b, w, v + 5, device="cuda")[..., :v]
        words = torch.randint(-(1 << 31), 1 << 31, (w, 4), device="cuda").int().expand(b, -1, -1)
        for mask in (words[:1, :1].expand(b, w, -1), words.contiguous(), words.contiguous()[..., :(v + 31) // 32]):
            got = beam_logits(x, tokens, None, None, None, pres, bias, mask)
            want = x - pres[..., None] * torch.zeros_like(x).scatter_(2, tokens.long(), 1.0) + bias
            ok = (mask[..., None] >> torch.arange(32, device="cuda", dtype=torch.int32) & 1).flatten(-2)[..., :v]
            assert torch.equal(got, want.masked_fill(ok == 0, -INF))


def test_stream_graph_and_selection():
    """Captured, replayed on new contents, and followed by the selection, which takes only what the mask allows."""
    torch.manual_seed(5)
    x = torch.randn(2, 3, 5000, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, 5000, (2, 3, 64), dtype=torch.int32, device="cuda")
    freq, scores = torch.rand(2, 3, device="cuda"), torch.zeros(2, 3, device="cuda")
    mask = torch.zeros(2, 3, 157, dtype=torch.int32, device="cuda")
    mask[:, :, 100] = 0b1011
    want = beam_logits(x, tokens, None, None, freq, mask=mask)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = beam_logits(x, tokens, None, None, freq, mask=mask)
    side.synchronize()
    assert torch.equal(got, want)
    x2 = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = beam_logits(x2, tokens, None, None, freq, mask=mask)
        best = beam_select(y, scores)
    x2.copy_(-x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, beam_logits(-x, tokens, None, None, freq, mask=mask))
    assert set(best[2].flatten().tolist()) <= {3200, 3201, 3203}


def test_empty_and_refused():
    x = torch.zeros(2, 3, 40, device="cuda")
    t, n, f = torch.zeros(2, 3, 5, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.ones(2, 3, device="cuda")
    assert beam_logits(x[:0], t[:0], n[:0], f[:0]).shape == (0, 3, 40)
    assert beam_logits(x[:, :0]).shape == (2, 0, 40)
    assert torch.equal(beam_logits(x + 1, t[..., :0], None, f), x + 1)
    assert torch.equal(beam_logits(x + 1), x + 1)
    buf = torch.zeros(500, device="cuda")
    for bad, kind in [
        (lambda: beam_logits(x[0]), ValueError), (lambda: beam_logits(x.cpu()), ValueError), (lambda: beam_logits(x.half()), GdnError),
        (lambda: beam_logits(x.transpose(1, 2)), ValueError), (lambda: beam_logits(x.transpose(0, 1)), ValueError),
        (lambda: beam_logits(x[:, :1].expand(-1, 3, -1)), ValueError), (lambda: beam_logits(x[:1, :1].expand(1, 3, -1)), GdnError),
        (lambda: beam_logits(x[..., :0]), GdnError), (lambda: beam_logits(x, None, None, f), ValueError), (lambda: beam_logits(x, None, n), ValueError),
        (lambda: beam_logits(x, t.long(), n, f), ValueError), (lambda: beam_logits(x, t[:, :2], n, f), ValueError),
        (lambda: beam_logits(x, t[..., ::2], n, f), ValueError), (lambda: beam_logits(x, t, n.long(), f), ValueError),
        (lambda: beam_logits(x, t, n[:1], f), ValueError), (lambda: beam_logits(x, t, n, f.double()), ValueError),
        (lambda: beam_logits(x, t, n, f[0]), ValueError), (lambda: beam_logits(x, bias=x[0, 0, :39]), ValueError),
        (lambda: beam_logits(x, bias=x[:1]), ValueError), (lambda: beam_logits(x, bias=x.cpu()), ValueError),
        (lambda: beam_logits(x, mask=n), ValueError), (lambda: beam_logits(x, mask=t[0, 0, :1]), ValueError),
        (lambda: beam_logits(x, mask=t.long()), ValueError), (lambda: beam_logits(x, mask=t[0, 0, ::2]), ValueError),
        (lambda: beam_logits(x, out=x[:1]), ValueError), (lambda: beam_logits(x, out=x.bfloat16()), ValueError),
        (lambda: beam_logits(buf[:240].view(2, 3, 40), out=buf[4:244].view(2, 3, 40)), GdnError),
        (lambda: beam_logits(buf[:480].view(2, 3, 80)[..., :40], out=buf[:240].view(2, 3, 40)), GdnError),
    ]:
        with pytest.raises(kind):
            bad()
    torch.cuda.synchronize()

"""Rotary positions against 64 bits, from exact fractions of a turn.

Tolerances.  Of an angle in turns the kernel keeps 32 bits (2 pi 2^-32 < 2^-29 radians), and rounds its rest, up to pi / 4, to 24
(2^-25); the series' next terms are below 2^-28, their evaluation below three roundings of a result up to 1: sines and cosines
are off by less than 2^-22.  The amplitude and the two products add three roundings: 2^-21 of |a| + |b|.  Then half a step
of bf16 (subnormal steps: 2^-134)."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def qkv(seqs, tokens, q_heads, heads, dim, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(seqs, tokens, q_heads + 2 * heads, dim, generator=g).to(torch.bfloat16).cuda()
    return x, x[:, :, :q_heads], x[:, :, q_heads:q_heads + heads]


def check(got, x, lens, plan):
    turns = [int(t) % (1 << 64) for t in plan.turns.tolist()]
    want, spread = plain.turned(plain.f64(x), lens, turns, plan.interleaved, np.float64(np.float32(plan.amplitude)))
    off = np.abs(plain.f64(got) - want)
    by = np.where(spread > 0, spread * 2.0 ** -21 + np.abs(want) * 2.0 ** -8 + 2.0 ** -134, 0.0)
    assert (off <= by).all(), f"off by {np.max(off / np.maximum(by, 1e-300))} of what it may be"


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("seqs,tokens,q_heads,heads,dim,rotary", (
    (1, 1, 1, 1, 16, 16), (1, 1, 16, 16, 64, 64), (3, 1, 5, 1, 64, 32), (2, 7, 8, 2, 128, 128), (5, 3, 3, 3, 128, 16), (1, 33, 6, 2, 128, 96),
    (2, 5, 2, 1, 80, 48), (1, 9, 4, 4, 256, 256), (2, 4, 1, 1, 240, 16), (1, 2100, 3, 1, 64, 48), (2, 1030, 40, 8, 128, 128), (64, 1, 40, 8, 128, 64)))
def test_shapes(lib, seqs, tokens, q_heads, heads, dim, rotary, interleaved):
    say(f"rope {seqs} x {tokens}, {q_heads}/{heads} heads of {dim}, {rotary} turned, interleaved {interleaved}")
    x, q, k = qkv(seqs, tokens, q_heads, heads, dim, dim + tokens)
    lens = [tokens + 3 + 1000 * i for i in range(seqs)]
    plan = lib.rope(rotary, interleaved=interleaved)
    yq, yk = lib.w8a8_rope(q, k, torch.tensor(lens, dtype=torch.int32).cuda(), plan)
    if tokens > 1000:                                     # (the plain form is a loop: some tokens of the last sequence)
        pick = [0, 1, 511, 1023, tokens - 1]
        for t in pick:
            at = [n - tokens + t + 1 for n in lens]
            check(yq[:, t:t + 1], q[:, t:t + 1], at, plan)
            check(yk[:, t:t + 1], k[:, t:t + 1], at, plan)
    else:
        check(yq, q, lens, plan)
        check(yk, k, lens, plan)
    assert yq.is_contiguous() and yk.is_contiguous()


@pytest.mark.parametrize("scaling", (dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                     dict(scaling="wavelength", factor=8.0, original=8192), dict(scaling="yarn", factor=32.0), dict(base=1e6)))
def test_far_positions(lib, scaling):
    """Up to the last position that a length can give."""
    plan = lib.rope(64, **scaling)
    lens = [1, 2, 4096, 131072, (1 << 20) + 1, (1 << 24) + 3, (1 << 30) - 1, (1 << 31) - 1]
    x, q, k = qkv(len(lens), 1, 2, 1, 64, 5)
    yq, yk = lib.w8a8_rope(q, k, torch.tensor(lens, dtype=torch.int32).cuda(), plan)
    check(yq, q, lens, plan)
    check(yk, k, lens, plan)


def test_all_of_a_turn(lib):
    """Frequencies of every kind: none, a quarter turn, a turn less a bit, and the signs of every octant."""
    turns = [0, 1 << 62, 1 << 63, 3 << 62, (1 << 64) - 1, 1 << 61, (1 << 61) - 1, 7 << 61] + [(i << 60) + 12345 for i in range(16)]
    plan = lib.Rope(torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64).cuda(), False, 1.0)
    x, q, k = qkv(1, 40, 2, 1, 64, 6)
    yq, yk = lib.w8a8_rope(q, k, torch.tensor([40], dtype=torch.int32).cuda(), plan)
    check(yq, q, [40], plan)
    check(yk, k, [40], plan)


@pytest.mark.parametrize("tokens", (1, 6))
def test_rows_without_a_position(lib, tokens):
    """Sequences shorter than the call's tokens, empty ones and negative lengths: those rows are copied."""
    lens = [tokens + 5, 3, 0, -4, 1, tokens]
    x, q, k = qkv(len(lens), tokens, 4, 2, 64, 7)
    plan = lib.rope(64, interleaved=True)
    yq, yk = lib.w8a8_rope(q, k, torch.tensor(lens, dtype=torch.int32).cuda(), plan)
    check(yq, q, lens, plan)
    check(yk, k, lens, plan)
    assert torch.equal(yq[3], q[3]) and torch.equal(yk[2], k[2])


def test_in_place_and_given_outputs(lib):
    x, q, k = qkv(3, 5, 4, 2, 64, 8)
    lens = torch.tensor([9, 5, 2], dtype=torch.int32).cuda()
    plan = lib.rope(32)
    yq, yk = lib.w8a8_rope(q, k, lens, plan)
    v = x[:, :, 6:].clone()
    got = lib.w8a8_rope(q, k, lens, plan, out=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk) and got[0].data_ptr() == q.data_ptr()
    assert torch.equal(x[:, :, 6:], v)                                     # what lies beside them stays
    x, q, k = qkv(3, 5, 4, 2, 64, 8)
    wide = torch.zeros_like(x)
    lib.w8a8_rope(q, k, lens, plan, out=(wide[:, :, :4], wide[:, :, 4:6]))
    assert torch.equal(wide[:, :, :4], yq) and torch.equal(wide[:, :, 4:6], yk) and not wide[:, :, 6:].any()
    only, none = lib.w8a8_rope(q, None, lens, plan)
    assert torch.equal(only, yq) and none is None


def test_lengths_and_frequencies_that_begin_anywhere(lib):
    x, q, k = qkv(3, 2, 4, 2, 64, 9)
    plan = lib.rope(64)
    lens = torch.tensor([77, 9, 5, 2], dtype=torch.int32).cuda()
    odd = torch.cat((plan.turns[:1], plan.turns))[1:]
    a = lib.w8a8_rope(q, k, lens[1:], plan._replace(turns=odd))
    b = lib.w8a8_rope(q, k, lens[1:].clone(), plan)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_values_that_are_not_finite_stay_in_their_pair(lib):
    x, q, k = qkv(2, 3, 4, 2, 64, 10)
    lens, plan = torch.tensor([9, 5], dtype=torch.int32).cuda(), lib.rope(32)
    want = lib.w8a8_rope(q, k, lens, plan)[0]
    q[1, 1, 2, 3], q[0, 0, 0, 40] = float("nan"), float("inf")
    got = lib.w8a8_rope(q, k, lens, plan)[0]
    same = torch.ones_like(got, dtype=torch.bool)
    same[1, 1, 2, 3] = same[1, 1, 2, 19] = same[0, 0, 0, 40] = False
    assert torch.equal(got[same], want[same]) and got[1, 1, 2, [3, 19]].isnan().all() and got[0, 0, 0, 40] == float("inf")


def test_empty_and_refused(lib):
    plan = lib.rope(64)
    x, q, k = qkv(2, 3, 4, 2, 64, 11)
    lens = torch.tensor([9, 5], dtype=torch.int32).cuda()
    assert lib.w8a8_rope(q[:, :0], k[:, :0], lens, plan)[0].shape == (2, 0, 4, 64)
    assert lib.w8a8_rope(q[:0], k[:0], lens[:0], plan)[0].shape == (0, 3, 4, 64)
    with pytest.raises(lib.W8A8Error, match="BAD_SHAPE"):
        lib.w8a8_rope(q, k, lens, lib.rope(128))
    with pytest.raises(lib.W8A8Error, match="BAD_SHAPE"):
        lib.w8a8_rope(q, k, lens, lib.rope(8))
    with pytest.raises(lib.W8A8Error, match="BAD_ARGUMENT"):
        lib.w8a8_rope(q, k, lens, plan._replace(amplitude=float("inf")))
    with pytest.raises(ValueError, match="tokens"):
        lib.w8a8_rope(q, k[:, :2], lens, plan)
    with pytest.raises(ValueError, match="q: expected"):
        lib.w8a8_rope(q, k, lens[:1].clone(), plan)
    with pytest.raises(ValueError, match="dense"):
        lib.w8a8_rope(q[:, :, ::2], k, lens, plan)
    with pytest.raises(ValueError, match="q_out"):
        lib.w8a8_rope(q, k, lens, plan, out=(torch.empty(2, 3, 3, 64, dtype=torch.bfloat16, device="cuda"), None))
    with pytest.raises(TypeError):
        lib.w8a8_rope(q.float(), k, lens, plan)
    with pytest.raises(TypeError):
        lib.w8a8_rope(q, k, lens.long(), plan)


def test_captured_and_replayed(lib):
    """A captured call follows lens as it grows."""
    x, q, k = qkv(4, 1, 8, 2, 128, 12)
    plan, lens = lib.rope(128), torch.full((4,), 100, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q), torch.empty_like(k)
    lib.w8a8_rope(q, k, lens, plan, out=out)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        lens.add_(1)
        lib.w8a8_rope(q, k, lens, plan, out=out)
    for i in range(4):
        lens.fill_(100 + 10 * i)
        graph.replay()
        torch.cuda.synchronize()
        want = lib.w8a8_rope(q, k, torch.full((4,), 101 + 10 * i, dtype=torch.int32, device="cuda"), plan)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])

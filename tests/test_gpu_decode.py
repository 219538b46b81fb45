"""The decoder layer that runs the few-token operators together: against the same formulas in 64 bits, one
token at a time against whole prompts, and captured into a HIP graph."""
import numpy as np
import pytest
import torch

import plain_decode as P
from parity import say

pytestmark = pytest.mark.gpu

HIDDEN, Q_HEADS, HEADS, DIM, FFN, GROUP, PAGE = 512, 8, 2, 64, 640, 64, 32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    shapes = (((Q_HEADS + 2 * HEADS) * DIM, HIDDEN), (HIDDEN, Q_HEADS * DIM), (2 * FFN, HIDDEN), (HIDDEN, FFN))
    return [(torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16) for n, k in shapes]


def make(lib, few, seed=5):
    from w8a8_quantized_linear_amd.decode import DecoderLayer
    return DecoderLayer(*[w.cuda() for w in weights(seed)], Q_HEADS, HEADS, DIM, GROUP, few)


def paged(lib, seqs, length, seed=3):
    width = -(-length // PAGE)
    cache = lib.kv_cache(seqs * width + 2, HEADS, PAGE, DIM)
    table = torch.randperm(seqs * width + 2, generator=torch.Generator().manual_seed(seed))[:seqs * width]
    return cache, table.view(seqs, width).to(torch.int32).cuda()


def rel(a, b):
    a, b = (t.double().cpu().numpy() if torch.is_tensor(t) else t for t in (a, b))
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def plain(ws, x, done, k_all, v_all):
    """The layer in fp64 with unquantized weights and cache: x [seqs, tokens, hidden] after `done` tokens."""
    wqkv, wo, wgu, wd = (w.double().numpy() for w in ws)
    seqs, tokens, _ = x.shape
    qkv = (x @ wqkv.T).reshape(seqs, tokens, Q_HEADS + 2 * HEADS, DIM)
    q, k, v = np.split(qkv, (Q_HEADS, Q_HEADS + HEADS), axis=2)
    k_all, v_all = np.concatenate((k_all, k), 1), np.concatenate((v_all, v), 1)
    a = np.zeros_like(q)
    for b in range(seqs):
        for i in range(tokens):
            for h in range(Q_HEADS):
                kk, vv = (t[b, :done + i + 1, h // (Q_HEADS // HEADS)] for t in (k_all, v_all))
                s = kk @ q[b, i, h] * DIM ** -0.5
                p = np.exp(s - s.max())
                a[b, i, h] = p @ vv / p.sum()
    x = x + a.reshape(seqs, tokens, -1) @ wo.T
    g, u = np.split(x @ wgu.T, 2, axis=-1)
    return x + (g / (1 + np.exp(-g)) * u) @ wd.T, k_all, v_all


# Drift: a 4-bit weight in groups of 64 has an error of (amax / 7) / sqrt(12) for amax ~ 2.6 sigma, 0.11 of each
# projection's output; two projections in a row and their products add to ~0.2 of a branch.  The residual
# carries x itself (rms 1), beside branches of rms < 0.7: the layer's output is off by less than 0.2.  8-bit
# weights, codes and activations: 0.01 each, below 0.03 together.
@pytest.mark.parametrize("few,limit", ((1 << 20, 0.2), (0, 0.03)))
def test_layer_against_64_bits(lib, few, limit):
    seqs, prompt, steps = 3, 37, 4
    say(f"decoder layer, few={few}")
    layer, ws = make(lib, few), weights(5)
    cache, table = paged(lib, seqs, prompt + steps)
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    x = torch.randn(seqs, prompt + steps, HIDDEN, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    k_all = v_all = np.zeros((seqs, 0, HEADS, DIM))
    done = 0
    for n in (prompt,) + (1,) * steps:
        part = x[:, done:done + n]
        lens += n
        y = layer(part.cuda().contiguous(), cache, table, lens)
        ref, k_all, v_all = plain(ws, part.double().numpy(), done, k_all, v_all)
        d = rel(y, ref)
        say(f"after {done + n} tokens: drift {d:.4f}")
        assert d < limit
        done += n


def test_steps_equal_the_operators_one_by_one(lib):
    """4-bit projections of the layer are the library's calls: bitwise, and within the plain form's tolerance."""
    layer, ws = make(lib, 64), weights(5)
    cache, table = paged(lib, 2, 9)
    lens = torch.full((2,), 9, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 9, HIDDEN, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    y = layer(x, cache, table, lens)
    qkv = layer.qkv(x.view(18, HIDDEN))
    codes, scales = lib.w8a8_w4_quantize(ws[0].cuda(), GROUP)
    ref = P.w4_linear(x.view(18, HIDDEN).float().cpu().numpy(), P.w4_codes(codes.cpu().numpy(), HIDDEN),
                      scales.float().cpu().numpy(), GROUP, None)
    assert np.all(np.abs(qkv.double().cpu().numpy() - ref) <= 2 ** -8 * np.abs(ref) + 1e-3 * np.sqrt(np.mean(ref ** 2)))
    other, _ = paged(lib, 2, 9)
    q, k, v = qkv.view(2, 9, -1, DIM).split((Q_HEADS, HEADS, HEADS), dim=2)
    lib.w8a8_kv_append(k.contiguous(), v.contiguous(), other, table, lens)
    a = lib.w8a8_kv_attention(q.contiguous(), other, table, lens)
    r = x.view(18, HIDDEN) + layer.o(a.view(18, -1))
    h = layer.gateup(r)
    z = r + layer.down(lib.w8a8_swiglu(h[:, :FFN], h[:, FFN:]))
    assert torch.equal(z.view_as(y), y)


def test_a_captured_step_follows_the_lengths(lib):
    """One step captured once and replayed while lens grows, eager work between the replays: the eager step's bytes."""
    seqs, first, steps = 4, 30, 5                        # the third step opens a page
    layer = make(lib, 64)
    x = torch.randn(steps + 1, seqs, 1, HIDDEN, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    start = torch.randn(seqs, first, HIDDEN, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()

    def fresh():
        cache, table = paged(lib, seqs, first + steps)
        lens = torch.full((seqs,), first, dtype=torch.int32, device="cuda")
        layer(start, cache, table, lens)
        return cache, table, lens
    cache, table, lens = fresh()
    eager = []
    for i in range(steps):
        lens += 1
        eager.append(layer(x[i], cache, table, lens).clone())
    cache, table, lens = fresh()
    xin = x[0].clone()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        lens.add_(1)
        y = layer(xin, cache, table, lens)
    for i in range(steps):
        xin.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i]), f"replay {i} differs from the eager step"
        (x[i] * 2).sum().item()
    assert lens.tolist() == [first + steps] * seqs


def test_refuses_weights_that_disagree(lib):
    from w8a8_quantized_linear_amd.decode import DecoderLayer
    ws = [w.cuda() for w in weights(5)]
    with pytest.raises(ValueError):
        DecoderLayer(*ws, Q_HEADS, HEADS + 1, DIM, GROUP)
    layer = DecoderLayer(*ws, Q_HEADS, HEADS, DIM, GROUP)
    cache, table = paged(lib, 1, 4)
    with pytest.raises(TypeError):
        layer(torch.zeros(1, 2, HIDDEN, dtype=torch.float32, device="cuda"), cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"))

"""The decoder layer with root-mean-square norms, rotary positions and E4M3 projections with block scales: against 64 bits, against its
operators one by one, two layers chained, and as a captured step."""
import numpy as np
import pytest
import torch

import plain_layer as plain
from parity import say
from test_gpu_decode import DIM, FFN, GROUP, HEADS, HIDDEN, Q_HEADS, paged, rel, weights

pytestmark = pytest.mark.gpu

EPS = 1e-5
FORMS = (("4 bits", dict(few=1 << 20)), ("8 bits", dict(few=0)), ("blocks", dict(blocks=True)))


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def norm_weights(seed):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.2 * torch.randn(HIDDEN, generator=g)).to(torch.bfloat16) for _ in range(2)]


def make(form, seed=5):
    from w8a8_quantized_linear_amd.decode import DecoderLayer
    n1, n2 = (n.cuda() for n in norm_weights(seed))
    return DecoderLayer(*[w.cuda() for w in weights(seed)], Q_HEADS, HEADS, DIM, GROUP, norm1=n1, norm2=n2, eps=EPS, **form)


def by_norm(x, w):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * plain.f64(w)


def plain_layer(ws, norms, x, done, k_all, v_all, turns, interleaved):
    """The layer in fp64 with unquantized weights and cache: x [seqs, tokens, hidden] after `done` tokens."""
    wqkv, wo, wgu, wd = (w.double().numpy() for w in ws)
    seqs, tokens, _ = x.shape
    qkv = (by_norm(x, norms[0]) @ wqkv.T).reshape(seqs, tokens, Q_HEADS + 2 * HEADS, DIM)
    q, k, v = np.split(qkv, (Q_HEADS, Q_HEADS + HEADS), axis=2)
    q, k = (plain.turned(t, [done + tokens] * seqs, turns, interleaved, 1.0)[0] for t in (q, k))
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
    g, u = np.split(by_norm(x, norms[1]) @ wgu.T, 2, axis=-1)
    return x + (g / (1 + np.exp(-g)) * u) @ wd.T, k_all, v_all


# Drift: per weight 0.11 of a projection's output with 4-bit codes and 0.01 with 8-bit ones, as in the layer without norms; E4M3 codes
# are off by a uniform part of half a step, 2^-4 of the value at most and 0.027 rms, for weights and activations each: 0.038 of
# each projection's output.  Norms bring the branches' inputs to rms 1, as x is, so branches and limits are those of the layer
# without: 0.2 and 0.03; blocks between them by 0.038 / 0.11: 0.07.
@pytest.mark.parametrize("form,limit", (("4 bits", 0.2), ("8 bits", 0.03), ("blocks", 0.07)))
@pytest.mark.parametrize("interleaved,rotary", ((False, DIM), (True, DIM // 2)))
def test_against_64_bits(lib, form, limit, interleaved, rotary):
    seqs, prompt, steps = 3, 37, 4
    say(f"layer with norms and positions, {form}, interleaved {interleaved}, {rotary} turned")
    layer, ws, norms = make(dict(FORMS)[form]), weights(5), norm_weights(5)
    cache, table = paged(lib, seqs, prompt + steps)
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    rope = lib.rope(rotary, interleaved=interleaved)
    turns = [int(t) % (1 << 64) for t in rope.turns.tolist()]
    x = torch.randn(seqs, prompt + steps, HIDDEN, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    k_all = v_all = np.zeros((seqs, 0, HEADS, DIM))
    done = 0
    for n in (prompt,) + (1,) * steps:
        lens += n
        y = layer(x[:, done:done + n].contiguous().cuda(), cache, table, lens, rotate=rope)
        want, k_all, v_all = plain_layer(ws, norms, x[:, done:done + n].double().numpy(), done, k_all, v_all, turns, interleaved)
        off = rel(y, want)
        say(f"  {n} tokens behind {done}: off by {off:.4f}")
        assert off < limit
        done += n


@pytest.mark.parametrize("form", [f[0] for f in FORMS])
def test_one_by_one_and_chained(lib, form):
    """Bit for bit the operators one by one; and two layers chained by step, the sums left to the norms."""
    one, two = make(dict(FORMS)[form], 5), make(dict(FORMS)[form], 6)
    rope = lib.rope(DIM, scaling="linear", factor=2.0)
    (c1, table), (c2, _), (d1, _), (d2, _) = (paged(lib, 2, 30) for _ in range(4))
    done = 0
    for tokens in (29, 1):
        lens = torch.full((2,), done + tokens, dtype=torch.int32, device="cuda")
        x = torch.randn(2, tokens, HIDDEN, generator=torch.Generator().manual_seed(tokens)).to(torch.bfloat16).cuda()
        y, r = one.step(x, None, c1, table, lens, rotate=rope)
        y, r = two.step(y, r, c2, table, lens, rotate=rope)
        rows, delta = x.view(2 * tokens, HIDDEN), None
        for layer, cache in ((one, d1), (two, d2)):
            w1, w2 = layer.norm1, layer.norm2
            rows, delta = (delta, rows) if delta is not None else (rows, None)       # (what is added, to what)
            if form == "blocks":
                q, s, h = lib.w8a8_rmsnorm_quantize_block_packed(rows, w1, delta, EPS)
                qkv = lib.w8a8_fp8_block_gemm_packed(q, s, layer.qkv.w, layer.qkv.s, 2 * tokens, layer.qkv.N, HIDDEN)
            elif form == "8 bits":
                q, s, h = lib.w8a8_rmsnorm_quantize_packed(rows, w1, delta, EPS)
                qkv = lib.w8a8_gemm_dequant_packed(q, s, layer.qkv.w8, layer.qkv.s8, HIDDEN)
            else:
                n, h = lib.w8a8_rmsnorm(rows, w1, delta, EPS)
                qkv = lib.w8a8_w4_linear(n, *layer.qkv.w4, layer.qkv.N, GROUP)
            rows = rows if h is None else h
            q, k, v = qkv.view(2, tokens, -1, DIM).split((Q_HEADS, HEADS, HEADS), dim=2)
            q, k = lib.w8a8_rope(q, k, lens, rope)
            lib.w8a8_kv_append(k, v, cache, table, lens)
            a = layer.o(lib.w8a8_kv_attention(q, cache, table, lens).view(2 * tokens, -1))
            if form == "blocks":
                q, s, rows = lib.w8a8_rmsnorm_quantize_block_packed(a, w2, rows, EPS)
                g = lib.w8a8_fp8_block_gemm_packed(q, s, layer.gateup.w, layer.gateup.s, 2 * tokens, 2 * FFN, HIDDEN)
                g = lib.w8a8_swiglu(g[:, :FFN], g[:, FFN:])
            elif form == "8 bits":
                q, s, rows = lib.w8a8_rmsnorm_quantize_packed(a, w2, rows, EPS)
                g = lib.w8a8_gemm_swiglu_packed(q, s, layer.gateup.w8, layer.gateup.s8, HIDDEN)
            else:
                n, rows = lib.w8a8_rmsnorm(a, w2, rows, EPS)
                g = lib.w8a8_w4_linear(n, *layer.gateup.w4, 2 * FFN, GROUP)
                g = lib.w8a8_swiglu(g[:, :FFN], g[:, FFN:])
            delta = layer.down(g)
        assert torch.equal(y.view_as(delta), delta) and torch.equal(r.view_as(rows), rows)
        done += tokens


@pytest.mark.parametrize("form", [f[0] for f in FORMS])
def test_captured_step(lib, form):
    layer, rope = make(dict(FORMS)[form]), lib.rope(DIM)
    (cache, table), (other, _) = paged(lib, 2, 40), paged(lib, 2, 40)
    x = torch.randn(2, 30, HIDDEN, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for c in (cache, other):
        layer(x, c, table, torch.full((2,), 30, dtype=torch.int32, device="cuda"), rotate=rope)
    one, lens = x[:, :1].clone(), torch.full((2,), 30, dtype=torch.int32, device="cuda")
    spare, _ = paged(lib, 2, 40)
    layer(one, spare, table, lens, rotate=rope)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        lens.add_(1)
        y = layer(one, cache, table, lens, rotate=rope)
    lens.fill_(30)
    for i in range(5):
        one.copy_(x[:, i:i + 1])
        graph.replay()
        torch.cuda.synchronize()
        want = layer(x[:, i:i + 1].contiguous(), other, table, torch.full((2,), 31 + i, dtype=torch.int32, device="cuda"), rotate=rope)
        assert torch.equal(y, want), i


@pytest.mark.parametrize("form", [f[0] for f in FORMS])
@pytest.mark.parametrize("seqs,tokens", ((0, 1), (2, 0)))
def test_a_call_without_a_token(lib, form, seqs, tokens):
    layer, rope = make(dict(FORMS)[form]), lib.rope(DIM)
    cache, table = paged(lib, 2, 20)
    lens = torch.full((seqs,), 5, dtype=torch.int32, device="cuda")
    x = torch.zeros(seqs, tokens, HIDDEN, dtype=torch.bfloat16, device="cuda")
    assert layer(x, cache, table[:seqs], lens, rotate=rope).shape == (seqs, tokens, HIDDEN)

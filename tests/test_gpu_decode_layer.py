"""The decoder layer with the caller's norms and rotation of q and k, and calls without a token."""
import pytest
import torch

from parity import say
from test_gpu_decode import DIM, FFN, GROUP, HEADS, HIDDEN, Q_HEADS, paged, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def norm(by):
    return lambda x: (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6) * by).to(torch.bfloat16)


def rotation(first, tokens):
    """Pairs (i, i + dim / 2) turned by position * 10000^(-2 i / dim)."""
    at = torch.arange(first, first + tokens, device="cuda")[:, None] * 10000.0 ** (-torch.arange(DIM // 2, device="cuda") * 2 / DIM)
    c, s = at.cos()[:, None], at.sin()[:, None]

    def turn(x):
        a, b = x.float().split(DIM // 2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1).to(torch.bfloat16)
    return lambda q, k: (turn(q), turn(k))


@pytest.mark.parametrize("few", (0, 1 << 20))
def test_norms_and_rotation(lib, few):
    """Bit for bit the operators one by one, for a prompt and for a token behind it."""
    from w8a8_quantized_linear_amd.decode import DecoderLayer
    ws = [w.cuda() for w in weights(5)]
    layer = DecoderLayer(*ws, Q_HEADS, HEADS, DIM, GROUP, few, norm1=norm(1.5), norm2=norm(0.7))
    (cache, table), (other, _) = paged(lib, 2, 20), paged(lib, 2, 20)
    done = 0
    for tokens in (19, 1):
        say(f"layer with norms and rotation, few={few}, {tokens} tokens behind {done}")
        x = torch.randn(2, tokens, HIDDEN, generator=torch.Generator().manual_seed(tokens)).to(torch.bfloat16).cuda()
        lens = torch.full((2,), done + tokens, dtype=torch.int32, device="cuda")
        y = layer(x, cache, table, lens, rotate=rotation(done, tokens))
        rows = x.view(2 * tokens, HIDDEN)
        q, k, v = layer.qkv(norm(1.5)(rows)).view(2, tokens, -1, DIM).split((Q_HEADS, HEADS, HEADS), dim=2)
        q, k = rotation(done, tokens)(q, k)
        lib.w8a8_kv_append(k, v, other, table, lens)
        rows = rows + layer.o(lib.w8a8_kv_attention(q, other, table, lens).view(2 * tokens, -1))
        h = norm(0.7)(rows)
        if few:
            h = layer.gateup(h)
            h = lib.w8a8_swiglu(h[:, :FFN], h[:, FFN:])
        else:
            h = lib.w8a8_gateup_swiglu_packed(h, layer.gateup.w8, FFN, layer.gateup.s8)
        assert torch.equal(y.view_as(rows), rows + layer.down(h))
        bare = DecoderLayer(*ws, Q_HEADS, HEADS, DIM, GROUP, few)
        assert not torch.equal(bare(x, paged(lib, 2, 20)[0], table, torch.full_like(lens, tokens)), y)
        done += tokens


@pytest.mark.parametrize("seqs,tokens", ((0, 1), (2, 0)))
def test_a_call_without_a_token(lib, seqs, tokens):
    from w8a8_quantized_linear_amd.decode import DecoderLayer
    layer = DecoderLayer(*[w.cuda() for w in weights(5)], Q_HEADS, HEADS, DIM, GROUP)
    cache, table = paged(lib, 2, 20)
    lens = torch.full((seqs,), 5, dtype=torch.int32, device="cuda")
    x = torch.zeros(seqs, tokens, HIDDEN, dtype=torch.bfloat16, device="cuda")
    assert layer(x, cache, table[:seqs], lens).shape == (seqs, tokens, HIDDEN)

"""Appending to and reading back the paged 8-bit cache, bit for bit against the formula's single fp32
operations, and against 64 bits where those can round either way."""
import numpy as np
import pytest
import torch

import plain_decode as P
from parity import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def filled(lib, pages, heads, page, dim, seed):
    """A cache full of codes and scales from the seed (its tensors on the GPU)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = lib.kv_cache(pages, heads, page, dim)
    for t in (c.k_codes, c.v_codes):
        t.copy_((torch.randn(t.shape, generator=g, device="cuda") * 36).round().clamp(-127, 127))
    for t in (c.k_scale, c.v_scale):
        t.copy_(0.01 + 0.02 * torch.rand(t.shape, generator=g, device="cuda"))
    return c


def tables(lens, page, extra, seed):
    """Shuffled pages for sequences of these lengths: (table int32, pages)."""
    used = [max(0, -(-max(n, 0) // page)) for n in lens]
    pages = sum(used) + extra
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(lens), max(1, max(used))), -7, dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at:at + u]
        at += u
    return table, pages


def rows_of(seqs, tokens, heads, dim, seed, by=1.0, pad=64):
    """bf16 [seqs, tokens, heads, dim], a slice of a wider projection."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(seqs, tokens, heads * dim + pad, generator=g) * by
    return wide.to(torch.bfloat16).cuda()[..., pad // 2:pad // 2 + heads * dim].unflatten(-1, (heads, dim))


def host(cache):
    return [t.cpu().numpy().copy() for t in cache]


def append_and_check(lib, cache, k, v, table, lens, what):
    kc, vc, ks, vs = host(cache)
    P.append(k.float().cpu().numpy(), kc, ks, table.numpy(), lens)
    P.append(v.float().cpu().numpy(), vc, vs, table.numpy(), lens)
    lib.w8a8_kv_append(k, v, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    got = host(cache)
    for name, a, b in zip(("k codes", "v codes", "k scale", "v scale"), got, (kc, vc, ks, vs)):
        bad = np.argwhere(a.view(np.int32 if a.dtype == np.float32 else a.dtype) != b.view(np.int32 if b.dtype == np.float32 else b.dtype))
        assert len(bad) == 0, f"{what}: {name}: {len(bad)} differ, first at {bad[0]}: {a[tuple(bad[0])]} for {b[tuple(bad[0])]}"
    return got


@pytest.mark.parametrize("page", (16, 32, 64, 128))
@pytest.mark.parametrize("dim", (64, 128))
@pytest.mark.parametrize("tokens", (1, 2, 17, 150))
def test_append(lib, page, dim, tokens):
    """Lengths that end a page, begin one, fall inside one; shorter than the tokens given; empty; negative."""
    lens = [tokens, tokens + 1, tokens + page - 1, tokens + page, 3 * page + tokens // 2, tokens // 2, 0, -3, 5 * page]
    lens = [min(n, 6 * page) if tokens < 100 else n for n in lens]
    say(f"append page={page} dim={dim} tokens={tokens} lens={lens}")
    table, pages = tables(lens, page, 2, seed=tokens)
    cache = filled(lib, pages, 3, page, dim, seed=page + dim)
    k, v = rows_of(len(lens), tokens, 3, dim, 1), rows_of(len(lens), tokens, 3, dim, 2, by=3.0)
    append_and_check(lib, cache, k, v, table, lens, "append")


def test_token_by_token(lib):
    """Forty single tokens of growing size: every step moves the page's codes to a new scale."""
    page, dim, heads = 16, 64, 2
    table, pages = tables([41, 41], page, 1, seed=1)
    cache = filled(lib, pages, heads, page, dim, seed=5)
    for i in range(40):
        k, v = (rows_of(2, 1, heads, dim, 10 * i + j, by=1.05 ** i) for j in (0, 1))
        append_and_check(lib, cache, k, v, table, [i + 1, i + 2], f"token {i}")


def test_smaller_tokens_leave_the_page_as_it_is(lib):
    page, dim = 32, 128
    table, pages = tables([20], page, 0, seed=1)
    cache = filled(lib, pages, 1, page, dim, seed=5)
    before = host(cache)
    k = rows_of(1, 1, 1, dim, 1, by=1e-3)
    got = append_and_check(lib, cache, k, k, table, [20], "small")
    for a, b in zip(got[:2], before[:2]):
        assert np.array_equal(a[:, :, :19], b[:, :, :19]) and np.array_equal(a[:, :, 20:], b[:, :, 20:])


def test_zeros_and_extreme_scales(lib):
    """Blocks of zeros (scale 0), subnormal scales, the largest bf16 values, and zeros behind held zeros."""
    page, dim = 16, 64
    lens = [16, 16, 16, 16]
    table, pages = tables(lens, page, 0, seed=3)
    cache = filled(lib, pages, 1, page, dim, seed=5)
    k = rows_of(4, 16, 1, dim, 9).clone()
    k[0] = 0
    k[1] *= 2.0 ** -125
    k[2] = 3.3e38
    k[3, :, :, ::2] = -0.0
    append_and_check(lib, cache, k, -k, table, lens, "extremes")
    more = rows_of(4, 1, 1, dim, 10).clone()
    more[0] = 0
    table2 = torch.cat((table, table), 1)                    # position 16 opens the same page again: overwritten
    append_and_check(lib, cache, more, more, table2, [17] * 4, "zero behind")
    more[0] = 1.0
    append_and_check(lib, cache, more, more, table, [2] * 4, "one behind zero")


def test_pages_that_do_not_exist(lib):
    """Tokens whose table entry is outside the cache, or past the table, are dropped; nothing else changes."""
    page, dim = 16, 64
    table = torch.tensor([[0, -1, 2], [3, 99, 2147483647], [-2147483648, 4, 5]], dtype=torch.int32)
    cache = filled(lib, 6, 2, page, dim, seed=5)
    k = rows_of(3, 60, 2, dim, 9)
    append_and_check(lib, cache, k, k, table, [60, 48, 2000], "missing pages")


def test_codes_are_the_nearest_in_64_bits(lib):
    page, dim, tokens = 64, 128, 640
    table, pages = tables([tokens], page, 0, seed=1)
    cache = lib.kv_cache(pages, 4, page, dim)
    k = rows_of(1, tokens, 4, dim, 3)
    lens = torch.tensor([tokens], dtype=torch.int32).cuda()
    lib.w8a8_kv_append(k, k, cache, table.cuda(), lens)
    x = k[0].double().cpu().numpy().reshape(pages, page, 4, dim).transpose(0, 2, 1, 3)
    codes, scale = (t.cpu().numpy()[table[0].numpy()] for t in (cache.k_codes, cache.k_scale))
    s = np.abs(x).max((2, 3)) / 127
    assert np.allclose(scale, s, rtol=2 ** -23)
    off = np.abs(codes - x / s[:, :, None, None])
    assert off.max() <= 0.5 + 1e-4                            # 127 units of fp32 rounding at most


@pytest.mark.parametrize("length", (1, 37, 96))
@pytest.mark.parametrize("page,dim", ((16, 64), (64, 128), (128, 64)))
def test_read(lib, page, dim, length):
    lens = [0, 1, 36, 37, 38, 96, 200, -1]
    table, pages = tables(lens, page, 1, seed=4)
    table[3, 0] = -1                                          # a hole reads as zeros
    cache = filled(lib, pages, 3, page, dim, seed=5)
    out = [torch.full((len(lens), length, 3, dim), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = lib.w8a8_kv_read(cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), length, out=out)
    kc, vc, ks, vs = host(cache)
    for got, codes, scale in ((k, kc, ks), (v, vc, vs)):
        ref = np.zeros((len(lens), length, 3, dim), dtype=np.float32)
        for b, n in enumerate(lens):
            n = min(max(n, 0), length, table.shape[1] * page)
            for h in range(3):
                if n:
                    ref[b, :n, h] = P.gathered(codes, scale, table[b].numpy(), n, h)[0]
        assert torch.equal(got.cpu(), torch.from_numpy(ref).to(torch.bfloat16))


def test_offsets_past_2_31_bytes(lib):
    """A cache of 2.2 GB of codes each for keys and values; the last pages are used."""
    heads, page, dim = 8, 128, 128
    pages = 2 ** 31 // (heads * page * dim) + 60
    say("cache past 2^31 bytes")
    cache = lib.kv_cache(pages, heads, page, dim)
    mark = 2 ** 31 // (heads * page * dim)
    table = torch.tensor([[mark - 1, mark, pages - 1]], dtype=torch.int32)
    tokens = 3 * page - 5
    k, v = rows_of(1, tokens, heads, dim, 1), rows_of(1, tokens, heads, dim, 2)
    lens = torch.tensor([tokens], dtype=torch.int32)
    lib.w8a8_kv_append(k, v, cache, table.cuda(), lens.cuda())
    used = table[0].long().cuda()
    small = [t[used].cpu().numpy() for t in cache]
    want = [np.zeros_like(a) for a in small]
    here = np.arange(3, dtype=np.int32)[None]
    P.append(k.float().cpu().numpy(), want[0], want[2], here, [tokens])
    P.append(v.float().cpu().numpy(), want[1], want[3], here, [tokens])
    for a, b in zip(small[:2], want[:2]):
        assert np.array_equal(a[:2], b[:2]) and np.array_equal(a[2, :, :page - 5], b[2, :, :page - 5])
    for a, b in zip(small[2:], want[2:]):
        assert np.array_equal(a, b)
    kr, _ = lib.w8a8_kv_read(cache, table.cuda(), lens.cuda(), tokens)
    for h in (0, heads - 1):
        ref = P.gathered(want[0], want[2], here[0], tokens, h)[0].astype(np.float32)
        assert torch.equal(kr[0, :, h].cpu(), torch.from_numpy(ref).to(torch.bfloat16))


def test_refusals(lib):
    cache = filled(lib, 4, 2, 16, 64, 1)
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    k = rows_of(1, 1, 2, 64, 1)
    lib.w8a8_kv_append(k, k, cache, table, lens)
    lib.w8a8_kv_append(k[:, :0], k[:, :0], cache, table, lens)             # no tokens: nothing to do
    lib.w8a8_kv_append(k[:0], k[:0], cache, table[:0], lens[:0])           # no sequences
    assert lib.w8a8_kv_read(cache, table, lens, 0)[0].shape == (1, 0, 2, 64)
    for bad in (dict(k=k.float()), dict(table=table.long()), dict(lens=lens.long()), dict(cache=cache._replace(k_scale=cache.k_scale.half()))):
        with pytest.raises(TypeError):
            lib.w8a8_kv_append(**{**dict(k=k, v=k, cache=cache, table=table, lens=lens), **bad})
    for bad in (dict(k=k[..., :32]), dict(v=rows_of(1, 2, 2, 64, 1)), dict(table=table.repeat(2, 1)), dict(lens=lens.cpu()),
                dict(k=k.transpose(2, 3).contiguous().transpose(2, 3)), dict(cache=cache._replace(v_scale=cache.v_scale[:3].contiguous())),
                dict(k=rows_of(1, 1, 4, 64, 1), v=rows_of(1, 1, 4, 64, 1))):
        with pytest.raises(ValueError):
            lib.w8a8_kv_append(**{**dict(k=k, v=k, cache=cache, table=table, lens=lens), **bad})
    odd = filled(lib, 2, 1, 16, 64, 1)
    for shape in ((2, 1, 24, 64), (2, 1, 16, 96)):
        c = lib.KVCache(*(torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in "kv"), odd.k_scale, odd.v_scale)
        x = torch.zeros(1, 1, 1, shape[3], dtype=torch.bfloat16, device="cuda")
        with pytest.raises(lib.W8A8Error):
            lib.w8a8_kv_append(x, x, c, table, lens)
    wide = torch.zeros(1, 2, 132, dtype=torch.bfloat16, device="cuda")[..., :128].unflatten(-1, (2, 64))
    with pytest.raises(lib.W8A8Error):                                     # rows 132 elements apart
        lib.w8a8_kv_append(wide, wide, cache, table, lens)
    shifted = torch.zeros(136, dtype=torch.bfloat16, device="cuda")[4:132].view(1, 1, 2, 64)
    with pytest.raises(lib.W8A8Error):                                     # not 16-byte aligned
        lib.w8a8_kv_append(shifted, shifted, cache, table, lens)

"""Attention where a piece of a sequence is many times what is held at once of the page table, where many pieces meet,
and at the end of the running sum's range: against 64 bits, with the tolerance of test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

from parity import say
from test_gpu_kv_attention import attend, check
from test_gpu_kv_cache import filled, rows_of, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


# Pages of 16 tokens, 64 of which a wave holds at once: one long sequence among so many short ones that it is read in
# one piece (4,500 tokens: 282 pages) or two (219 pages each, the second from page 219 on), by four waves, one
# block of rows or two (17 rows and more)
@pytest.mark.parametrize("tokens,q_heads", ((1, 4), (1, 40), (5, 16), (17, 4)))
@pytest.mark.parametrize("dim,seqs,length", ((128, 33, 4500), (128, 32, 7000), (64, 66, 4500), (64, 64, 7000)))
def test_pieces_of_many_pages(lib, dim, seqs, length, tokens, q_heads):
    heads, page = 4, 16
    say(f"pieces of many pages dim={dim} seqs={seqs} length={length} tokens={tokens} heads={q_heads}/{heads}")
    lens = [int(n) for n in np.random.RandomState(seqs).randint(0, 60, seqs)]
    lens[seqs // 2] = length
    table, pages = tables(lens, page, 0, 11)
    need = lib.kv_attention_workspace_bytes(seqs, tokens, q_heads, heads, dim, page, table.shape[1])
    most = 2 if length == 7000 else 1
    assert need <= 4 * seqs * tokens * q_heads * most * (dim + 2) + 255      # no more pieces than meant
    cache = filled(lib, pages, heads, page, dim, 12)
    q = rows_of(seqs, tokens, q_heads, dim, 13, by=2.0)
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "many pages")


@pytest.mark.parametrize("lens,q_heads,heads,dim,page", (
    ([30000], 1, 1, 128, 16), ([30000, 17000], 5, 1, 64, 32), ([131072], 2, 1, 128, 128), ([131072], 1, 1, 64, 16), ([90001], 4, 2, 64, 64)))
def test_more_than_64_pieces(lib, lens, q_heads, heads, dim, page):
    """One token over up to 131,072 others, in 65 pieces and more, all of them with keys."""
    say(f"many pieces lens={lens} heads={q_heads}/{heads} dim={dim} page={page}")
    table, pages = tables(lens, page, 0, 21)
    need = lib.kv_attention_workspace_bytes(len(lens), 1, q_heads, heads, dim, page, table.shape[1])
    assert need >= 4 * len(lens) * q_heads * 65 * (dim + 2)
    cache = filled(lib, pages, heads, page, dim, 22)
    q = rows_of(len(lens), 1, q_heads, dim, 23, by=2.0)
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "many pieces")


def test_the_sum_over_a_long_sequence_of_small_values(lib):
    """2^24 tokens whose values have the smallest scale that counts, 2^-90, and whose scores lie 7.9 powers of two above
    the first ones, which the running maximum does not follow: the sum of p / scale passes 2^128.  All tokens but the
    first page's share one page, so the cache is small; 512 heads, so the sequence is one piece.

    y is 100 * 2^-90 but for the first page's 128 tokens (2^-17 of it): fp32 sums of 2^17 equal steps in a row err by up
    to 2^-8 each, outputs and sum, and bf16 by 2^-9, so within 2^-6."""
    heads, dim, page, length = 512, 64, 128, 1 << 24
    say("2^24 tokens of 512 heads")
    cache = lib.kv_cache(2, heads, page, dim)
    for t in cache[:2]:
        t.zero_()
    cache.k_codes[1, :, :, 0] = 79
    cache.v_codes[0], cache.v_codes[1] = 10, 100
    cache.k_scale.fill_(7.9 / 79 * float(np.log(2)))
    cache.v_scale.fill_(2.0 ** -90)
    table = torch.ones(1, length // page, dtype=torch.int32)
    table[0, 0] = 0
    assert lib.kv_attention_workspace_bytes(1, 1, heads, heads, dim, page, table.shape[1]) == 0
    q = torch.zeros(1, 1, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    y = attend(lib, q, cache, table, [length], 1.0).double().cpu() * 2.0 ** 90
    assert float((y / 100 - 1).abs().max()) < 2 ** -6, y.flatten()[:4]

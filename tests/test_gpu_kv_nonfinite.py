"""Attention beside pages whose scales are not finite, and softmax scales of every sign: against 64 bits, with the
tolerance of test_gpu_kv_attention.py."""
import numpy as np
import pytest
import torch

import plain_decode as P
from parity import say
from test_gpu_kv_attention import attend, check, host, long_table
from test_gpu_kv_cache import filled, rows_of, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


# Sequences of `length` tokens, the last `tokens` of them new, a page boundary among those; tables that fit, of `width`
# pages, or (-1) with work for the prompt form.  So: eight waves, four waves in pieces with one block of rows and
# with two, whole prompts in either form, pages smaller and larger than a step or a tile.
SHAPES = ((1, 306, 5, 4, 2, 64, 16, 0), (1, 322, 5, 4, 2, 128, 32, 0), (1, 306, 5, 4, 2, 64, 16, 200), (2, 322, 5, 4, 2, 128, 32, 100),
          (3, 708, 9, 4, 2, 64, 16, 900), (2, 900, 20, 4, 2, 128, 64, 300), (1, 200, 200, 4, 2, 64, 16, 0),
          (1, 333, 333, 4, 2, 128, 32, -1), (2, 260, 260, 6, 2, 64, 16, -1), (1, 700, 650, 8, 2, 128, 128, -1))


@pytest.mark.parametrize("which", ("v_scale", "k_scale"))
@pytest.mark.parametrize("seqs,length,tokens,q_heads,heads,dim,page,width", SHAPES)
def test_a_page_of_infinite_scale_spoils_only_the_queries_that_see_it(lib, seqs, length, tokens, q_heads, heads, dim, page, width, which):
    """The pages from a middle new token on have an infinite scale, as append leaves it behind an infinite value: the
    queries before them give what they give over a finite cache."""
    say(f"infinite {which} length={length} tokens={tokens} heads={q_heads}/{heads} dim={dim} page={page} width={width}")
    lens = [length] * seqs
    table, pages = tables(lens, page, 0, 3)
    cache = filled(lib, pages, heads, page, dim, 4)
    q = rows_of(seqs, tokens, q_heads, dim, 5, by=2.0)
    first = -(-(length - tokens + 1 + (tokens - 1) // 2) // page) * page     # the first position of the infinite pages
    first = min(first, (length - 1) // page * page)
    before = first - (length - tokens)                                         # new tokens that see none of them
    assert 0 < before < tokens
    kc, vc, ks, vs = host(cache)
    ref, spread = P.attention(q.float().cpu().numpy(), kc, vc, ks, vs, table.numpy(), lens, dim ** -0.5)
    getattr(cache, which)[table[:, first // page:].reshape(-1).long()] = float("inf")
    if width == -1:
        table = long_table(table, seqs, tokens * q_heads // heads, heads, page)
    elif width > table.shape[1]:
        table = torch.cat((table, torch.full((seqs, width - table.shape[1]), -1, dtype=torch.int32)), 1)
    y = attend(lib, q, cache, table, lens).float().cpu().numpy().astype(np.float64)[:, :before]
    assert np.isfinite(y).all(), f"{(~np.isfinite(y)).any(-1).sum()} of {y[..., 0].size} rows before the page are not finite"
    over = np.abs(y - ref[:, :before]) - (2 ** -8 * np.abs(ref[:, :before]) + 2 ** -10 * spread[:, :before])
    assert over.max() <= 0


def test_an_infinite_value_appended_last(lib):
    """Through append: the last token's value is infinite, its page begins with it, the other proposed tokens stay finite."""
    lens, tokens, dim, page = [65], 5, 64, 16
    table, pages = tables(lens, page, 0, 3)
    cache = filled(lib, pages, 1, page, dim, 4)
    q, k, v = rows_of(1, tokens, 4, dim, 5), rows_of(1, tokens, 1, dim, 6), rows_of(1, tokens, 1, dim, 7).clone()
    td, ld = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    v[0, -1, 0, 3] = float("inf")
    lib.w8a8_kv_append(k, v, cache, td, ld)
    assert torch.isinf(cache.v_scale[table[0, 4].long()]).all()
    y = attend(lib, q, cache, table, lens)
    assert torch.isfinite(y[:, :-1].float()).all()


# one row, rows in one and two blocks, and the prompt form
FORMS = ((1, False), (6, False), (12, True), (70, True))


@pytest.mark.parametrize("scale", (0.0, -0.125, -2.0))
@pytest.mark.parametrize("tokens,wide", FORMS)
def test_softmax_scales_that_are_not_positive(lib, tokens, wide, scale):
    """0 averages what a query sees; a negative scale is the positive one with the queries' signs turned, bit for bit.
    (Against 64 bits while the scores stay small: with -2, probabilities below f16's range are all that some elements
    have, which the tolerance has no term for.)"""
    lens, dim, page = [300, 100], 64, 32
    table, pages = tables(lens, page, 2, 1)
    if wide:
        table = long_table(table, 2, 4 * tokens, 2, page)
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(2, tokens, 8, dim, 3, by=2.0)
    y = attend(lib, q, cache, table, lens, scale)
    assert torch.equal(y, attend(lib, -q, cache, table, lens, -scale))
    if scale > -1:
        check(y, q, cache, table, lens, scale, f"scale {scale}")


@pytest.mark.parametrize("bad", (float("inf"), -float("inf")))
@pytest.mark.parametrize("tokens,wide", FORMS)
def test_an_infinite_query_spoils_its_own_row_only(lib, tokens, wide, bad):
    """(Its scores are infinities of both signs or NaN, so its own outputs are NaN.)"""
    lens, dim, page = [300, 100], 64, 32
    table, pages = tables(lens, page, 2, 1)
    if wide:
        table = long_table(table, 2, 4 * tokens, 2, page)
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(2, tokens, 8, dim, 3, by=2.0).clone()
    clean = q.clone()
    q[1, tokens // 2, 5, 7] = bad
    y = attend(lib, q, cache, table, lens)
    assert torch.isnan(y[1, tokens // 2, 5].float()).all()
    y[1, tokens // 2, 5] = attend(lib, clean, cache, table, lens)[1, tokens // 2, 5]
    check(y, clean, cache, table, lens, dim ** -0.5, "beside an infinity")

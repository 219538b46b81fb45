"""Attention over the paged 8-bit cache on the GPU against its formula in 64 bits.

Tolerance.  The output is rounded once to bf16: 2^-9 of its value.  Each probability carries a relative error of
at most 2^-11 from its f16 rounding, and a few 2^-23 times the score's size (below 100 here) from fp32 scores and
exp2: with A = sum(p |v|) / sum(p) that moves an output by less than 2^-10 A.  So |y - ref| <= 2^-8 |ref| + 2^-10 A."""
import numpy as np
import pytest
import torch

import plain_decode as P
from parity import say
from test_gpu_kv_cache import filled, host, rows_of, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def attend(lib, q, cache, table, lens, scale=None):
    """The call with output and workspace full of NaN beforehand."""
    seqs, tokens, q_heads, dim = q.shape
    _, heads, page, _ = cache.k_codes.shape
    need = lib.kv_attention_workspace_bytes(seqs, tokens, q_heads, heads, dim, page, table.shape[1])
    ws = torch.full((max(need // 4, 1),), float("nan"), device="cuda")
    out = torch.full((seqs, tokens, q_heads, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    return lib.w8a8_kv_attention(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale, workspace=ws, out=out)


def check(y, q, cache, table, lens, scale, what):
    y = y.float().cpu().numpy().astype(np.float64)
    kc, vc, ks, vs = host(cache)
    ref, spread = P.attention(q.float().cpu().numpy(), kc, vc, ks, vs, table.numpy(), lens, scale)
    over = np.abs(y - ref) - (2 ** -8 * np.abs(ref) + 2 ** -10 * spread)
    assert np.isfinite(y).all(), f"{what}: {np.argwhere(~np.isfinite(y))[0]} is not finite"
    assert over.max() <= 0, f"{what}: {(over > 0).sum()} of {over.size} off, by up to {over.max()} at {np.unravel_index(over.argmax(), over.shape)}"


def run(lib, lens, tokens, q_heads, heads, dim, page, seed=0, q_by=2.0, scale=None):
    say(f"attention lens={lens} tokens={tokens} heads={q_heads}/{heads} dim={dim} page={page}")
    table, pages = tables(lens, page, 2, seed)
    cache = filled(lib, pages, heads, page, dim, seed + 1)
    q = rows_of(len(lens), tokens, q_heads, dim, seed + 2, by=q_by)
    y = attend(lib, q, cache, table, lens, scale)
    check(y, q, cache, table, lens, dim ** -0.5 if scale is None else scale, "attention")
    return y, q, cache, table


@pytest.mark.parametrize("page", (16, 32, 64, 128))
@pytest.mark.parametrize("dim", (64, 128))
def test_single_tokens(lib, dim, page):
    run(lib, [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 300, 0, 517], 1, 8, 2, dim, page, seed=page)


@pytest.mark.parametrize("group", (1, 2, 3, 5, 8, 16, 17, 40))
def test_head_layouts(lib, group):
    run(lib, [77, 200], 1, 2 * group, 2, 64, 32, seed=group)
    run(lib, [77, 1], 2, group, 1, 128, 16, seed=group)


@pytest.mark.parametrize("tokens", (2, 3, 5, 8, 16, 17, 33, 64, 65, 130))
def test_several_tokens(lib, tokens):
    """Causal among themselves; sequences shorter than the tokens given leave their first queries empty."""
    run(lib, [tokens, tokens + 1, tokens + 100, tokens // 2, 0, 1, -5], tokens, 6, 2, 64, 32, seed=tokens)
    run(lib, [tokens + 37], tokens, 5, 1, 128, 64, seed=tokens)


@pytest.mark.parametrize("lens,tokens,q_heads,heads,dim,page", (
    ([2300], 1, 40, 8, 128, 64), ([4500], 1, 8, 8, 64, 16), ([9000, 31], 1, 4, 1, 128, 128),
    ([5000], 3, 8, 2, 64, 16), ([2500, 2100], 40, 4, 1, 128, 32)))
def test_long_sequences(lib, lens, tokens, q_heads, heads, dim, page):
    """Cut into pieces, and pieces longer than what is held at once of the page table."""
    run(lib, lens, tokens, q_heads, heads, dim, page, seed=9)


def test_many_sequences_of_one_piece(lib):
    """So many that none is cut: the pieces are whole sequences, longer than 2,048 tokens for one of them."""
    lens = [int(n) for n in np.random.RandomState(1).randint(0, 40, 520)]
    lens[3], lens[100] = 2200, 4100
    run(lib, lens, 1, 4, 2, 64, 64, seed=2)


def test_prompt(lib):
    run(lib, [333, 300], 300, 6, 2, 128, 64, seed=4)


# both sizes of the prompt form's workgroups (tables to 1,024 tokens and past them), pieces of a sequence, rows that
# do not fill a block, groups that straddle one, lengths around a page and a tile, sequences shorter than the call
@pytest.mark.parametrize("lens,tokens,q_heads,heads,dim,page", (
    ([700, 699], 65, 2, 2, 128, 32), ([513, 1, 64], 130, 8, 1, 64, 128), ([1300, 40, 0], 200, 4, 2, 64, 16),
    ([1025], 1025, 2, 1, 128, 128), ([3000, 2999], 70, 3, 1, 128, 64), ([2049], 33, 40, 8, 64, 16), ([127, 129, 128], 129, 5, 1, 64, 32)))
def test_prompt_shapes(lib, lens, tokens, q_heads, heads, dim, page):
    run(lib, lens, tokens, q_heads, heads, dim, page, seed=len(lens) + tokens)


def long_table(table, seqs, rows, heads, page, seed=77):
    """The table with columns past every sequence, named at random, until there is work for the prompt form."""
    width = -(-2 * (256 * 16 * 1536 * 2 + 1) // (rows * seqs * heads * page))
    more = torch.randint(-5, 10 ** 6, (table.shape[0], max(width - table.shape[1], 0)), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    return torch.cat((table, more), 1)


# two blocks of 16 rows a workgroup: 17 to 64 rows and tables for many tokens, in pieces and (many sequences) in one
@pytest.mark.parametrize("lens,tokens,q_heads,heads,dim,page,width", (
    ([700, 5, 0], 5, 10, 2, 64, 32, 700), ([1500, 129], 4, 16, 2, 128, 64, 400), ([3000], 3, 6, 1, 64, 128, 520),
    ([333, 40, 1300], 9, 7, 1, 128, 16, 1500), ([9, 300] * 70, 5, 12, 2, 64, 16, 40), ([200] * 130, 17, 2, 2, 128, 64, 6)))
def test_two_blocks_of_rows(lib, lens, tokens, q_heads, heads, dim, page, width):
    assert len(lens) * heads * width * page > 256 * 256 and 16 < tokens * q_heads // heads <= 64
    say(f"two blocks lens={lens[:3]} tokens={tokens} heads={q_heads}/{heads} dim={dim} page={page}")
    table, pages = tables(lens, page, 0, 5)
    more = torch.randint(-5, 10 ** 6, (len(lens), width - table.shape[1]), generator=torch.Generator().manual_seed(6), dtype=torch.int32)
    table = torch.cat((table, more), 1)
    cache = filled(lib, pages, heads, page, dim, 6)
    q = rows_of(len(lens), tokens, q_heads, dim, 7, by=2.0)
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "two blocks")


# eight waves on one piece, one piece of four waves, pieces: lengths about the limits of the rules, holes among the pages
@pytest.mark.parametrize("dim,page", ((64, 16), (64, 128), (128, 32), (128, 64)))
@pytest.mark.parametrize("seqs,heads,length", ((3, 2, 1024), (3, 2, 1040), (2, 4, 1536), (2, 4, 1600), (9, 15, 500), (9, 16, 640), (70, 4, 256), (5, 1, 130)))
def test_forms_of_few_rows(lib, seqs, heads, length, dim, page):
    say(f"few rows seqs={seqs} heads={heads} length={length} dim={dim} page={page}")
    lens = [max(length - 37 * b, 0) if b % 4 else length for b in range(seqs)]
    table, pages = tables(lens, page, 0, seqs)
    table[0, 0] = -1
    cache = filled(lib, pages, heads, page, dim, 3)
    q = rows_of(seqs, 2, 2 * heads, dim, 4, by=2.0)
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "few rows")


# the same shapes in the prompt form, whose pieces are then mostly empty, and shapes that are large enough by themselves
@pytest.mark.parametrize("lens,tokens,q_heads,heads,dim,page", (
    ([700, 699], 65, 2, 2, 128, 32), ([513, 1, 64], 130, 8, 1, 64, 128), ([1300, 40, 0], 200, 4, 2, 64, 16),
    ([1025], 1025, 2, 1, 128, 128), ([3000, 2999], 70, 3, 1, 128, 64), ([2049], 33, 40, 8, 64, 16), ([127, 129, 128], 129, 5, 1, 64, 32),
    ([1300, 900], 900, 8, 2, 64, 32), ([1200], 1150, 10, 2, 128, 64), ([1030, 1, 1029], 700, 6, 2, 128, 16)))
def test_prompt_form(lib, lens, tokens, q_heads, heads, dim, page):
    say(f"prompt form lens={lens} tokens={tokens} heads={q_heads}/{heads} dim={dim} page={page}")
    table, pages = tables(lens, page, 2, 5)
    table = long_table(table, len(lens), tokens * q_heads // heads, heads, page)
    cache = filled(lib, pages, heads, page, dim, 6)
    q = rows_of(len(lens), tokens, q_heads, dim, 7, by=2.0)
    y = attend(lib, q, cache, table, lens)
    check(y, q, cache, table, lens, dim ** -0.5, "prompt form")


@pytest.mark.parametrize("dim,page,length", ((64, 16, 600), (128, 64, 1500)))
def test_prompt_form_with_holes_and_pages_of_zeros(lib, dim, page, length):
    lens, tokens = [length, length - 37, 90], 100
    table, pages = tables(lens, page, 3, 8)
    cache = filled(lib, pages, 2, page, dim, 9)
    g = torch.Generator(device="cuda").manual_seed(10)
    cache.v_scale.mul_(2.0 ** torch.randint(-30, 10, cache.v_scale.shape, generator=g, device="cuda"))
    cache.v_scale[table[0, 1::4].long()] = 0
    cache.k_scale[table[1, ::3].long()] = 0
    table[0, 2], table[1, 0] = -1, 2147483647
    used = torch.zeros(pages, dtype=torch.bool)
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // page)].long()
        used[ids[(ids >= 0) & (ids < pages)]] = True
    table = long_table(table, 3, 300, 2, page)
    q = rows_of(3, tokens, 6, dim, 11)
    y = attend(lib, q, cache, table, lens)
    check(y, q, cache, table, lens, dim ** -0.5, "prompt form with holes")
    for s in (cache.k_scale, cache.v_scale):
        s[~used.cuda()] = float("nan")
    assert torch.equal(attend(lib, q, cache, table, lens).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("apart", (2.0 ** 20, 2.0 ** 60))
def test_prompt_form_and_large_values_that_are_not_attended(lib, apart):
    lens, dim, page, tokens = [300, 200], 64, 32, 100
    table, pages = tables(lens, page, 0, 1)
    cache = filled(lib, pages, 1, page, dim, 2)
    q = rows_of(1, 1, 2, dim, 3).expand(2, tokens, 2, dim).contiguous()
    q[:, :, 1] = q[:, :, 0]
    toward = q[0, 0, 0].sign()
    cache.k_codes[:] = (toward * 60).to(torch.int8)
    cache.k_codes[..., ::3] = cache.v_codes[..., ::3] // 2
    cache.k_scale.fill_(0.5)
    for p in (int(table[0, 0]), int(table[1, 2])):
        cache.k_codes[p] = (-100 * toward).to(torch.int8)
        cache.v_scale[p] *= apart
    table = long_table(table, 2, 2 * tokens, 1, page)
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "not attended")


@pytest.mark.parametrize("dim,page,length", ((64, 16, 600), (128, 64, 1500), (128, 128, 4000)))
def test_prompt_with_holes_and_pages_of_zeros(lib, dim, page, length):
    """Holes, pages of zero scales or of scales far apart, and whatever stands where nothing is held."""
    lens, tokens = [length, length - 37, 90], 100
    table, pages = tables(lens, page, 3, 8)
    cache = filled(lib, pages, 2, page, dim, 9)
    g = torch.Generator(device="cuda").manual_seed(10)
    cache.v_scale.mul_(2.0 ** torch.randint(-30, 10, cache.v_scale.shape, generator=g, device="cuda"))
    cache.v_scale[table[0, 1::4].long()] = 0
    cache.k_scale[table[1, ::3].long()] = 0
    table[0, 2], table[0, -1], table[1, 0] = -1, pages, 2147483647
    q = rows_of(3, tokens, 6, dim, 11)
    y = attend(lib, q, cache, table, lens)
    check(y, q, cache, table, lens, dim ** -0.5, "prompt with holes")
    used = torch.zeros(pages, dtype=torch.bool)
    for b, n in enumerate(lens):
        ids = table[b, :-(-n // page)].long()
        used[ids[(ids >= 0) & (ids < pages)]] = True
    for s in (cache.k_scale, cache.v_scale):
        s[~used.cuda()] = float("nan")
    for b, n in enumerate(lens):
        p = int(table[b, n // page]) if n % page else -1
        if 0 <= p < pages:
            cache.k_codes[p, :, n % page:] = 127
            cache.v_codes[p, :, n % page:] = -127
    again = attend(lib, q, cache, table, lens)
    assert torch.equal(again.view(torch.int16), y.view(torch.int16))


def test_peaked_scores(lib):
    """Scores of several hundred: one key takes nearly everything, the running maximum moves late."""
    lens, dim, page = [700, 90], 64, 32
    table, pages = tables(lens, page, 0, 1)
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(2, 1, 4, dim, 3).clone()
    for pos in (695, 300):
        p = int(table[0, pos // page])
        cache.k_codes[p, :, pos % page] = (q[0, 0, ::2].sign() * (127 if pos == 695 else 100)).to(torch.int8)
    q *= 4
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "peaked")


def test_scales_far_apart(lib):
    """Pages whose scales differ by many powers of two, and pages of zeros, in keys and in values."""
    lens, dim, page = [1000, 500, 64], 128, 16
    table, pages = tables(lens, page, 0, 1)
    cache = filled(lib, pages, 2, page, dim, 2)
    g = torch.Generator(device="cuda").manual_seed(5)
    cache.v_scale.mul_(2.0 ** torch.randint(-40, 30, cache.v_scale.shape, generator=g, device="cuda"))
    cache.k_scale.mul_(2.0 ** torch.randint(-20, 1, cache.k_scale.shape, generator=g, device="cuda"))
    cache.v_scale[::7] = 0
    cache.k_scale[::5] = 0
    cache.v_scale[table[2, :4].long()] = 0                   # a sequence whose values are all zeros
    q = rows_of(3, 2, 4, dim, 3)
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "scales")


@pytest.mark.parametrize("tokens", (1, 100))
@pytest.mark.parametrize("apart", (2.0 ** 20, 2.0 ** 40, 2.0 ** 60))
def test_large_values_that_are_not_attended(lib, tokens, apart):
    """A page of values 2^20 and more times the others', first or in the middle, whose keys score far below theirs."""
    lens, dim, page = [300, 200], 64, 32
    table, pages = tables(lens, page, 0, 1)
    cache = filled(lib, pages, 1, page, dim, 2)
    q = rows_of(1, 1, 2, dim, 3).expand(2, tokens, 2, dim).contiguous()
    q[:, :, 1] = q[:, :, 0]
    toward = q[0, 0, 0].sign()
    cache.k_codes[:] = (toward * 60).to(torch.int8)
    cache.k_codes[..., ::3] = cache.v_codes[..., ::3] // 2     # (some spread of the scores)
    cache.k_scale.fill_(0.5)
    for p in (int(table[0, 0]), int(table[1, 2])):
        cache.k_codes[p] = (-100 * toward).to(torch.int8)
        cache.v_scale[p] *= apart
    check(attend(lib, q, cache, table, lens), q, cache, table, lens, dim ** -0.5, "not attended")


@pytest.mark.parametrize("by", (2.0 ** -60, 2.0 ** -20, 2.0 ** 40))
def test_query_sizes(lib, by):
    """Tiny and huge queries, with a softmax scale that makes up for it."""
    run(lib, [50, 300], 1, 4, 2, 64, 32, seed=1, q_by=2 * by, scale=0.125 / by)


@pytest.mark.parametrize("tokens,wide", ((1, False), (6, False), (6, True), (70, False), (70, True)))
def test_a_query_that_is_not_finite_spoils_its_own_row_only(lib, tokens, wide):
    lens, dim, page = [300, 100], 64, 32
    table, pages = tables(lens, page, 2, 1)
    if wide:
        table = long_table(table, 2, 4 * tokens, 2, page)
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(2, tokens, 8, dim, 3, by=2.0).clone()
    clean = q.clone()
    q[1, tokens // 2, 5, 7] = float("nan")
    y = attend(lib, q, cache, table, lens)
    assert torch.isnan(y[1, tokens // 2, 5].float()).all()
    y[1, tokens // 2, 5] = attend(lib, clean, cache, table, lens)[1, tokens // 2, 5]
    check(y, clean, cache, table, lens, dim ** -0.5, "beside a NaN")


def test_zero_queries_average_the_values(lib):
    run(lib, [100, 3], 2, 4, 2, 64, 16, seed=1, q_by=0.0)


def test_queries_of_mixed_size(lib):
    """A row's elements spread over 60 powers of two: the small ones still count where the large are zero keys."""
    lens, dim, page = [200], 64, 32
    table, pages = tables(lens, page, 0, 1)
    cache = filled(lib, pages, 1, page, dim, 2)
    q = rows_of(1, 1, 2, dim, 3).clone()
    q[..., ::2] *= 2.0 ** -12
    cache.k_codes[..., 1::2] = 0
    check(attend(lib, q, cache, table, lens, 40.0), q, cache, table, lens, 40.0, "mixed")


def test_what_is_not_held_does_not_count(lib):
    """Pages and rows past the lengths, holes in the table: NaN scales and any codes there change nothing."""
    lens, dim, page = [33, 100, 0, 64], 64, 32
    table, pages = tables(lens, page, 3, 1)
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(4, 3, 4, dim, 3)
    y = attend(lib, q, cache, table, lens)
    used = torch.zeros(pages, dtype=torch.bool)
    for b, n in enumerate(lens):
        used[table[b, :-(-n // page)].long()] = True
    for t in (cache.k_scale, cache.v_scale):
        t[~used.cuda()] = float("nan")
    for b, n in enumerate(lens):                              # rows of a last page that are not held
        if n % page:
            p = int(table[b, n // page])
            cache.k_codes[p, :, n % page:] = 127
            cache.v_codes[p, :, n % page:] = -127
    wide = torch.cat((table, torch.full_like(table, pages - 1)), 1)
    wide[:, table.shape[1]:] = int(torch.nonzero(~used)[0])   # longer rows, naming a page of NaN scales
    assert torch.equal(attend(lib, q, cache, table, lens).view(torch.int16), y.view(torch.int16))
    check(attend(lib, q, cache, wide, lens), q, cache, wide, lens, dim ** -0.5, "wide table")


def test_holes_in_the_table(lib):
    """Blocks whose entry names no page are not seen; a sequence of nothing but holes gives zeros."""
    lens, dim, page = [100, 64, 160], 64, 32
    table, pages = tables(lens, page, 0, 1)
    table[0, 1], table[0, 3] = -1, pages
    table[1, :] = 2147483647
    table[2, 0] = -2147483648
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(3, 5, 4, dim, 3)
    y = attend(lib, q, cache, table, lens)
    check(y, q, cache, table, lens, dim ** -0.5, "holes")
    assert not y[1].any()


def test_longer_than_the_table(lib):
    """A length past what the table addresses: the keys are those of the table, the positions those of the length."""
    dim, page = 64, 16
    table, pages = tables([64, 64], page, 0, 1)
    cache = filled(lib, pages, 1, page, dim, 2)
    q = rows_of(2, 2, 2, dim, 3)
    check(attend(lib, q, cache, table, [70, 2147483647]), q, cache, table, [70, 2147483647], dim ** -0.5, "long")


def test_shared_pages(lib):
    """Two sequences with a common prefix read the same pages."""
    dim, page = 128, 16
    table, pages = tables([80, 40], page, 0, 1)
    table[1, :2] = table[0, :2]
    cache = filled(lib, pages, 2, page, dim, 2)
    q = rows_of(2, 1, 4, dim, 3)
    check(attend(lib, q, cache, table, [80, 40]), q, cache, table, [80, 40], dim ** -0.5, "shared")


def test_offsets_past_2_31_bytes(lib):
    heads, page, dim = 8, 128, 128
    pages = 2 ** 31 // (heads * page * dim) + 60
    say("cache past 2^31 bytes")
    cache = lib.kv_cache(pages, heads, page, dim)
    mark = 2 ** 31 // (heads * page * dim)
    at = torch.tensor([mark - 1, mark, pages - 1])
    small = filled(lib, 3, heads, page, dim, 3)
    for big, s in zip(cache, small):
        big[at.cuda()] = s
    lens = [3 * page - 5]
    q = rows_of(1, 1, heads, dim, 3)
    y = attend(lib, q, cache, at[None].to(torch.int32), lens)
    check(y, q, small, torch.arange(3, dtype=torch.int32)[None], lens, dim ** -0.5, "large")


def test_repeat_stream_and_graph(lib):
    """Same bytes on every call, on a side stream, and in every replay of a captured step (append, then attend)."""
    lens, tokens, dim, page = [1500, 700, 0], 1, 128, 64
    table, pages = tables(lens, page, 0, 1)
    cache = filled(lib, pages, 2, page, dim, 2)
    q, k, v = rows_of(3, tokens, 10, dim, 3), rows_of(3, tokens, 2, dim, 4), rows_of(3, tokens, 2, dim, 5)
    td, ld = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    need = lib.kv_attention_workspace_bytes(3, tokens, 10, 2, dim, page, table.shape[1])
    assert need > 0
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(3, tokens, 10, dim, dtype=torch.bfloat16, device="cuda")

    def step():
        lib.w8a8_kv_append(k, v, cache, td, ld)
        lib.w8a8_kv_attention(q, cache, td, ld, workspace=ws, out=out)

    step()
    torch.cuda.synchronize()
    first = out.clone()
    check(first, q, cache, table, lens, dim ** -0.5, "step")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out.fill_(float("nan"))
        step()
    side.synchronize()
    assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        out.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), f"replay {i}"
        (q.float() @ q.float().transpose(2, 3).contiguous()).sum().item()


def test_refusals(lib):
    cache = filled(lib, 4, 2, 16, 64, 1)
    table, lens = torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    q = rows_of(1, 1, 4, 64, 1)
    assert lib.w8a8_kv_attention(q, cache, table, lens).shape == (1, 1, 4, 64)
    assert lib.w8a8_kv_attention(q[:, :0], cache, table, lens).shape == (1, 0, 4, 64)
    assert lib.w8a8_kv_attention(q[:0], cache, table[:0], lens[:0]).shape == (0, 1, 4, 64)
    with pytest.raises(TypeError):
        lib.w8a8_kv_attention(q.half(), cache, table, lens)
    for bad in (q[..., :32], q[0], q.transpose(2, 3).contiguous().transpose(2, 3), q.cpu()):
        with pytest.raises(ValueError):
            lib.w8a8_kv_attention(bad, cache, table, lens)
    with pytest.raises(lib.W8A8Error):                        # 3 query heads for 2 cache heads
        lib.w8a8_kv_attention(rows_of(1, 1, 3, 64, 1), cache, table, lens)
    with pytest.raises(lib.W8A8Error):
        lib.w8a8_kv_attention(q, cache, table, lens, scale=float("nan"))
    with pytest.raises(ValueError):
        lib.w8a8_kv_attention(q, cache, table, lens, out=torch.empty(1, 1, 4, 32, dtype=torch.bfloat16, device="cuda"))
    big = torch.zeros(1, 300, dtype=torch.int32, device="cuda")
    assert lib.kv_attention_workspace_bytes(1, 1, 4, 2, 64, 16, 300) > 256
    with pytest.raises(ValueError):
        lib.w8a8_kv_attention(q, cache, big, lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))

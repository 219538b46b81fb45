"""Calls of more workgroups than one launch takes (2^32 threads: 2^24 workgroups of 256): every sequence is served, those
on both sides of the mark against the same sequences in a small call."""
import pytest
import torch

from parity import say
from test_gpu_kv_cache import filled

pytestmark = pytest.mark.gpu

HEADS, PAGE, DIM = 1024, 16, 64


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


def test_attention(lib):
    """2^14 + 5 sequences of one token, 1,024 heads: a workgroup for each, 2^24 of them and more."""
    seqs = (1 << 14) + 5
    say(f"attention of {seqs} sequences, {HEADS} heads")
    cache = filled(lib, 6, HEADS, PAGE, DIM, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    table = torch.randint(0, 6, (seqs, 2), generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(0, 33, (seqs,), generator=g, device="cuda").to(torch.int32)
    q = torch.randn(seqs, 1, HEADS, DIM, generator=g, device="cuda", dtype=torch.bfloat16)
    out = torch.full_like(q, float("nan"))
    lib.w8a8_kv_attention(q, cache, table, lens, out=out)
    assert not torch.isnan(out).any()
    for a in (0, 8190, (1 << 14) - 3):
        few = slice(a, a + 8)
        small = lib.w8a8_kv_attention(q[few], cache, table[few].contiguous().clone(), lens[few].clone())
        assert torch.equal(out[few].view(torch.int16), small.view(torch.int16)), a


def test_append(lib):
    """2^13 + 5 sequences of one token, keys and values of 1,024 heads; all but a few have no page, so drop it."""
    seqs = (1 << 13) + 5
    say(f"append of {seqs} sequences, {HEADS} heads")
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(seqs, 1, HEADS, DIM, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.full((seqs, 1), -1, dtype=torch.int32, device="cuda")
    held = torch.tensor([0, 4095, 4096, (1 << 13) - 2, (1 << 13) - 1, 1 << 13, seqs - 1], device="cuda")
    table[held, 0] = torch.arange(len(held), device="cuda").to(torch.int32)
    lens = torch.full((seqs,), 7, dtype=torch.int32, device="cuda")
    big, small = filled(lib, len(held), HEADS, PAGE, DIM, 4), filled(lib, len(held), HEADS, PAGE, DIM, 4)
    lib.w8a8_kv_append(k, v, big, table, lens)
    lib.w8a8_kv_append(k[held], v[held], small, table[held].contiguous(), lens[held].contiguous())
    for a, b in zip(big, small):
        assert torch.equal(a, b)
    assert not torch.equal(small.k_codes, filled(lib, len(held), HEADS, PAGE, DIM, 4).k_codes)


def test_read(lib):
    """2^20 sequences of 257 positions, 17 workgroups each: keys and values of 69 GB, read in two launches of 986,895
    sequences at most."""
    seqs, length, page, dim = 1 << 20, 257, 128, 128
    say(f"read of {seqs} sequences of {length}")
    cache = filled(lib, 5, 1, page, dim, 5)
    g = torch.Generator(device="cuda").manual_seed(6)
    table = torch.randint(0, 5, (seqs, 3), generator=g, device="cuda").to(torch.int32)
    lens = torch.randint(0, 300, (seqs,), generator=g, device="cuda").to(torch.int32)
    k, v = lib.w8a8_kv_read(cache, table, lens, length)
    for a in (0, 61679, 986892, seqs - 8):
        few = slice(a, a + 8)
        for big, small in zip((k, v), lib.w8a8_kv_read(cache, table[few].clone(), lens[few].clone(), length)):
            assert torch.equal(big[few], small), a
    del k, v
    torch.cuda.empty_cache()

"""Few-token calls on views as a program makes them: tables and lengths that begin in the middle of a larger tensor."""
import pytest
import torch

from test_gpu_kv_cache import filled, rows_of, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


@pytest.mark.parametrize("start", (1, 2, 3, 4))
def test_some_of_the_sequences(lib, start):
    """lens[start:] and table[start:] of an odd width (addresses that are not multiples of 16) give what copies give."""
    lens, page, dim = [40, 70, 33, 140, 16, 90], 32, 64
    table, pages = tables(lens, page, 1, 1)
    assert table.shape[1] % 4
    td, ld = table.cuda()[start:], torch.tensor(lens, dtype=torch.int32).cuda()[start:]
    q, k, v = (rows_of(len(lens), 2, h, dim, s) for h, s in ((4, 1), (2, 2), (2, 3)))
    one, two = filled(lib, pages, 2, page, dim, 4), filled(lib, pages, 2, page, dim, 4)
    got, want = [], []
    for cache, t, n, res in ((one, td, ld, got), (two, td.clone(), ld.clone(), want)):
        lib.w8a8_kv_append(k[start:], v[start:], cache, t, n)
        res += list(cache) + [lib.w8a8_kv_attention(q[start:], cache, t, n)] + list(lib.w8a8_kv_read(cache, t, n, 100))
    assert all(torch.equal(a, b) for a, b in zip(got, want))

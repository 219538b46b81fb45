"""The decoder layer on slices of a prompt: what it gives for a copy of them."""
import pytest
import torch

from test_gpu_decode import HIDDEN, paged
from test_gpu_layer_operators import FORMS, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    import w8a8_quantized_linear_amd as lib
    return lib


@pytest.mark.parametrize("form", [f[0] for f in FORMS])
@pytest.mark.parametrize("norms", ("weights", "functions", "none"))
def test_last_tokens_of_prompts(lib, form, norms):
    layer, rope = make(dict(FORMS)[form]), lib.rope(16)
    if norms != "weights":
        layer.norm1 = layer.norm2 = (lambda h: h * 2) if norms == "functions" else None
    x = torch.randn(2, 30, HIDDEN, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    delta = torch.randn(2, 30, HIDDEN, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    for one, two in ((x[:, -3:], delta[:, 2:5]), (x[:, -1:], None), (x[:, 7:8], delta[:, -1:])):
        lens = torch.full((2,), one.shape[1], dtype=torch.int32, device="cuda")
        (a, table), (b, _) = paged(lib, 2, 20), paged(lib, 2, 20)
        y, r = layer.step(one, two, a, table, lens, rotate=rope)
        z, s = layer.step(one.clone(memory_format=torch.contiguous_format), None if two is None else two.clone(memory_format=torch.contiguous_format),
                          b, table, lens, rotate=rope)
        assert torch.equal(y, z) and torch.equal(r, s)

"""Limits of the projections with block scales that the sizes of workspaces and the calls have to agree on (on the CPU)."""
import pytest

from test_abi import A, SHAPE
from test_layer_abi import lib  # noqa: F401 (a fixture)


@pytest.mark.parametrize("m,k,fits", ((1 << 25, 131072, True), ((1 << 25) + 32, 131072, False), (1 << 30, 4096, True), (1 << 30, 4096 + 128, False)))
def test_more_codes_than_a_workspace_holds(lib, m, k, fits):  # noqa: F811
    """x of up to 2^42 values; where the call refuses the shape there is no size for it."""
    assert (lib.w8a8_fp8_block_workspace_bytes(m, 16, k) > 0) == fits
    if not fits:
        assert lib.w8a8_fp8_block_linear_packed(A, A, A, None, A, m, 16, k, A, 1 << 62, None) == SHAPE

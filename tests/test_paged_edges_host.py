"""Host-side tests of the paged 8-bit KV cache at the ends of what its calls
accept (no GPU needed): what is refused is refused before any CUDA call."""
import pytest

import tiled_online_softmax_02_gb300 as attn
from test_paged_host import attend, lib  # noqa: F401  (lib is the module's fixture)


@pytest.mark.parametrize("block,width", [(16, 2 ** 27 - 1), (32, 2 ** 26 - 2), (64, 2 ** 25 - 1), (128, 2 ** 24)])
def test_tables_too_wide_for_32_bit_positions(lib, block, width):  # noqa: F811
    """Tiles of 128 keys are counted in 32 bits: a position rounded up to its tile's end has to fit."""
    assert 2 ** 31 - 128 < block * width
    assert attend(lib, block=block, width=width) == attn.ATTN_ERR_INVALID_ARG
    assert attend(lib, block=block, width=width, T=0) == attn.ATTN_ERR_INVALID_ARG
    widest = (2 ** 31 - 128) // block
    assert attend(lib, block=block, width=widest, T=0) == attn.ATTN_OK

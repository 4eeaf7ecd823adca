"""CPU tests of limits that the training step's calls state: sizes and rates."""
import os

import pytest

import fp8_moe_grouped_amd as G


def _lib():
    if not os.path.exists(G.LIB_PATH):
        pytest.skip("library not built")
    return G.lib()


@pytest.mark.parametrize("dtype", [G.F32, G.BF16])
def test_quantizer_workspace_is_what_a_cut_uses(dtype):
    """A word a column of each part.  Blocks keep 768 rows or more, of 128 columns in f32 384, which are taken for K up to
    9216 alone: no column has more than 24 parts."""
    L, n = _lib(), 2 * 256
    for K in range(128, 16384 + 1, 128):
        rows = 384 if dtype == G.F32 and K <= 9216 else 768
        parts = -(-K // rows)
        need = L.fp8gmm_workspace_bytes(G.OP_QUANT_WEIGHTS, 0, K, 256, 2, dtype)
        assert parts <= 24 and need == (4 * n * parts if parts > 1 else 0), K

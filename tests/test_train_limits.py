"""CPU tests of limits that the training step's calls state: sizes and rates."""
import os

import pytest
import torch

import fp8_moe_grouped_amd as G
from tests.test_train_abi import _adamw


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


LARGEST = float(torch.finfo(torch.float32).max)


@pytest.mark.parametrize("bits", [32, 8])
def test_rates_whose_coefficients_pass_f32(bits):
    """An infinite lr / (1 - beta1) makes NaN of parameters without a gradient, and an eps whose reciprocal is subnormal 0 of
    steps that are not: refused, with what is just inside answered (an empty tensor: nothing is launched)."""
    L = _lib()
    none = dict(size=0, p=None, g=None, m=None, v=None, ms=None, vs=None)
    for bad, fine in ((dict(eps=2.0 ** 126 * 1.001), dict(eps=2.0 ** 126)), (dict(eps=1e300), dict(eps=2.0 ** -126)),
                      (dict(lr=1e38, beta1=0.9), dict(lr=1e37, beta1=0.9)),
                      (dict(lr=LARGEST * 1.001, beta1=0.0), dict(lr=LARGEST, beta1=0.0)),
                      (dict(lr=1e30, weight_decay=1e9), dict(lr=1e30, weight_decay=1e8)),
                      (dict(lr=1.0, beta1=1 - 2.0 ** -53, weight_decay=1e39), dict(lr=1.0, beta1=1 - 2.0 ** -53))):
        assert _adamw(L, bits, **none, **bad) == G.ERR_UNSUPPORTED, bad
        assert _adamw(L, bits, **none, **fine) == G.OK, fine
    assert _adamw(L, bits, **none, lr=1e39, lr_dev=0x900000) == G.OK      # lr_dev's value is taken as it is

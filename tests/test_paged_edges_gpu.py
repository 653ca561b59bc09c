"""Paged-cache calls at their edges on the GPU: values at the ends of their types, the smallest
shapes, calls from several threads, tables and outputs that a caller got wrong."""
import numpy as np
import pytest

import test_paged_gpu as base

pytestmark = pytest.mark.gpu

# Head sizes and pool alignments that take each of the kernels: tensor cores, and rows of no whole 16 bytes.
LAYOUTS = [(64, 0), (128, 0), (256, 0), (64, 1)]


@pytest.mark.parametrize("hd,pool_off", LAYOUTS)
def test_attn_keeps_all_bits_of_large_f32_keys(qkv, hd, pool_off):
    """Keys of 1e34 and both signs: the part below their leading 11 bits is above 1e30 itself.  q is small, so the
    scores are ordinary; the bound is that of ordinary keys (the remainders of q, 2^-12 * 1e-34, are normal
    numbers)."""
    def large(c, x):
        c.k *= np.float32(1e34)
        x *= np.float32(1e-34)

    base.run_attn(4, 2, hd, "f32", 16, [40, 90], change=large, pool_off=pool_off, weights=True)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hd,pool_off", LAYOUTS)
def test_attn_infinite_key_against_a_large_query(qkv, hd, pool_off, sign):
    """A score of -inf from an infinite f32 key of either sign has weight 0, however large the query element that
    makes it is (the element's other keys are 0, so all other scores are ordinary)."""
    def change(c, x):
        c.k[..., 3] = 0
        x[0, 3], x[0, hd + 3] = -sign * 1e12, -sign * 3e20  # both q heads of kv head 0
        c.k[c.row(0, 5)][3] = sign * np.inf

    base.run_attn(4, 2, hd, "f32", 16, [40, 90], change=change, pool_off=pool_off)

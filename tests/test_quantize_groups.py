"""Group quantisation of the synthetic weights: group by group the same as the
per-tensor quantiser, and round trips.  No GPU needed."""
import numpy as np
import pytest

from lossless_entropy_coded_huffman_amd import synth


@pytest.mark.parametrize("asymmetric", [False, True])
@pytest.mark.parametrize("rows,cols,group", [(3, 64, 32), (5, 72, 32), (2, 40, 40), (1, 128, 64), (4, 8, 32)])
def test_each_group_is_quantised_as_a_tensor(rows, cols, group, asymmetric):
    x = np.random.default_rng(rows * cols).normal(0, 0.02, (rows, cols)).astype(np.float32)
    codes, scales, zeros = synth.quantize_u4_groups(x, group, asymmetric)
    assert scales.shape == zeros.shape == (rows, -(-cols // group)) and codes.shape == x.shape
    for r in range(rows):
        for g in range(scales.shape[1]):
            part = slice(g * group, (g + 1) * group)
            assert np.array_equal(codes[r, part], synth.quantize_u4(x[r, part], asymmetric))
    assert codes.max() <= 15 and np.isfinite(scales).all() and (scales > 0).all()


def test_constant_rows_and_bits():
    codes, scales, zeros = synth.quantize_u4_groups(np.zeros((2, 32), np.float32), 32, False)
    assert (codes == 8).all() and (scales == 1).all() and (zeros == 8).all()
    codes, scales, zeros = synth.quantize_u4_groups(np.full((2, 32), 0.5, np.float32), 32, True)
    assert (scales == 1).all()
    x = np.random.default_rng(0).normal(0, 1, 1000).astype(np.float32)
    b = synth.bf16_rne(x)
    assert np.array_equal(synth.bf16_rne(synth.bf16_to_f32(b)), b)

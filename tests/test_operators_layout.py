"""How inputs are laid out for the operators' kernels: rows that are kept as they
are, and strides that need a copy.  No GPU needed."""
import pytest
import torch

from lossless_entropy_coded_huffman_amd import ops


def wide(rows, cols, step, offset=0):
    """A [rows, cols] view of row stride `step`; the storage holds only zeros."""
    return torch.zeros((rows - 1) * step + cols + offset, dtype=torch.bfloat16)[offset:].as_strided((rows, cols), (step, 1), offset)


@pytest.mark.parametrize("t,kept", [
    (torch.zeros(3, 64, dtype=torch.float16), True),
    (wide(3, 64, 72), True),
    (wide(2, 64, 1 << 21), True),                       # the largest stride
    (wide(2, 64, (1 << 21) + 8), False),                # the last token of a long prompt
    (wide(3, 64, 68), False),
    (wide(3, 64, 64, 4), False),                        # 8-byte aligned
    (torch.zeros(64, 1, dtype=torch.float16).t(), False),   # one row: contiguous, with a stride of 1
    (torch.zeros(64, 3, dtype=torch.float16).t(), False),
    (torch.zeros(1, 64, dtype=torch.float16).expand(5, 64), False),
    (torch.zeros(0, 64, dtype=torch.float16), True),
])
def test_rows(t, kept):
    r = ops._rows16(t)
    assert (r is t) == kept
    assert r.shape == t.shape and torch.equal(r, t)
    step, one = r.stride()
    assert one == 1 and step % 8 == 0 and t.shape[1] <= step <= 1 << 21 and r.data_ptr() % 16 == 0


def test_copies_have_contiguous_strides():
    assert ops._copied(torch.zeros(7, 1).t()).stride() == (7, 1)

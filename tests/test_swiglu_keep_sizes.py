"""The sizes that ep_swiglu_keep and its backward pass take are the documented ones: rows * inner_size / 128 < 2^31."""
import pytest
import torch

from combine_ep_layout_03_gb300 import ep

A, B, C, D = (1 << 40), (1 << 41), (1 << 42), (1 << 43)   # never dereferenced


def keep(rows, inner):
    return ep.lib.ep_swiglu_keep(A, None, rows, inner, None, B, C, D, None)


def keep_grad(rows, inner):
    return ep.lib.ep_swiglu_keep_grad(A, B, None, C, rows, inner, None, D, None, None, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="a call that is accepted would be launched")
@pytest.mark.parametrize("call", [keep, keep_grad])
@pytest.mark.parametrize("inner", [128, 256, 384, 1024, 65536])
def test_the_largest_sizes(call, inner):
    most = (2 ** 31 - 1) // (inner // 128)
    for rows in (most, most - 1, most - 63):
        assert call(rows, inner) == ep.EP_ERR_CUDA   # accepted, and there is no device
    assert call(most + 1, inner) == ep.EP_ERR_INVALID_ARG


@pytest.mark.parametrize("groups", [1, 2, 3, 8, 512])
def test_units_of_the_largest_sizes(groups):
    """The forward kernel's indexes: 32 units a CTA, in 32 bits, of which those outside the rows are left out."""
    rows = (2 ** 31 - 1) // groups
    last = (rows * groups + 31) // 32 * 32 - 1
    assert last < 2 ** 31 and last // groups >= rows - 1
    for unit in range(last - 64, last + 1):
        row = unit // groups
        assert (row < rows) == (unit < rows * groups) and row < 2 ** 31

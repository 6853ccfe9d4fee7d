"""The largest operands of the layer operators, where the host has to refuse them (CPU only: nothing is enqueued)."""
import ctypes
import os

import pytest

import nvfp4_block_scaled_elem_amd as nv
from nvfp4_block_scaled_elem_amd import build as nvbuild
from nvfp4_block_scaled_elem_amd import layer

INVALID, SHAPE = -1, -2
FAKE = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        nvbuild.build()
    return nv.lib()


@pytest.mark.parametrize("rows,cols", [(1, (1 << 35) - 32), (1, (1 << 35) - 2047), (3, 11453246112)])
def test_operands_whose_grid_would_overflow(L, rows, cols):
    """The codec takes a thread per eight columns, in work-groups of 256: from 2^35 - 2^11 values on (columns counted in
    whole blocks of 32) that is a grid of 2^32 threads, one more than a launch can have."""
    assert rows * -(-cols // 32) * 32 > (1 << 35) - (1 << 11)
    assert L.nvfp4_mxfp8_quantize(FAKE, cols, 0, rows, cols, FAKE, FAKE, None) == SHAPE
    assert L.nvfp4_mxfp8_dequantize(FAKE, cols, FAKE, rows, cols, FAKE, 0, None) == SHAPE
    assert L.nvfp4_rms_norm(FAKE, cols, None, 0, FAKE, 0, 0, rows, cols, 1e-6, None, FAKE, None, 0, None) == SHAPE


def test_a_product_whose_input_is_decoded_keeps_to_the_same_bound(L):
    m, k = (1 << 23) - 1, 4096
    a = layer._LinearArgs(x=FAKE, ldx=k, x_scales=FAKE, x_dtype=2, M=m, K=k, N=16, codes=FAKE, scales=FAKE, alpha=FAKE,
                          y=FAKE, workspace=FAKE, workspace_bytes=0)
    assert m * k == (1 << 35) - 4096 and L.nvfp4_linear_workspace_bytes(m, k, 16, 2, 0, 0) > 0  # the largest of these
    a.M = m + 1
    assert L.nvfp4_linear(ctypes.byref(a)) == SHAPE

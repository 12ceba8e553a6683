"""Sizes of the bias gradients' sums in nvfp4_linear_backward's workspace (CPU, no call reaches a kernel)."""
import os

import pytest
import torch

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "block_scale_search_amd", "libnvfp4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libnvfp4.so not built")


@pytest.mark.parametrize("T, E, out", [(4, 1024, 16392), (512, 1024, 28672), (0, 1024, 28672), (1023, 1024, 28672),
                                       (1024, 1024, 28672), (100, 128, 131080), (8, 2048, 8200), (0, 8, 2100000),
                                       (65534, 65535, 8191)])
def test_many_biases_of_few_rows_have_a_share(T, E, out):
    """More than 2^24 biases and fewer rows than matrices: at least one sum for each bias."""
    from block_scale_search_amd import nvfp4 as nv
    need = nv.nvfp4_linear_backward_workspace_size
    for dtype in (torch.bfloat16, torch.float32):
        assert need(dtype, T, E, out, 16, True) - need(dtype, T, E, out, 16, False) >= E * out * 4
